// Causal attention over packed prompts.
#include "kv4_attn.cuh"

namespace sdv {

struct PromptArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, kv_stride;
  int hq, hkv, G, R;
  const int32_t* cu_q;
  const int32_t* cu_k;
  Kv4Score s;
  uint16_t* out;
  float* lse;
};

// A warp per row and query head, D / 32 dims a lane, one key at a time.
template <int D>
__global__ void __launch_bounds__(256) k_prompt_attn(PromptArgs a, int rows) {
  const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= (int64_t)rows * a.hq) return;
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31, row = (int)(i / a.hq), h = (int)(i - (int64_t)row * a.hq);
  const int r = request_of(a.cu_q, a.R, row);
  const int m = a.cu_q[r + 1] - a.cu_q[r], n = a.cu_k[r + 1] - a.cu_k[r];
  const int p = n - m + row - a.cu_q[r];
  float q[N], o[N] = {};
  for (int d = 0; d < N; d++) q[d] = bf2f(a.q[row * a.q_stride + h * D + lane * N + d]);
  float top = -INFINITY, l = 0.f;
  const float slope = a.s.slopes ? a.s.slopes[h] * kLog2e : 0.f;
  for (int j = a.s.window > 0 ? max(0, p - a.s.window + 1) : 0; j <= p; j++) {
    const int64_t at = (int64_t)(a.cu_k[r] + j) * a.kv_stride + h / a.G * D + lane * N;
    float x[1] = {0.f};
    for (int d = 0; d < N; d++) x[0] += q[d] * bf2f(a.k[at + d]);
    for (int e = 16; e > 0; e >>= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], e);
    float y[2] = {x[0], x[0]};
    kv4_cap(a.s, y);
    const float t = fmaf(slope, (float)(j - p), y[0]);
    const float up = fmaxf(top, t), us = up == -INFINITY ? 0.f : up;
    const float f = ex2(top - us), w = ex2(t - us);
    l = l * f + w;
    for (int d = 0; d < N; d++) o[d] = o[d] * f + w * bf2f(a.v[at + d]);
    top = up;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  for (int d = 0; d < N; d++) a.out[i * D + lane * N + d] = f2bf(o[d] * inv);
  if (lane == 0 && a.lse) a.lse[i] = l == 0.f ? -INFINITY : (top + log2f(l)) * (1.f / kLog2e);
}

}  // namespace sdv

using namespace sdv;

extern "C" size_t sd_prompt_attn_workspace(int32_t head_dim) {
  return head_dim == 64 || head_dim == 128 ? 256 : 0;
}

extern "C" int sd_prompt_attn(const uint16_t* q, int64_t q_stride, int32_t n_q_heads, const uint16_t* k, const uint16_t* v,
                              int64_t kv_stride, int32_t n_kv_heads, int32_t head_dim, const int32_t* cu_q,
                              const int32_t* cu_q_host, const int32_t* cu_k, const int32_t* cu_k_host, int32_t R,
                              const sd_kv4_score* score, uint16_t* out, float* lse, void* workspace,
                              size_t workspace_bytes, int32_t* status, void* stream) {
  const char* who = "sd_prompt_attn";
  if (head_dim != 64 && head_dim != 128) return kv4_bad(SD_ERR_UNSUPPORTED, who, "head_dim must be 64 or 128");
  if (n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads || n_q_heads / n_kv_heads > 128)
    return kv4_bad(SD_ERR_UNSUPPORTED, who, "n_q_heads must be a multiple of n_kv_heads, at most 128 a kv head");
  if (R < 1) return kv4_bad(SD_ERR_INVALID_ARG, who, "R must be at least 1");
  if (int rc = kv4_check_rows(cu_q, cu_q_host, R, who)) return rc;
  if (!cu_k != !cu_k_host) return kv4_bad(SD_ERR_INVALID_ARG, who, "cu_k and cu_k_host go together");
  if (!cu_k) cu_k = cu_q, cu_k_host = cu_q_host;
  if (int rc = kv4_check_rows(cu_k, cu_k_host, R, who)) return rc;
  PromptArgs a = {};
  if (int rc = kv4_check_score(score, who, &a.s, head_dim)) return rc;
  if (a.s.start) return kv4_bad(SD_ERR_INVALID_ARG, who, "score->start must be null: requests are packed");
  const int rows = cu_q_host[R], keys = cu_k_host[R];
  if (rows == 0) return SD_OK;
  if (!q || !out || (keys && (!k || !v))) return kv4_bad(SD_ERR_INVALID_ARG, who, "null argument");
  if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)out) & 15)
    return kv4_bad(SD_ERR_INVALID_ARG, who, "q, k, v and out must be 16-byte aligned");
  if (q_stride < (int64_t)n_q_heads * head_dim || q_stride % 8 || kv_stride < (int64_t)n_kv_heads * head_dim || kv_stride % 8)
    return kv4_bad(SD_ERR_INVALID_ARG, who, "strides must cover a row and be multiples of 8");
  if (!workspace || ((uintptr_t)workspace & 255)) return kv4_bad(SD_ERR_INVALID_ARG, who, "workspace must be set and 256-byte aligned");
  if (workspace_bytes < sd_prompt_attn_workspace(head_dim)) return kv4_bad(SD_ERR_WORKSPACE, who, "workspace too small");
  a.q = q, a.k = k, a.v = v, a.q_stride = q_stride, a.kv_stride = kv_stride;
  a.hq = n_q_heads, a.hkv = n_kv_heads, a.G = n_q_heads / n_kv_heads, a.R = R;
  a.cu_q = cu_q, a.cu_k = cu_k, a.out = out, a.lse = lse;
  const int64_t blocks = ((int64_t)rows * n_q_heads + 7) / 8;
  if (blocks > 0x7FFFFFFF) return kv4_bad(SD_ERR_UNSUPPORTED, who, "too many rows");
  (head_dim == 128 ? k_prompt_attn<128> : k_prompt_attn<64>)<<<(unsigned)blocks, 256, 0, (cudaStream_t)stream>>>(a, rows);
  SD_CK(cudaGetLastError());
  return SD_OK;
}
