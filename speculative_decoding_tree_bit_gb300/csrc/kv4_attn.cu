// Attention over the 4-bit cache, and the weight its keys collect.
#include <algorithm>

#include "kv4.cuh"

namespace sdv {

struct Kv4AttnArgs {
  Kv4View c;
  Kv4Score s;
  const uint16_t* q;
  int64_t q_stride, kv_stride;
  const uint16_t* k_new;
  const uint16_t* v_new;
  const int32_t* cu;
  const uint64_t* anc;
  const int32_t* row_pos;
  int R, hq, G;
  uint16_t* out;
  float* lse;
  int32_t* status;
};

__device__ __forceinline__ float nib(uint32_t byte, int d) { return (float)(int)((byte >> (4 * (d & 1))) & 15) - 8.f; }

__device__ __forceinline__ float kv4_score(const Kv4Score& s, float qk, float slope, int q_pos, int k_pos, int start) {
  float t = qk * s.scale;
  if (s.cap > 0.f) t = s.cap * tanhf(t / s.cap);
  if (s.slopes) t = fmaf(slope, (float)(k_pos - q_pos), t);
  if ((s.window > 0 && q_pos - k_pos >= s.window) || k_pos < start) t = -INFINITY;
  return t;
}

// One CTA per (row, query head): a thread per key for the scores, a thread
// per dim for the values.  Right for every case, and the measure of the rest.
template <int D>
__global__ void __launch_bounds__(128) k_kv4_attn_simple(Kv4AttnArgs a) {
  __shared__ float sq[D], sp[128], red[4];
  const int e = blockIdx.x, hq = blockIdx.y, h = hq / a.G, tid = threadIdx.x;
  int r = 0;
  while (r + 1 < a.R && a.cu[r + 1] <= e) r++;
  const int n0 = a.cu[r], i = e - n0, m = a.cu[r + 1] - n0;
  int ctx = a.c.ctx_len[r];
  if (ctx < 0 || ctx > a.c.cap) {
    if (tid == 0) set_status(a.status, SD_ERR_CAPACITY);
    ctx = ctx < 0 ? 0 : (int)a.c.cap;
  }
  if (tid < D) sq[tid] = bf2f(a.q[(int64_t)e * a.q_stride + hq * D + tid]);
  __syncthreads();
  const int qp = a.row_pos ? a.row_pos[e] : ctx + i;
  const int p0 = a.row_pos ? a.row_pos[n0] : ctx;
  const float slope = a.s.slopes ? a.s.slopes[hq] : 0.f;
  const int start = a.s.start ? a.s.start[r] : INT32_MIN;
  const int first = kv4_first(a.s, r, ctx, p0);
  const uint64_t sees = a.anc ? a.anc[e] : (2ull << i) - 1;
  const int own = a.k_new ? m : 0;
  float mx = -INFINITY, l = 0.f, o = 0.f;
  for (int base = first; base < ctx + own; base += 128) {
    const int t = base + tid;
    float sc = -INFINITY;
    if (t < ctx) {
      const uint8_t* rec = a.c.record(D, r, h, t / 32);
      if (!rec) {
        set_status(a.status, SD_ERR_CAPACITY);
      } else {
        const uint32_t sm = *reinterpret_cast<const uint32_t*>(rec + 16 * D + (t & 31) * 4);
        float dot = 0.f, qs = 0.f;
        for (int d = 0; d < D; d++) {
          dot = fmaf(sq[d], nib(rec[(t & 31) * (D / 2) + d / 2], d), dot);
          qs += sq[d];
        }
        dot = fmaf(bf2f((uint16_t)sm), dot, bf2f((uint16_t)(sm >> 16)) * qs);
        sc = kv4_score(a.s, dot, slope, qp, a.c.pos[a.c.slot0(r, h) + t], start);
      }
    } else if (t < ctx + own && (sees >> (t - ctx) & 1)) {
      const int j = n0 + t - ctx;
      float dot = 0.f;
      for (int d = 0; d < D; d++) dot = fmaf(sq[d], bf2f(a.k_new[(int64_t)j * a.kv_stride + h * D + d]), dot);
      sc = kv4_score(a.s, dot, slope, qp, a.row_pos ? a.row_pos[j] : ctx + t - ctx, start);
    }
    float w = sc;
    for (int x = 16; x > 0; x >>= 1) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, x));
    if ((tid & 31) == 0) red[tid >> 5] = w;
    __syncthreads();
    const float mn = fmaxf(mx, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float ms = mn == -INFINITY ? 0.f : mn;
    const float al = __expf(mx - ms);
    sp[tid] = __expf(sc - ms);
    __syncthreads();
    mx = mn;
    l *= al;
    o *= al;
    for (int j = 0; j < 128 && base + j < ctx + own; j++) {
      const float p = sp[j];
      l += p;
      if (p == 0.f || tid >= D) continue;
      const int u = base + j;
      float val;
      if (u < ctx) {
        const uint8_t* rec = a.c.record(D, r, h, u / 32) + kv4_half(D);
        const uint32_t sm = *reinterpret_cast<const uint32_t*>(rec + 16 * D + (u & 31) * 4);
        val = fmaf(bf2f((uint16_t)sm), nib(rec[(u & 31) * (D / 2) + kv4_vbyte<D>(u, tid / 2)], tid),
                   bf2f((uint16_t)(sm >> 16)));
      } else {
        val = bf2f(a.v_new[(int64_t)(n0 + u - ctx) * a.kv_stride + h * D + tid]);
      }
      o = fmaf(p, val, o);
    }
    __syncthreads();
  }
  if (tid < D) a.out[((int64_t)e * a.hq + hq) * D + tid] = f2bf(l > 0.f ? o / l : l == 0.f ? 0.f : l);
  if (tid == 0 && a.lse) a.lse[(int64_t)e * a.hq + hq] = l == 0.f ? -INFINITY : mx + logf(l);
}

struct Kv4ObserveArgs {
  Kv4AttnArgs a;
  const float* lse_in;
  const float* row_weight;
  float decay;
  float* out;
};

// One thread per slot of a (request, kv head), over every row and query head.
template <int D>
__global__ void __launch_bounds__(128) k_kv4_observe_simple(Kv4ObserveArgs b) {
  const Kv4AttnArgs& a = b.a;
  __shared__ float sq[D];
  const int h = blockIdx.y, r = blockIdx.z, tid = threadIdx.x;
  int ctx = a.c.ctx_len[r];
  if (ctx < 0 || ctx > a.c.cap) {
    if (tid == 0) set_status(a.status, SD_ERR_CAPACITY);
    ctx = ctx < 0 ? 0 : (int)a.c.cap;
  }
  const int n0 = a.cu[r], m = a.cu[r + 1] - n0;
  const int start = a.s.start ? a.s.start[r] : INT32_MIN;
  for (int base = blockIdx.x * 128; base < ctx; base += gridDim.x * 128) {
    const int t = base + tid;
    const uint8_t* rec = t < ctx ? a.c.record(D, r, h, t / 32) : nullptr;
    if (t < ctx && !rec) set_status(a.status, SD_ERR_CAPACITY);
    const int kp = t < ctx ? a.c.pos[a.c.slot0(r, h) + t] : 0;
    float sum = 0.f;
    for (int i = 0; i < m; i++) {
      const float rw = b.row_weight ? b.row_weight[n0 + i] : 1.f;
      if (rw == 0.f) continue;
      const int qp = a.row_pos ? a.row_pos[n0 + i] : ctx + i;
      for (int gq = 0; gq < a.G; gq++) {
        const int hq = h * a.G + gq;
        __syncthreads();
        if (tid < D) sq[tid] = bf2f(a.q[(int64_t)(n0 + i) * a.q_stride + hq * D + tid]);
        __syncthreads();
        const float lse = b.lse_in[(int64_t)(n0 + i) * a.hq + hq];
        if (!rec || lse == -INFINITY) continue;
        const uint32_t sm = *reinterpret_cast<const uint32_t*>(rec + 16 * D + (t & 31) * 4);
        float dot = 0.f, qs = 0.f;
        for (int d = 0; d < D; d++) {
          dot = fmaf(sq[d], nib(rec[(t & 31) * (D / 2) + d / 2], d), dot);
          qs += sq[d];
        }
        dot = fmaf(bf2f((uint16_t)sm), dot, bf2f((uint16_t)(sm >> 16)) * qs);
        const float sc = kv4_score(a.s, dot, a.s.slopes ? a.s.slopes[hq] : 0.f, qp, kp, start);
        sum = fmaf(rw, __expf(sc - lse), sum);
      }
    }
    if (t < ctx) {
      const int64_t o = a.c.slot0(r, h) + t;
      b.out[o] = fmaf(b.decay, a.c.weight[o], sum);
    }
  }
}

// ---------------------------------------------------------------- checks --

static int check_call(const char* who, const sd_kv4* c, const uint16_t* q, int64_t q_stride, int32_t hq,
                      const int32_t* cu, const int32_t* cu_host, int32_t R, const sd_kv4_score* score, int32_t max_ctx,
                      Kv4AttnArgs* a) {
  if (int rc = kv4_check(c, R, who, &a->c)) return rc;
  if (int rc = kv4_check_rows(cu, cu_host, R, who)) return rc;
  if (int rc = kv4_check_score(score, who, &a->s, c->head_dim)) return rc;
  if (!q || (reinterpret_cast<uintptr_t>(q) & 15)) return kv4_bad(SD_ERR_INVALID_ARG, who, "q must be set and 16-byte aligned");
  if (hq < c->n_kv_heads || hq % c->n_kv_heads)
    return kv4_bad(SD_ERR_INVALID_ARG, who, "n_q_heads must be a multiple of n_kv_heads");
  if (hq / c->n_kv_heads > 16) return kv4_bad(SD_ERR_UNSUPPORTED, who, "at most 16 query heads a kv head");
  if (q_stride < (int64_t)hq * c->head_dim || q_stride % 8)
    return kv4_bad(SD_ERR_INVALID_ARG, who, "q_stride must cover a row and be a multiple of 8");
  if (max_ctx < 0) return kv4_bad(SD_ERR_INVALID_ARG, who, "max_ctx must not be negative");
  for (int r = 0; r < R; r++)
    if (cu_host[r + 1] - cu_host[r] > 64) return kv4_bad(SD_ERR_UNSUPPORTED, who, "at most 64 rows a request");
  a->q = q;
  a->q_stride = q_stride;
  a->cu = cu;
  a->R = R;
  a->hq = hq;
  a->G = hq / c->n_kv_heads;
  return SD_OK;
}

}  // namespace sdv

using namespace sdv;

extern "C" size_t sd_kv4_attn_workspace(int32_t R, int32_t rows, int32_t n_q_heads, int32_t n_kv_heads,
                                        int32_t head_dim) {
  if (R < 1 || rows < 0 || n_kv_heads < 1 || n_q_heads < n_kv_heads || n_q_heads % n_kv_heads ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  return 256;
}

extern "C" int sd_kv4_attn(const sd_kv4* c, const uint16_t* q, int64_t q_stride, int32_t n_q_heads, const int32_t* cu,
                           const int32_t* cu_host, int32_t R, const uint16_t* k_new, const uint16_t* v_new,
                           int64_t kv_stride, const uint64_t* anc, const int32_t* row_pos, const sd_kv4_score* score,
                           int32_t max_ctx, uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                           int32_t* status, void* stream) {
  const char* who = "sd_kv4_attn";
  Kv4AttnArgs a = {};
  if (int rc = check_call(who, c, q, q_stride, n_q_heads, cu, cu_host, R, score, max_ctx, &a)) return rc;
  if (!out || (reinterpret_cast<uintptr_t>(out) & 15)) return kv4_bad(SD_ERR_INVALID_ARG, who, "out must be set and 16-byte aligned");
  if (!k_new != !v_new) return kv4_bad(SD_ERR_INVALID_ARG, who, "k_new and v_new go together");
  if (k_new) {
    if (((reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) & 15) ||
        kv_stride < (int64_t)c->n_kv_heads * c->head_dim || kv_stride % 8)
      return kv4_bad(SD_ERR_INVALID_ARG, who,
                     "k_new and v_new must be 16-byte aligned, kv_stride must cover a row and be a multiple of 8");
  }
  const int rows = cu_host[R];
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return kv4_bad(SD_ERR_INVALID_ARG, who, "workspace must be set and 256-byte aligned");
  if (workspace_bytes < sd_kv4_attn_workspace(R, rows, n_q_heads, c->n_kv_heads, c->head_dim))
    return kv4_bad(SD_ERR_WORKSPACE, who, "workspace too small");
  if (rows == 0) return SD_OK;
  a.k_new = k_new;
  a.v_new = v_new;
  a.kv_stride = kv_stride;
  a.anc = anc;
  a.row_pos = row_pos;
  a.out = out;
  a.lse = lse;
  a.status = status;
  auto kern = c->head_dim == 128 ? k_kv4_attn_simple<128> : k_kv4_attn_simple<64>;
  kern<<<dim3(rows, n_q_heads), 128, 0, (cudaStream_t)stream>>>(a);
  SD_CK(cudaGetLastError());
  return SD_OK;
}

extern "C" int sd_kv4_observe(const sd_kv4* c, const uint16_t* q, int64_t q_stride, int32_t n_q_heads,
                              const float* lse, const int32_t* cu, const int32_t* cu_host, int32_t R,
                              const int32_t* row_pos, const float* row_weight, const sd_kv4_score* score,
                              int32_t max_ctx, float decay, float* weight_out, int32_t* status, void* stream) {
  const char* who = "sd_kv4_observe";
  Kv4ObserveArgs b = {};
  if (int rc = check_call(who, c, q, q_stride, n_q_heads, cu, cu_host, R, score, max_ctx, &b.a)) return rc;
  if (!lse) return kv4_bad(SD_ERR_INVALID_ARG, who, "null lse");
  if (!weight_out || (reinterpret_cast<uintptr_t>(weight_out) & 15))
    return kv4_bad(SD_ERR_INVALID_ARG, who, "weight_out must be set and 16-byte aligned");
  if (!(decay >= 0.f) || !(decay <= 1e30f)) return kv4_bad(SD_ERR_INVALID_ARG, who, "decay must be finite and not negative");
  b.a.row_pos = row_pos;
  b.a.status = status;
  b.lse_in = lse;
  b.row_weight = row_weight;
  b.decay = decay;
  b.out = weight_out;
  const int64_t most = max_ctx > 0 ? std::min<int64_t>(max_ctx, b.a.c.cap) : b.a.c.cap;
  const unsigned gx = (unsigned)std::max<int64_t>(1, std::min<int64_t>((most + 127) / 128, 1024));
  auto kern = c->head_dim == 128 ? k_kv4_observe_simple<128> : k_kv4_observe_simple<64>;
  kern<<<dim3(gx, c->n_kv_heads, R), 128, 0, (cudaStream_t)stream>>>(b);
  SD_CK(cudaGetLastError());
  return SD_OK;
}
