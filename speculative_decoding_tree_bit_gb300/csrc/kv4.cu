// The 4-bit key/value cache: storing rows, reading them back, eviction.
#include "kv4.cuh"

namespace sdv {

// ---------------------------------------------------------------- append --
//
// One warp stores the key and the value row of one (row, kv head): a half
// warp each, D / 16 values a lane (one or half a 32-bit word of codes).  The
// row's least and greatest value come from four shuffles.  Bound: bytes (4 D
// in, D + 12 out per row and head).

// The row of a call that entry e is, by a search over the request offsets.
__device__ __forceinline__ int request_of(const int32_t* __restrict__ cu, int R, int e) {
  int lo = 0, hi = R;  // cu[lo] <= e < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= e) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <int D>
__global__ void __launch_bounds__(256) k_kv4_append(Kv4View c, const uint16_t* __restrict__ k,
                                                    const uint16_t* __restrict__ v, int64_t row_stride, int n_src,
                                                    const int32_t* __restrict__ cu, int R, int rows,
                                                    const int32_t* __restrict__ src, const int32_t* __restrict__ count,
                                                    const int32_t* __restrict__ pos, const int32_t* at, bool advance,
                                                    int32_t* status) {
  constexpr int kV = D / 16;  // values of a lane
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= (int64_t)rows * c.hkv) return;
  const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
  const int e = (int)(w / c.hkv), h = (int)(w - (int64_t)e * c.hkv);
  const int r = request_of(cu, R, e);
  const int i = e - cu[r];
  const int n = count ? min(max(count[r], 0), cu[r + 1] - cu[r]) : cu[r + 1] - cu[r];
  const int a = at[r];
  if (a < 0 || (int64_t)a + n > c.cap) {
    if (lane == 0) set_status(status, SD_ERR_CAPACITY);
    return;
  }
  if (i == 0 && h == 0 && lane == 0 && advance) c.ctx_len[r] = a + n;
  if (i >= n) return;
  const int s = src ? src[e] : e;
  if (s < 0 || s >= n_src) {
    if (lane == 0) set_status(status, SD_ERR_CAPACITY);
    return;
  }
  const int t = a + i;
  uint8_t* rec = c.record(D, r, h, t / kKvGroup);
  if (!rec) {
    if (lane == 0) set_status(status, SD_ERR_CAPACITY);
    return;
  }
  const uint16_t* x = (half ? v : k) + (int64_t)s * row_stride + h * D + l * kV;
  uint32_t raw[kV / 2];
  if constexpr (kV == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(x);
    raw[0] = u.x, raw[1] = u.y, raw[2] = u.z, raw[3] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(x);
    raw[0] = u.x, raw[1] = u.y;
  }
  float f[kV], lo = INFINITY, hi = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int j = 0; j < kV; j++) {
    f[j] = bf2f((uint16_t)(raw[j >> 1] >> (16 * (j & 1))));
    lo = fminf(lo, f[j]);
    hi = fmaxf(hi, f[j]);
    nan |= f[j] != f[j];  // fminf and fmaxf pass NaN over
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const uint32_t bad = __ballot_sync(0xffffffffu, nan) >> (16 * half) & 0xFFFFu;
  const float range = hi - lo;
  float sc = rbf(__fdiv_rn(range, 15.f)), md = rbf(fmaf(8.f, sc, lo));
  if (bad || !(range <= 3.4028234e38f)) sc = md = __int_as_float(0x7FC00000);  // not finite: the row is held as NaN
  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < kV; j++) {
    // the quotient is a true division: a product with 1 / s could fall on the
    // other side of a half.  NaN and s = 0 give code 8.
    const float qf = sc > 0.f ? rintf(__fdiv_rn(f[j] - md, sc)) : 0.f;
    word |= (uint32_t)((int)fminf(fmaxf(qf, -8.f), 7.f) + 8) << (4 * j);
  }
  uint8_t* codes = rec + half * kv4_half(D) + (t & 31) * (D / 2);
  const int b = half ? kv4_vbyte<D>(t, l * (kV / 2)) : l * (kV / 2);
  if constexpr (kV == 8) *reinterpret_cast<uint32_t*>(codes + b) = word;
  else *reinterpret_cast<uint16_t*>(codes + b) = (uint16_t)word;
  if (l == 0) {
    *reinterpret_cast<uint32_t*>(rec + half * kv4_half(D) + 16 * D + (t & 31) * 4) =
        (uint32_t)f2bf(sc) | (uint32_t)f2bf(md) << 16;
    const int64_t o = c.slot0(r, h) + t;
    if (half) c.weight[o] = 0.f;
    else c.pos[o] = pos ? pos[e] : t;
  }
}

// ctx_len[r] += the rows stored, once they are (append in place).
__global__ void k_kv4_advance(int32_t* ctx_len, const int32_t* __restrict__ cu, const int32_t* __restrict__ count,
                              int R, int64_t cap) {
  const int r = blockIdx.x * blockDim.x + threadIdx.x;
  if (r >= R) return;
  const int n = count ? min(max(count[r], 0), cu[r + 1] - cu[r]) : cu[r + 1] - cu[r];
  const int a = ctx_len[r];
  if (a >= 0 && (int64_t)a + n <= cap) ctx_len[r] = a + n;
}

// ------------------------------------------------------------------ read --
//
// The warp and lane shape of the append, the other way.
template <int D>
__global__ void __launch_bounds__(256) k_kv4_read(Kv4View c, const int32_t* __restrict__ cu, int R, int rows,
                                                  const int32_t* __restrict__ at, uint16_t* __restrict__ k_out,
                                                  uint16_t* __restrict__ v_out, int32_t* status) {
  constexpr int kV = D / 16;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= (int64_t)rows * c.hkv) return;
  const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
  const int e = (int)(w / c.hkv), h = (int)(w - (int64_t)e * c.hkv);
  const int r = request_of(cu, R, e);
  const int64_t t64 = (int64_t)(at ? at[r] : 0) + e - cu[r];
  const uint8_t* rec = t64 >= 0 && t64 < c.cap ? c.record(D, r, h, (int)(t64 / kKvGroup)) : nullptr;
  if (!rec) {
    if (lane == 0) set_status(status, SD_ERR_CAPACITY);
    return;
  }
  const int t = (int)t64;
  const uint8_t* codes = rec + half * kv4_half(D) + (t & 31) * (D / 2);
  const int b = half ? kv4_vbyte<D>(t, l * (kV / 2)) : l * (kV / 2);
  const uint32_t word = kV == 8 ? *reinterpret_cast<const uint32_t*>(codes + b)
                                : *reinterpret_cast<const uint16_t*>(codes + b);
  const uint32_t sm = *reinterpret_cast<const uint32_t*>(rec + half * kv4_half(D) + 16 * D + (t & 31) * 4);
  const float sc = bf2f((uint16_t)sm), md = bf2f((uint16_t)(sm >> 16));
  uint32_t o[kV / 2];
#pragma unroll
  for (int j = 0; j < kV / 2; j++) {
    const int c0 = (int)(word >> (8 * j) & 15) - 8, c1 = (int)(word >> (8 * j + 4) & 15) - 8;
    o[j] = pack_bf16x2(fmaf(sc, (float)c0, md), fmaf(sc, (float)c1, md));
  }
  uint16_t* dst = (half ? v_out : k_out) + w * D + l * kV;
  if constexpr (kV == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
  else *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
}

// ----------------------------------------------------------------- evict --
//
// Which slots stay: one CTA per (request, kv head).  The weight of the last
// slot that stays is found by radix selection (four passes of eight bits over
// order-preserving integer keys); a last pass in slot order lists the slots
// that stay and moves their positions and weights.

constexpr int kSelThreads = 1024;

// Integers ordered as the weights; NaN is the least.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);  // -0 counts as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) k_kv4_select(Kv4View s, Kv4View d, int budget, int recent, int sinks,
                                                            int32_t* __restrict__ list, int32_t* status) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t s_prefix, s_need;
  __shared__ uint32_t s_cnt[2][32];
  const int h = blockIdx.x, r = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int ctx = s.ctx_len[r];
  if (ctx < 0 || ctx > s.cap) {
    if (tid == 0) set_status(status, SD_ERR_CAPACITY);
    ctx = ctx < 0 ? 0 : (int)s.cap;
  }
  const int kept = min(ctx, budget);
  if (h == 0 && tid == 0) d.ctx_len[r] = kept;
  const float* w = s.weight + s.slot0(r, h);
  const int32_t* pos = s.pos + s.slot0(r, h);
  float* wd = d.weight + d.slot0(r, h);
  int32_t* pd = d.pos + d.slot0(r, h);
  int32_t* out = list + ((int64_t)r * s.hkv + h) * budget;
  if (ctx <= budget) {
    for (int t = tid; t < ctx; t += kSelThreads) {
      out[t] = t;
      wd[t] = w[t];
      pd[t] = pos[t];
    }
    return;
  }
  const int lo = sinks, hi = ctx - recent;  // ctx > budget >= sinks + recent
  uint32_t prefix = 0, need = (uint32_t)(budget - sinks - recent);
  for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int t = lo + tid; t < hi; t += kSelThreads) {
      const uint32_t key = weight_key(w[t]);
      if (shift == 24 || key >> (shift + 8) == prefix >> (shift + 8)) atomicAdd(&hist[key >> shift & 255], 1u);
    }
    __syncthreads();
    if (warp == 0) {
      // the bucket in which the need-th greatest key lies, counted from the top
      uint32_t c[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; j++) sum += c[j] = hist[255 - (lane * 8 + j)];
      uint32_t run = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += v;
      }
      uint32_t before = run - sum;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        if (before < need && before + c[j] >= need) {
          s_prefix = prefix | (uint32_t)(255 - (lane * 8 + j)) << shift;
          s_need = need - before;
        }
        before += c[j];
      }
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    __syncthreads();
  }
  // prefix: the least key that stays; need: how many of that key, the lowest slots first
  const bool any = budget > sinks + recent;
  uint32_t n_eq = 0, n_out = 0;
  for (int base = 0; base < ctx; base += kSelThreads) {
    const int t = base + tid;
    const bool in = t < ctx;
    const bool safe = in && (t < lo || t >= hi);
    const float wt = in ? w[t] : 0.f;
    const uint32_t key = weight_key(wt);
    const bool eq = any && in && !safe && key == prefix;
    const bool gt = any && in && !safe && key > prefix;
    const uint32_t be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) s_cnt[0][warp] = __popc(be);
    __syncthreads();
    uint32_t eq_before = n_eq, eq_all = 0;
    for (int i = 0; i < 32; i++) {
      if (i < warp) eq_before += s_cnt[0][i];
      eq_all += s_cnt[0][i];
    }
    const uint32_t rank = eq_before + __popc(be & ((1u << lane) - 1));
    const bool stay = safe || gt || (eq && rank < need);
    const uint32_t bs = __ballot_sync(0xffffffffu, stay);
    if (lane == 0) s_cnt[1][warp] = __popc(bs);
    __syncthreads();
    uint32_t before = n_out, all = 0;
    for (int i = 0; i < 32; i++) {
      if (i < warp) before += s_cnt[1][i];
      all += s_cnt[1][i];
    }
    if (stay) {
      const uint32_t o = before + __popc(bs & ((1u << lane) - 1));
      if (o < (uint32_t)budget) {
        out[o] = t;
        wd[o] = wt;
        pd[o] = pos[t];
      }
    }
    n_eq += eq_all;
    n_out += all;
  }
}

// Moves the rows that stay: one warp per group of 32 slots of dst.
template <int D>
__global__ void __launch_bounds__(256) k_kv4_move(Kv4View s, Kv4View d, int R, int budget, int groups,
                                                  const int32_t* __restrict__ list, int32_t* status) {
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= (int64_t)R * s.hkv * groups) return;
  const int lane = threadIdx.x & 31;
  const int g = (int)(w % groups);
  const int h = (int)(w / groups % s.hkv), r = (int)(w / groups / s.hkv);
  const int kept = min(d.ctx_len[r], budget);
  if (g * kKvGroup >= kept) return;
  uint8_t* dst = d.record(D, r, h, g);
  if (!dst) {
    if (lane == 0) set_status(status, SD_ERR_CAPACITY);
    return;
  }
  const int t = g * kKvGroup + lane;
  int from = -1;
  const uint8_t* src = nullptr;
  if (t < kept) {
    from = list[((int64_t)r * s.hkv + h) * budget + t];
    src = s.record(D, r, h, from / kKvGroup);
    if (!src) set_status(status, SD_ERR_CAPACITY);
  }
  if (src) {
#pragma unroll
    for (int half = 0; half < 2; half++)
      *reinterpret_cast<uint32_t*>(dst + half * kv4_half(D) + 16 * D + lane * 4) =
          *reinterpret_cast<const uint32_t*>(src + half * kv4_half(D) + 16 * D + (from & 31) * 4);
  }
  constexpr int kCh = D / 32;      // 16-byte pieces of a row of codes
  constexpr int kKeys = 32 / kCh;  // rows moved at once
#pragma unroll
  for (int half = 0; half < 2; half++)
#pragma unroll
    for (int j0 = 0; j0 < 32; j0 += kKeys) {
      const int j = j0 + lane / kCh, ch = lane % kCh;
      const uint8_t* sj = reinterpret_cast<const uint8_t*>(
          __shfl_sync(0xffffffffu, (unsigned long long)reinterpret_cast<uintptr_t>(src), j));
      const int fj = __shfl_sync(0xffffffffu, from, j);
      if (!sj) continue;
      const int bs = half ? kv4_vbyte<D>(fj, ch * 16) : ch * 16, bd = half ? kv4_vbyte<D>(j, ch * 16) : ch * 16;
      *reinterpret_cast<uint4*>(dst + half * kv4_half(D) + j * (D / 2) + bd) =
          *reinterpret_cast<const uint4*>(sj + half * kv4_half(D) + (fj & 31) * (D / 2) + bs);
    }
}

// ---------------------------------------------------------------- checks --

int kv4_bad(int code, const char* who, const char* what) {
  set_error(std::string(who) + ": " + what);
  return code;
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int kv4_check(const sd_kv4* c, int32_t R, const char* who, Kv4View* view) {
  if (!c || !c->blocks || !c->pos || !c->weight || !c->page_table || !c->ctx_len)
    return kv4_bad(SD_ERR_INVALID_ARG, who, "null cache or cache pointer");
  if (R < 1 || R > 65535) return kv4_bad(SD_ERR_INVALID_ARG, who, "1 <= R <= 65535 required");
  if (c->n_pages < 1 || c->max_pages < 1 || c->n_kv_heads < 1 || c->n_kv_heads > 1024)
    return kv4_bad(SD_ERR_INVALID_ARG, who, "n_pages, max_pages and n_kv_heads (at most 1024) must be positive");
  if (c->head_dim != 64 && c->head_dim != 128) return kv4_bad(SD_ERR_UNSUPPORTED, who, "head_dim must be 64 or 128");
  if (c->page_size < kKvGroup || c->page_size % kKvGroup)
    return kv4_bad(SD_ERR_UNSUPPORTED, who, "page_size must be a multiple of 32");
  if ((int64_t)c->max_pages * c->page_size > 0x7FFFFFFF - 65536)
    return kv4_bad(SD_ERR_UNSUPPORTED, who, "a request's capacity must stay below 2^31 - 2^16 slots");
  if (!aligned16(c->blocks) || !aligned16(c->pos) || !aligned16(c->weight))
    return kv4_bad(SD_ERR_INVALID_ARG, who, "blocks, pos and weight must be 16-byte aligned");
  view->blocks = c->blocks;
  view->pos = c->pos;
  view->weight = c->weight;
  view->page_table = c->page_table;
  view->ctx_len = c->ctx_len;
  view->n_pages = c->n_pages;
  view->gpp = c->page_size / kKvGroup;
  view->hkv = c->n_kv_heads;
  view->max_pages = c->max_pages;
  view->cap = (int64_t)c->max_pages * c->page_size;
  return SD_OK;
}

int kv4_check_rows(const int32_t* cu, const int32_t* cu_host, int32_t R, const char* who) {
  if (!cu || !cu_host) return kv4_bad(SD_ERR_INVALID_ARG, who, "null cu or cu_host");
  if (cu_host[0] != 0) return kv4_bad(SD_ERR_INVALID_ARG, who, "cu[0] must be 0");
  for (int r = 0; r < R; r++)
    if (cu_host[r + 1] < cu_host[r]) return kv4_bad(SD_ERR_INVALID_ARG, who, "cu must not decrease");
  return SD_OK;
}

int kv4_check_score(const sd_kv4_score* sc, const char* who, Kv4Score* out, int head_dim) {
  *out = Kv4Score{};
  if (sc) {
    if (!(sc->softcap >= 0.f) || !(sc->softcap <= 1e30f) || !(sc->scale >= 0.f) || !(sc->scale <= 1e30f) || sc->window < 0)
      return kv4_bad(SD_ERR_INVALID_ARG, who, "scale, softcap and window must be finite and not negative");
    out->scale = sc->scale;
    out->cap = sc->softcap;
    out->slopes = sc->slopes;
    out->window = sc->window;
    out->start = sc->start;
  }
  if (out->scale == 0.f) out->scale = head_dim == 128 ? 0.08838834764831845f : 0.125f;
  return SD_OK;
}

}  // namespace sdv

using namespace sdv;

extern "C" int64_t sd_kv4_group_bytes(int32_t head_dim) {
  return head_dim == 64 || head_dim == 128 ? kv4_rec(head_dim) : 0;
}

extern "C" int sd_kv4_append(const sd_kv4* c, const uint16_t* k, const uint16_t* v, int64_t row_stride, int32_t n_src,
                             const int32_t* cu, const int32_t* cu_host, int32_t R, const int32_t* src,
                             const int32_t* count, const int32_t* pos, const int32_t* at, int32_t* status,
                             void* stream) {
  const char* who = "sd_kv4_append";
  Kv4View view;
  if (int rc = kv4_check(c, R, who, &view)) return rc;
  if (int rc = kv4_check_rows(cu, cu_host, R, who)) return rc;
  const int rows = cu_host[R];
  if (!k || !v || !aligned16(k) || !aligned16(v)) return kv4_bad(SD_ERR_INVALID_ARG, who, "k and v must be set and 16-byte aligned");
  if (row_stride < (int64_t)c->n_kv_heads * c->head_dim || row_stride % 8)
    return kv4_bad(SD_ERR_INVALID_ARG, who, "row_stride must cover a row and be a multiple of 8");
  if (n_src < 0 || (!src && n_src < rows)) return kv4_bad(SD_ERR_INVALID_ARG, who, "fewer rows in k and v than in cu");
  if (rows == 0) return SD_OK;
  const bool in_place = !at || at == c->ctx_len;
  const int64_t blocks = ((int64_t)rows * c->n_kv_heads + 7) / 8;
  if (blocks > 0x7FFFFFFF) return kv4_bad(SD_ERR_UNSUPPORTED, who, "too many rows");
  cudaStream_t st = (cudaStream_t)stream;
  auto kern = c->head_dim == 128 ? k_kv4_append<128> : k_kv4_append<64>;
  kern<<<(unsigned)blocks, 256, 0, st>>>(view, k, v, row_stride, n_src, cu, R, rows, src, count, pos,
                                         in_place ? c->ctx_len : at, !in_place, status);
  SD_CK(cudaGetLastError());
  if (in_place) {
    k_kv4_advance<<<(R + 127) / 128, 128, 0, st>>>(c->ctx_len, cu, count, R, view.cap);
    SD_CK(cudaGetLastError());
  }
  return SD_OK;
}

extern "C" int sd_kv4_read(const sd_kv4* c, const int32_t* cu, const int32_t* cu_host, int32_t R, const int32_t* at,
                           uint16_t* k_out, uint16_t* v_out, int32_t* status, void* stream) {
  const char* who = "sd_kv4_read";
  Kv4View view;
  if (int rc = kv4_check(c, R, who, &view)) return rc;
  if (int rc = kv4_check_rows(cu, cu_host, R, who)) return rc;
  if (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out))
    return kv4_bad(SD_ERR_INVALID_ARG, who, "k_out and v_out must be set and 16-byte aligned");
  const int rows = cu_host[R];
  if (rows == 0) return SD_OK;
  const int64_t blocks = ((int64_t)rows * c->n_kv_heads + 7) / 8;
  if (blocks > 0x7FFFFFFF) return kv4_bad(SD_ERR_UNSUPPORTED, who, "too many rows");
  auto kern = c->head_dim == 128 ? k_kv4_read<128> : k_kv4_read<64>;
  kern<<<(unsigned)blocks, 256, 0, (cudaStream_t)stream>>>(view, cu, R, rows, at, k_out, v_out, status);
  SD_CK(cudaGetLastError());
  return SD_OK;
}

extern "C" size_t sd_kv4_evict_workspace(int32_t R, int32_t n_kv_heads, int32_t budget) {
  if (R < 1 || n_kv_heads < 1 || budget < 1) return 0;
  return (size_t)R * n_kv_heads * budget * 4;
}

extern "C" int sd_kv4_evict(const sd_kv4* src, const sd_kv4* dst, int32_t R, int32_t budget, int32_t recent,
                            int32_t sinks, void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
  const char* who = "sd_kv4_evict";
  Kv4View s, d;
  if (int rc = kv4_check(src, R, who, &s)) return rc;
  if (int rc = kv4_check(dst, R, who, &d)) return rc;
  if (src->n_kv_heads != dst->n_kv_heads || src->head_dim != dst->head_dim)
    return kv4_bad(SD_ERR_INVALID_ARG, who, "src and dst differ in heads");
  if (src->pos == dst->pos || src->weight == dst->weight || src->ctx_len == dst->ctx_len)
    return kv4_bad(SD_ERR_INVALID_ARG, who, "dst needs pos, weight and ctx_len of its own");
  if (budget < 1 || recent < 0 || sinks < 0 || (int64_t)recent + sinks > budget)
    return kv4_bad(SD_ERR_INVALID_ARG, who, "budget must be positive and hold sinks + recent");
  if (d.cap < budget) return kv4_bad(SD_ERR_INVALID_ARG, who, "dst cannot hold the budget");
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return kv4_bad(SD_ERR_INVALID_ARG, who, "workspace must be set and 256-byte aligned");
  if (workspace_bytes < sd_kv4_evict_workspace(R, src->n_kv_heads, budget))
    return kv4_bad(SD_ERR_WORKSPACE, who, "workspace too small");
  cudaStream_t st = (cudaStream_t)stream;
  int32_t* list = (int32_t*)workspace;
  k_kv4_select<<<dim3(src->n_kv_heads, R), kSelThreads, 0, st>>>(s, d, budget, recent, sinks, list, status);
  SD_CK(cudaGetLastError());
  const int groups = (int)(((int64_t)budget + kKvGroup - 1) / kKvGroup);
  const int64_t blocks = ((int64_t)R * src->n_kv_heads * groups + 7) / 8;
  if (blocks > 0x7FFFFFFF) return kv4_bad(SD_ERR_UNSUPPORTED, who, "too many slots");
  auto kern = src->head_dim == 128 ? k_kv4_move<128> : k_kv4_move<64>;
  kern<<<(unsigned)blocks, 256, 0, st>>>(s, d, R, budget, groups, list, status);
  SD_CK(cudaGetLastError());
  return SD_OK;
}
