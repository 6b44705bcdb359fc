// The 4-bit key/value cache: storing rows, reading them back, eviction.
#include "kv4.cuh"

namespace sdv {

// ---------------------------------------------------------------- append --
//
// One warp stores a row's keys and values of kHeads kv heads: a half warp the
// key, the other the value, D / 16 values a lane (one or half a 32-bit word of
// codes); the next head's row is on its way while one is worked on.  A row's
// least and greatest value come from four shuffles.  The bytes are few (4 D in,
// D + 12 out per row and head); what bounds it is issue, 82% active: about 250
// instructions a warp per row and head.  Four heads a warp share the row's
// addresses and request (with one, storing and reading back 16384 rows took 92 us
// where four took 63; both take 52 now).  Measured: 16384 rows of 8 heads, D = 128,
// stored: 37 us, 2.3 TB/s of the 85 MB read and written.

constexpr int kHeads = 4;

__device__ __forceinline__ uint32_t bf2_min(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf2_max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t bf2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// N consecutive 16-bit values of a row as 32-bit words.
template <int N>
__device__ __forceinline__ void load_row(const uint16_t* p, uint32_t (&w)[N / 2]) {
  if constexpr (N == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x, w[1] = u.y;
  }
}

template <int D>
__global__ void __launch_bounds__(256) k_kv4_append(Kv4View c, const uint16_t* __restrict__ k,
                                                    const uint16_t* __restrict__ v, int64_t row_stride, int n_src,
                                                    const int32_t* __restrict__ cu, int R, int rows,
                                                    const int32_t* __restrict__ src, const int32_t* __restrict__ count,
                                                    const int32_t* __restrict__ pos, const int32_t* at, bool advance,
                                                    int32_t* status) {
  constexpr int kV = D / 16;  // values of a lane
  pdl_launch();
  const int e = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (e >= rows) return;
  const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
  const int h0 = blockIdx.y * kHeads, nh = min(kHeads, c.hkv - h0);
  const int s = src ? src[e] : e;
  const bool s_ok = s >= 0 && s < n_src;
  const uint16_t* x = (half ? v : k) + (s_ok ? (int64_t)s * row_stride : 0) + h0 * D + l * kV;
  uint32_t next[kV / 2] = {};
  if (s_ok) load_row<kV>(x, next);  // k and v may have no rows at all
  const int p = pos ? pos[e] : 0;
  const int r = request_of(cu, R, e);
  const int i0 = e - cu[r];
  const int n = count ? min(max(count[r], 0), cu[r + 1] - cu[r]) : cu[r + 1] - cu[r];
  const int a = at[r];
  if (a < 0 || (int64_t)a + n > c.cap) {
    if (lane == 0) set_status(status, SD_ERR_CAPACITY);
    return;
  }
  if (i0 == 0 && h0 == 0 && lane == 0 && advance) c.ctx_len[r] = a + n;
  if (i0 >= n) return;
  const int t = a + i0;
  uint8_t* rec = s_ok ? c.record(D, r, h0, t / kKvGroup) : nullptr;
  if (!rec) {
    if (lane == 0) set_status(status, SD_ERR_CAPACITY);
    return;
  }
#pragma unroll 1
  for (int i = 0; i < nh; i++) {
    uint32_t raw[kV / 2];
#pragma unroll
    for (int j = 0; j < kV / 2; j++) raw[j] = next[j];
    if (i + 1 < nh) load_row<kV>(x + (i + 1) * D, next);
    // least and greatest, bf16 pairs at a time; a NaN stays one
    uint32_t lo2 = raw[0], hi2 = raw[0];
#pragma unroll
    for (int j = 1; j < kV / 2; j++) lo2 = bf2_min(lo2, raw[j]), hi2 = bf2_max(hi2, raw[j]);
    // (greatest, minus the least) as one pair across the lanes
    uint32_t ext = bf2_max(prmt(hi2, lo2, 0x5410) ^ 0x80000000u, prmt(hi2, lo2, 0x7632) ^ 0x80000000u);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) ext = bf2_max(ext, __shfl_xor_sync(0xffffffffu, ext, o));
    const float lo = -__uint_as_float(ext & 0xFFFF0000u), range = __uint_as_float(ext << 16) - lo;
    // s: the product with 1 / 15 is within two units of the quotient; the
    // division decides where that could turn the rounding to bf16
    float sq = range * (1.f / 15.f);
    const uint32_t tail = (__float_as_uint(sq) & 0xFFFFu) - 0x7FFCu;
    if (__any_sync(0xffffffffu, tail <= 8u || !(sq > 1e-30f))) sq = __fdiv_rn(range, 15.f);
    float sc = rbf(sq), md = rbf(fmaf(8.f, sc, lo));
    if (!(range <= 3.4028234e38f)) sc = md = __int_as_float(0x7FC00000);  // not finite: the row is held as NaN
    // A code is the nearest step, halves to even: the low bits of (x - m) / s +
    // 8 + 1.5 2^23, clamped.  The product with the approximate 1 / s is within 2^-19
    // of the quotient (at most 8 or so); where that leaves a half in doubt
    // anywhere in the warp, the remainder x - m - n s, which is exact, decides.
    constexpr float kBase = 12582912.f;  // 1.5 2^23: integers to a unit
    const bool fine = sc > 1e-30f && sc < 1e30f;
    const float inv = fine ? __fdividef(1.f, sc) : 0.f;
    float far = 0.f, st[kV];
#pragma unroll
    for (int j = 0; j < kV; j += 2) {
      const uint64_t d = f2add(f2pack(__uint_as_float(raw[j >> 1] << 16), __uint_as_float(raw[j >> 1] & 0xFFFF0000u)),
                               f2pack(-md, -md));
      const uint64_t n = f2fma(d, f2pack(inv, inv), f2pack(kBase + 8.f, kBase + 8.f));
      // the distance to the step taken: (n - base) - d inv, its size alone counts
      const uint64_t off = f2fma(d, f2pack(-inv, -inv), f2add(n, f2pack(-kBase - 8.f, -kBase - 8.f)));
      float o0, o1;
      f2unpack(n, st[j], st[j + 1]);
      f2unpack(off, o0, o1);
      far = fmaxf(far, fmaxf(fabsf(o0), fabsf(o1)));
    }
    if (__any_sync(0xffffffffu, far > 0.5f - 4e-6f || !fine)) {
      const float h = 0.5f * sc;
#pragma unroll
      for (int j = 0; j < kV; j++) {
        const float d = __uint_as_float(j & 1 ? raw[j >> 1] & 0xFFFF0000u : raw[j >> 1] << 16) - md;
        if (fine) {
          const float r = fmaf(-(st[j] - (kBase + 8.f)), sc, d);
          const bool odd = __float_as_uint(st[j]) & 1u;
          if (r > h || (r == h && odd)) st[j] += 1.f;
          else if (r < -h || (r == -h && odd)) st[j] -= 1.f;
        } else {  // NaN and s = 0 give code 8
          st[j] = kBase + 8.f + (sc > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(d, sc)), -8.f), 7.f) : 0.f);
        }
      }
    }
    // (the constant bits 0x4B400000 of each, shifted like its code, add up to kOnes)
    constexpr uint32_t kOnes = kV == 8 ? 0x4B400000u * 0x11111111u : 0x4B400000u * 0x1111u;
    uint32_t word = 0u - kOnes;
#pragma unroll
    for (int j = 0; j < kV; j++) word += __float_as_uint(fminf(fmaxf(st[j], kBase), kBase + 15.f)) << (4 * j);
    uint8_t* const rh = rec + (int64_t)i * c.gpp * kv4_rec(D);
    uint8_t* codes = rh + half * kv4_half(D) + (t & 31) * (D / 2);
    const int b = half ? kv4_vbyte<D>(t, l * (kV / 2)) : l * (kV / 2);
    if constexpr (kV == 8) *reinterpret_cast<uint32_t*>(codes + b) = word;
    else *reinterpret_cast<uint16_t*>(codes + b) = (uint16_t)word;
    if (l == 0) {
      *reinterpret_cast<uint32_t*>(rh + half * kv4_half(D) + 16 * D + (t & 31) * 4) =
          (uint32_t)f2bf(sc) | (uint32_t)f2bf(md) << 16;
      const int64_t o = c.slot0(r, h0 + i) + t;
      if (half) c.weight[o] = 0.f;
      else c.pos[o] = pos ? p : t;
    }
  }
}

// ctx_len[r] += the rows stored, once they are (append in place).
__global__ void k_kv4_advance(int32_t* ctx_len, const int32_t* __restrict__ cu, const int32_t* __restrict__ count,
                              int R, int64_t cap) {
  pdl_wait();
  const int r = blockIdx.x * blockDim.x + threadIdx.x;
  if (r >= R) return;
  const int n = count ? min(max(count[r], 0), cu[r + 1] - cu[r]) : cu[r + 1] - cu[r];
  const int a = ctx_len[r];
  if (a >= 0 && (int64_t)a + n <= cap) ctx_len[r] = a + n;
}

// ------------------------------------------------------------------ read --
//
// The append's warp and lanes, the other way.  16384 rows of 8 heads, D = 128: 14
// us, 6.1 TB/s.
template <int D>
__global__ void __launch_bounds__(256) k_kv4_read(Kv4View c, const int32_t* __restrict__ cu, int R, int rows,
                                                  const int32_t* __restrict__ at, uint16_t* __restrict__ k_out,
                                                  uint16_t* __restrict__ v_out, int32_t* status) {
  constexpr int kV = D / 16;
  const int e = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (e >= rows) return;
  const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
  const int h0 = blockIdx.y * kHeads, nh = min(kHeads, c.hkv - h0);
  const int r = request_of(cu, R, e);
  const int64_t t64 = (int64_t)(at ? at[r] : 0) + e - cu[r];
  const uint8_t* rec = t64 >= 0 && t64 < c.cap ? c.record(D, r, h0, (int)(t64 / kKvGroup)) : nullptr;
  if (!rec && lane == 0) set_status(status, SD_ERR_CAPACITY);
  const int t = (int)t64;
  const int b = half ? kv4_vbyte<D>(t, l * (kV / 2)) : l * (kV / 2);
  uint32_t word[kHeads], sm[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; i++)
    if (!rec) {
      word[i] = 0, sm[i] = 0x7FC07FC0u;  // no such slot: NaN
    } else if (i < nh) {
      const uint8_t* part = rec + (int64_t)i * c.gpp * kv4_rec(D) + half * kv4_half(D);
      const uint8_t* codes = part + (t & 31) * (D / 2) + b;
      word[i] = kV == 8 ? *reinterpret_cast<const uint32_t*>(codes) : *reinterpret_cast<const uint16_t*>(codes);
      sm[i] = *reinterpret_cast<const uint32_t*>(part + 16 * D + (t & 31) * 4);
    }
#pragma unroll
  for (int i = 0; i < kHeads; i++) {
    if (i >= nh) break;
    // (code - 8) s + m in bf16 pairs, rounded once: 0x4300 | code is 128 + code,
    // and code - 8 is exact.  Pair n of a word: nibbles n and n + 4
    const uint32_t s2 = prmt(sm[i], 0, 0x1010), m2 = prmt(sm[i], 0, 0x3232);
    uint32_t o[kV / 2], p[4];
    const uint32_t wd = kV == 8 ? word[i] : (word[i] & 0xFFu) | (word[i] & 0xFF00u) << 8;
#pragma unroll
    for (int j = 0; j < kV / 2; j++) p[j] = bf2_fma(s2, bf2_sub((wd >> (4 * j) & 0x000F000Fu) | 0x43004300u, 0x43084308u), m2);
    if constexpr (kV == 8) {
      o[0] = prmt(p[0], p[1], 0x5410), o[1] = prmt(p[2], p[3], 0x5410);
      o[2] = prmt(p[0], p[1], 0x7632), o[3] = prmt(p[2], p[3], 0x7632);
    } else {
      o[0] = prmt(p[0], p[1], 0x5410), o[1] = prmt(p[0], p[1], 0x7632);
    }
    uint16_t* dst = (half ? v_out : k_out) + ((int64_t)e * c.hkv + h0 + i) * D + l * kV;
    if constexpr (kV == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
    else *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
  }
}

// ----------------------------------------------------------------- evict --
//
// Which slots stay: one CTA per (request, kv head).  The weight of the last
// slot that stays is found by radix selection (11, 11 and 10 bits of
// order-preserving integer keys); then each warp counts what stays of its run
// of slots, and lists them in slot order with their positions and weights.
// Bound: latency (the weights are read from the caches five times); the bytes
// are few.  16 requests of 5000 to 16384 slots, 8 heads: 21 us.

constexpr int kSelThreads = 1024;

// Integers ordered as the weights; NaN is the least.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);  // -0 counts as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) k_kv4_select(Kv4View s, Kv4View d, int budget, int recent, int sinks,
                                                            int32_t* __restrict__ list, int32_t* status) {
  __shared__ uint32_t hist[2048];
  __shared__ uint32_t s_prefix, s_need, s_sum[2][32];
  const int h = blockIdx.x, r = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch();
  int ctx = s.ctx_len[r];
  if (ctx < 0 || ctx > s.cap) {
    if (tid == 0) set_status(status, SD_ERR_CAPACITY);
    ctx = ctx < 0 ? 0 : (int)s.cap;
  }
  const int kept = min(ctx, budget);
  if (h == 0 && tid == 0) d.ctx_len[r] = kept;
  const float* __restrict__ w = s.weight + s.slot0(r, h);
  const int32_t* __restrict__ pos = s.pos + s.slot0(r, h);
  float* __restrict__ wd = d.weight + d.slot0(r, h);
  int32_t* __restrict__ pd = d.pos + d.slot0(r, h);
  int32_t* __restrict__ out = list + ((int64_t)r * s.hkv + h) * budget;
  if (ctx <= budget) {
    for (int t = tid; t < ctx; t += kSelThreads) {
      out[t] = t;
      wd[t] = w[t];
      pd[t] = pos[t];
    }
    return;
  }
  const int lo = sinks, hi = ctx - recent;  // ctx > budget >= sinks + recent
  const bool any = budget > sinks + recent;
  uint32_t prefix = 0, need = (uint32_t)(budget - sinks - recent);
  for (int pass = 0; pass < 3 && any; pass++) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    hist[tid] = hist[tid + 1024] = 0;
    __syncthreads();
#pragma unroll 4
    for (int t = lo + tid; t < hi; t += kSelThreads) {
      const uint32_t key = weight_key(w[t]);
      if (pass == 0 || (key ^ prefix) >> (shift + bits) == 0) atomicAdd(&hist[key >> shift & ((1u << bits) - 1)], 1u);
    }
    __syncthreads();
    // the bin in which the need-th greatest key lies, counted from the top: two
    // bins a thread
    const int b1 = 2047 - 2 * tid, b0 = b1 - 1;
    const uint32_t c1 = hist[b1], c0 = hist[b0];
    uint32_t run = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += v;
    }
    if (lane == 31) s_sum[0][warp] = run;
    __syncthreads();
    uint32_t warps = s_sum[0][lane];  // sums of the warps before this one
    warps = __reduce_add_sync(0xffffffffu, lane < warp ? warps : 0u);
    const uint32_t before = warps + run - c0 - c1;
    if (before < need && before + c1 >= need) {
      s_prefix = prefix | (uint32_t)b1 << shift;
      s_need = need - before;
    } else if (before + c1 < need && before + c1 + c0 >= need) {
      s_prefix = prefix | (uint32_t)b0 << shift;
      s_need = need - before - c1;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  // prefix: the least key that stays; need: how many of that key, the lowest slots first
  auto kind = [&](int t, float wt) {  // 0 goes, 1 stays, 2 has the least key
    if (t < lo || t >= hi) return 1;
    const uint32_t key = weight_key(wt);
    return !any ? 0 : key > prefix ? 1 : key == prefix ? 2 : 0;
  };
  const int per = (ctx + kSelThreads - 1) / kSelThreads * 32, t0 = warp * per, t1 = min(ctx, t0 + per);
  uint32_t n1 = 0, n2 = 0;
#pragma unroll 4
  for (int t = t0 + lane; t < t1; t += 32) {
    const int x = kind(t, w[t]);
    n1 += x == 1;
    n2 += x == 2;
  }
  n1 = __reduce_add_sync(0xffffffffu, n1);
  n2 = __reduce_add_sync(0xffffffffu, n2);
  __syncthreads();
  if (lane == 0) s_sum[0][warp] = n1, s_sum[1][warp] = n2;
  __syncthreads();
  n1 = lane < warp ? s_sum[0][lane] : 0;
  n2 = lane < warp ? s_sum[1][lane] : 0;
  uint32_t eq = __reduce_add_sync(0xffffffffu, n2);                         // of the least key, before this warp
  uint32_t o = __reduce_add_sync(0xffffffffu, n1) + min(eq, need);          // staying before this warp
  const uint32_t below = (1u << lane) - 1;
  for (int t4 = t0 + lane; t4 - lane < t1; t4 += 128) {
    float wt[4];
    int ps[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const int t = min(t4 + 32 * k, ctx - 1);
      wt[k] = w[t];
      ps[k] = pos[t];
    }
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const int t = t4 + 32 * k;
      const int x = t < t1 ? kind(t, wt[k]) : 0;
      const uint32_t be = __ballot_sync(0xffffffffu, x == 2);
      const bool stay = x == 1 || (x == 2 && eq + __popc(be & below) < need);
      const uint32_t bs = __ballot_sync(0xffffffffu, stay);
      const uint32_t at = o + __popc(bs & below);
      if (stay && at < (uint32_t)budget) {
        out[at] = t;
        wd[at] = wt[k];
        pd[at] = ps[k];
      }
      eq += __popc(be);
      o += __popc(bs);
    }
  }
}

// Moves the rows that stay: one warp per group of 32 slots of dst, all of its
// reads in flight before the first write.  Bound: bytes (2048 rows of 16 requests
// and 8 heads, D = 128, 143 MB in and out: 17 us, the writes still in the L2).
template <int D>
__global__ void __launch_bounds__(256) k_kv4_move(Kv4View s, Kv4View d, int budget, const int32_t* __restrict__ list,
                                                  int32_t* status) {
  pdl_wait();
  const int h = blockIdx.y, r = blockIdx.z, lane = threadIdx.x & 31;
  const int g = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int kept = min(d.ctx_len[r], budget);
  if (g * kKvGroup >= kept) return;
  uint8_t* dst = d.record(D, r, h, g);
  const int t = g * kKvGroup + lane;
  int from = 0;
  const uint8_t* src = nullptr;
  if (t < kept) {
    from = list[((int64_t)r * s.hkv + h) * budget + t];
    src = s.record(D, r, h, from / kKvGroup);
  }
  if (!dst || (t < kept && !src)) set_status(status, SD_ERR_CAPACITY);
  if (!dst) return;
  constexpr int kCh = D / 32;      // 16-byte pieces of a row of codes
  constexpr int kKeys = 32 / kCh;  // rows moved at once
  uint32_t sm[2];
  uint4 x[2][32 / kKeys];
  bool ok[32 / kKeys];
#pragma unroll
  for (int half = 0; half < 2; half++) {
    sm[half] = 0x7FC07FC0u;  // a kept row whose page is not there is held as NaN, whatever dst's record held
    if (src) sm[half] = *reinterpret_cast<const uint32_t*>(src + half * kv4_half(D) + 16 * D + (from & 31) * 4);
#pragma unroll
    for (int i = 0; i < 32 / kKeys; i++) {
      const int j = i * kKeys + lane / kCh, ch = lane % kCh;
      const uint8_t* sj = reinterpret_cast<const uint8_t*>(
          __shfl_sync(0xffffffffu, (unsigned long long)reinterpret_cast<uintptr_t>(src), j));
      const int fj = __shfl_sync(0xffffffffu, from, j);
      ok[i] = sj != nullptr;
      if (ok[i])
        x[half][i] = *reinterpret_cast<const uint4*>(sj + half * kv4_half(D) + (fj & 31) * (D / 2) +
                                                     (half ? kv4_vbyte<D>(fj, ch * 16) : ch * 16));
    }
  }
#pragma unroll
  for (int half = 0; half < 2; half++) {
    if (t < kept) *reinterpret_cast<uint32_t*>(dst + half * kv4_half(D) + 16 * D + lane * 4) = sm[half];
#pragma unroll
    for (int i = 0; i < 32 / kKeys; i++) {
      const int j = i * kKeys + lane / kCh, ch = lane % kCh;
      if (ok[i])
        *reinterpret_cast<uint4*>(dst + half * kv4_half(D) + j * (D / 2) + (half ? kv4_vbyte<D>(j, ch * 16) : ch * 16)) =
            x[half][i];
    }
  }
}

// ---------------------------------------------------------------- checks --

int kv4_bad(int code, const char* who, const char* what) {
  set_error(std::string(who) + ": " + what);
  return code;
}

// A kernel that may begin while the one before it ends (it calls pdl_wait()).
// Unlike launch() it leaves the L1 as it is: asking for the shared memory of
// the verify step's kernels costs an eviction of 16 x 16k keys 8 us.
template <typename... KArgs, typename... Args>
static cudaError_t launch_after(void (*kern)(KArgs...), dim3 grid, int block, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
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
  if (rows && (!k || !v || !aligned16(k) || !aligned16(v))) return kv4_bad(SD_ERR_INVALID_ARG, who, "k and v must be set and 16-byte aligned");
  if (row_stride < (int64_t)c->n_kv_heads * c->head_dim || row_stride % 8)
    return kv4_bad(SD_ERR_INVALID_ARG, who, "row_stride must cover a row and be a multiple of 8");
  if (n_src < 0 || (!src && n_src < rows)) return kv4_bad(SD_ERR_INVALID_ARG, who, "fewer rows in k and v than in cu");
  if (rows == 0) return SD_OK;
  const bool in_place = !at || at == c->ctx_len;
  const dim3 grid((rows + 7) / 8, (c->n_kv_heads + kHeads - 1) / kHeads);
  cudaStream_t st = (cudaStream_t)stream;
  auto kern = c->head_dim == 128 ? k_kv4_append<128> : k_kv4_append<64>;
  kern<<<grid, 256, 0, st>>>(view, k, v, row_stride, n_src, cu, R, rows, src, count, pos,
                                         in_place ? c->ctx_len : at, !in_place, status);
  SD_CK(cudaGetLastError());
  if (in_place) {
    SD_CK(launch_after(k_kv4_advance, dim3((R + 127) / 128), 128, st, c->ctx_len, cu, count, R, view.cap));
  }
  return SD_OK;
}

extern "C" int sd_kv4_read(const sd_kv4* c, const int32_t* cu, const int32_t* cu_host, int32_t R, const int32_t* at,
                           uint16_t* k_out, uint16_t* v_out, int32_t* status, void* stream) {
  const char* who = "sd_kv4_read";
  Kv4View view;
  if (int rc = kv4_check(c, R, who, &view)) return rc;
  if (int rc = kv4_check_rows(cu, cu_host, R, who)) return rc;
  const int rows = cu_host[R];
  if (rows == 0) return SD_OK;
  if (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out))
    return kv4_bad(SD_ERR_INVALID_ARG, who, "k_out and v_out must be set and 16-byte aligned");
  const dim3 grid((rows + 7) / 8, (c->n_kv_heads + kHeads - 1) / kHeads);
  auto kern = c->head_dim == 128 ? k_kv4_read<128> : k_kv4_read<64>;
  kern<<<grid, 256, 0, (cudaStream_t)stream>>>(view, cu, R, rows, at, k_out, v_out, status);
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
  auto kern = src->head_dim == 128 ? k_kv4_move<128> : k_kv4_move<64>;
  SD_CK(launch_after(kern, dim3((groups + 7) / 8, src->n_kv_heads, R), 256, st, s, d, budget, list, status));
  return SD_OK;
}
