// Tokens sampled from logits: temperature, top-k, min-p, top-p.
//
// A bf16 logit is one of 65536 keys, so a row is a histogram: everything a
// sampled token depends on follows from how often each key occurs, and its weight
// is computed once a key.  A row's keys are counted in shared memory; of each binade
// (128 keys) that occurs the count and the sum of weights are taken; one warp walks
// their running sums down to the cuts and the token's key, and the key's occurrence is
// looked up in the row.  Two kernels:
//  * many rows: a CTA a row, counters of the magnitudes 2^-24 .. 2^15 and of zero
//    (40 KB, two CTAs an SM); a row with others is left to the next kernel, which has 32
//    clusters for such rows, one after the other: one of 256 adds 19 us, and where all
//    have one (a mask of the type's lowest value; -inf is none) 256 rows of 151936 take
//    322 us for 57, of 32000 331 for 26;
//  * few rows: a cluster of up to 8 CTAs a row, 16-bit counters of all 65536 keys (so at
//    most 65528 tokens a CTA), summed through distributed shared memory.
//
// What bounds them: of 256 rows of 151936 (78 MB; 57 us, 1.4 TB/s) the counting takes half,
// 5.5 cycles a warp's atomic in shared memory with two CTAs an SM (bank conflicts of 32
// random keys), the walk of one warp 15% by its latency, the look-up 10%.  With counters of
// 16 bits and a cluster a row the same took 130 us.  One row (22 us, a cluster of 8): the
// latency of its phases (loads and clearing 5, counting 7, sums 6, the walk 8 and the
// look-up 4 thousand cycles) and of three cluster barriers (2 each); the five vectors that
// a thread keeps cost it about 200 bytes of spills.
//
// Weights are whole numbers, 2^44 exp((logit - most) / temperature), from pairs
// of fp32 values good to about 2^-46, and their sums are 64-bit whole numbers (2^44
// times 2^19 tokens): results do not depend on the order of a sum, and a u next
// to a border of 2^-17 (1 / vocab) falls on the right side.
#include <algorithm>

#include "common.cuh"

namespace sdv {

namespace sp {
constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kSlice = 65528;          // tokens of a CTA, at most: whole vectors, 16-bit counters
constexpr int kMaxCluster = 8;
constexpr int kMaxVocab = (1 << 19) - 128;
constexpr int kBlocks = 513;           // binades of either sign, and zero's once more
constexpr int kTable = 48;             // binades whose keys' counts and weights are kept
constexpr int kHeld = 5;               // vectors of 8 tokens that a thread keeps
constexpr int kOne = 44;               // weights are multiples of 2^-kOne
constexpr int kRowThreads = 512, kRowWarps = kRowThreads / 32;
constexpr int kLeast = 127 - 24, kSpan = 39;     // exponents of the row kernel's binades
constexpr int kRowKeys = kSpan * 128;            // of either sign
constexpr int kRowBlocks = 2 * kSpan + 1;        // positive ones falling, zero, negative ones
constexpr int kLater = INT32_MIN;                // token of a row that is left to the next kernel
constexpr float kLog2e = 1.4426950408889634f;
}  // namespace sp

// exp of a double by its series, at compile time (|x| < 1).
constexpr double cexp(double x) {
  double t = 1, s = 1;
  for (int i = 1; i < 30; i++) t *= x / i, s += t;
  return s;
}
struct Exp2Table {
  float hi[32], lo[32];
  constexpr Exp2Table() : hi(), lo() {
    for (int j = 0; j < 32; j++) {
      const double v = cexp(0.693147180559945309417 * j / 32);
      hi[j] = (float)v;
      lo[j] = (float)(v - (double)hi[j]);
    }
  }
};
__device__ const Exp2Table kExp2 = Exp2Table();

// What a row's weights go by.
struct RowScale {
  float most;    // greatest logit
  float ch, cl;  // 2 log2(e) / temperature as a pair; 0 where greedy
};

// A weight 2^n (h + l), h + l in [1, 2].
struct Weight {
  float h, l;
  int n;
  // in multiples of 2^-44: h has 24 bits, a whole number times 2^-24 at least
  __device__ __forceinline__ uint64_t whole() const {
    const uint64_t v = ((uint64_t)(uint32_t)(h * 16777216.f) << (sp::kOne - 24)) + (int64_t)(int)rintf(l * 0x1p44f);
    return n == 0 ? v : n < -sp::kOne - 2 ? 0 : (v + (1ull << (-n - 1))) >> -n;
  }
  __device__ __forceinline__ float value() const { return h * __int_as_float((127 + max(n, -126)) << 23); }
  __device__ __forceinline__ bool at_least(float p) const {
    const float q = p * __int_as_float((127 + min(-n, 126)) << 23) * __int_as_float((127 + max(-n - 126, 0)) << 23);
    return __fadd_rn(__fadd_rn(h, -q), l) >= 0.f;
  }
};

// The weight of logit l <= most; n = -200 where it is below 2^-151, less than any min_p.
__device__ __forceinline__ Weight weight_here(float l, const RowScale& r, const float2* s_exp2) {
  // (l - most) / 2 = s + d (l - most may pass fp32), log2 of the weight p + e
  const float half = 0.5f * r.most;
  const float s = __fmaf_rn(l, 0.5f, -half), b = __fmaf_rn(l, -0.5f, s);
  const float d = __fadd_rn(__fmaf_rn(l, 0.5f, -__fadd_rn(s, -b)), __fadd_rn(-half, -b));
  float p = __fmul_rn(s, r.ch);
  float e = __fmaf_rn(s, r.ch, -p);
  e = __fmaf_rn(s, r.cl, e);
  e = __fmaf_rn(d, r.ch, e);
  const bool one = l >= r.most, none = !one && !(p > -151.f);  // beside +inf too
  if (one || none) p = e = 0.f;
  // p + e = m / 32 + f + e, |f| <= 1 / 64
  const float mf = rintf(p * 32.f);
  const int m = (int)mf;
  const float f = __fmaf_rn(mf, -1.f / 32.f, p);
  constexpr double kLn2 = 0.693147180559945309417;
  constexpr float ln2h = (float)kLn2, ln2l = (float)(kLn2 - (double)ln2h);
  const float th = __fmul_rn(f, ln2h);
  float tl = __fmaf_rn(f, ln2h, -th);
  tl = __fmaf_rn(f, ln2l, tl);
  tl = __fmaf_rn(e, ln2h, tl);
  // e^t - 1 = t + t^2 / 2 + ..., t and t^2 / 2 as pairs
  const float sq = __fmul_rn(th, th);
  const float sqe = __fmaf_rn(th, tl + tl, __fmaf_rn(th, th, -sq));
  const float c3 = __fmul_rn(__fmul_rn(sq, th), __fmaf_rn(th, __fmaf_rn(th, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f));
  const float h = 0.5f * sq;
  const float sh = __fadd_rn(th, h);
  const float se = __fadd_rn(h, -__fadd_rn(sh, -th));
  const float sl = __fadd_rn(se, __fadd_rn(c3, __fmaf_rn(0.5f, sqe, tl)));
  // times 2^(j / 32)
  const float2 t = s_exp2[m & 31];
  const float ph = __fmul_rn(t.x, sh);
  float pl = __fmaf_rn(t.x, sh, -ph);
  pl = __fmaf_rn(t.x, sl, pl);
  pl = __fmaf_rn(t.y, sh, pl);
  Weight w;
  w.h = __fadd_rn(t.x, ph);
  w.l = __fadd_rn(__fadd_rn(__fadd_rn(ph, -__fadd_rn(w.h, -t.x)), pl), t.y);
  w.n = none ? -200 : m >> 5;
  return w;
}
// Called where one weight is wanted; where four are, they are worked out side by side.
__device__ __noinline__ Weight weight_at(float l, float most, float ch, float cl, const float2* s_exp2) {
  return weight_here(l, RowScale{most, ch, cl}, s_exp2);
}
__device__ __forceinline__ Weight weight_of(float l, const RowScale& r, const float2* s_exp2) {
  return weight_at(l, r.most, r.ch, r.cl, s_exp2);
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_cluster_u2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void st_cluster_2u64(uint32_t addr, uint64_t a, uint64_t b) {
  asm volatile("st.shared::cluster.v2.u64 [%0], {%1, %2};" ::"r"(addr), "l"(a), "l"(b) : "memory");
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

struct SampleArgs {
  const uint16_t* logits;
  int64_t stride;
  int rows, V, slice;  // slice: tokens of a CTA, a multiple of 8
  sd_sampling s;
  const float* u;
  int32_t* tokens;
  float* logprob;
  int32_t* kept;
};

struct SampleShared {
  uint32_t bins[32768];           // counters of keys 2 i and 2 i + 1
  uint64_t weight[sp::kTable][128];  // of the first CTA: the row's keys by falling logit, weights
  uint32_t keys[sp::kTable][128];    // and counts
  uint64_t mass[sp::kBlocks];     // of the binades that occur, by falling logit: sums of weights, and counts;
  uint32_t count[sp::kBlocks];    // then running ones
  float2 exp2[32];
  float top[sp::kWarps];
  uint32_t lo[sp::kWarps], hi[sp::kWarps];
  uint32_t span[3];               // of the CTA: greatest logit (fp32 bits), least and greatest magnitude
  uint32_t key, nth;              // the token's key and which of the CTA's occurrences it is (-1: none here)
  uint32_t tot[8 * sp::kWarps];   // occurrences a round of vectors and warp
};

// The binades that occur, by falling logit: those of magnitudes e1 .. e0, zero's
// and the subnormals' (0), then the negative ones.
struct Binades {
  int e0, e1;
  __device__ __forceinline__ int n() const { return 2 * (e1 - e0 + 1) + (e0 > 0); }
  // raw bits of the binade's first key, the greatest; the others follow by step
  __device__ __forceinline__ uint32_t exponent(int i, bool& neg) const {
    const int m = e1 - e0 + 1;
    neg = i >= m + (e0 > 0);
    return neg ? e0 + (i - m - (e0 > 0)) : i < m ? e1 - i : 0;
  }
};

// Key `j` of 0 .. 127 of a binade in falling order, as raw bits.
__device__ __forceinline__ uint32_t key_bits(uint32_t e, bool neg, int j) {
  return (neg ? 0x8000u : 0u) | e << 7 | (neg ? j : 127 - j);
}

// The counts of a lane's four keys 4 lane .. 4 lane + 3 (falling order) of a
// binade, over the cluster.
template <int C>
__device__ __forceinline__ void lane_counts(uint32_t bins, uint32_t e, bool neg, int lane, uint32_t (&c)[4]) {
  const uint32_t word = ((neg ? 0x8000u : 0u) | e << 7) / 2 + (neg ? 2 * lane : 62 - 2 * lane);
  uint2 w[C];
#pragma unroll
  for (int k = 0; k < C; k++) w[k] = ld_cluster_u2(cluster_map(bins + 4 * word, k));
  c[0] = c[1] = c[2] = c[3] = 0;
#pragma unroll
  for (int k = 0; k < C; k++) c[0] += w[k].x & 0xFFFF, c[1] += w[k].x >> 16, c[2] += w[k].y & 0xFFFF, c[3] += w[k].y >> 16;
  if (!neg) {
    const uint32_t a = c[0], b = c[1];
    c[0] = c[3], c[1] = c[2], c[2] = b, c[3] = a;
  }
}
// Their weights too.
template <int C>
__device__ __forceinline__ void lane_keys(uint32_t bins, const Binades& b, int i, const RowScale& rs, const float2* s_exp2, int lane,
                                          uint32_t (&k)[4], uint64_t (&w)[4]) {
  bool neg;
  const uint32_t e = b.exponent(i, neg);
  lane_counts<C>(bins, e, neg, lane, k);
#pragma unroll
  for (int x = 0; x < 4; x++) {
    const uint64_t v = weight_here(bf2f((uint16_t)key_bits(e, neg, 4 * lane + x)), rs, s_exp2).whole();
    w[x] = k[x] ? v : 0;  // a key that does not occur may lie above the greatest logit
  }
}

// Sums of `v` over the lanes before this one.
template <typename T>
__device__ __forceinline__ T before_lane(T v, int lane) {
  T run = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T x = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += x;
  }
  return run - v;
}

// ceil or floor of p W for a float 0 <= p < 1.
__device__ __noinline__ uint64_t share_of(float p, uint64_t W, bool up) {
  if (!(p > 0.f)) return 0;
  const uint32_t b = __float_as_uint(p);
  const int e = b >> 23;
  const uint64_t m = (b & 0x7FFFFF) | (e ? 0x800000 : 0);
  const int k = 150 - (e ? e : 1);  // p = m 2^-k, k >= 24
  const uint64_t lo = m * W, hi = __umul64hi(m, W);
  uint64_t q, rest;
  if (k < 64) {
    q = hi << (64 - k) | lo >> k;
    rest = lo << (64 - k);
  } else {
    q = k < 128 ? hi >> (k - 64) : 0;
    rest = (k < 128 ? hi << 1 << (127 - k) : hi) | lo;
  }
  return q + (up && rest);
}

// A place in the falling order: binade i, key j.
struct Place {
  int i, j;
  uint64_t count, mass;  // before key j
  uint64_t w;            // the key's weight
};

// The row's keys as the cluster's first CTA keeps them.
struct LaneKeys {
  uint32_t k[4];
  uint64_t w[4];
};
template <int C>
__device__ __noinline__ LaneKeys keys_not_kept(uint32_t bins, int e0, int e1, int i, float most, float ch, float cl, const float2* s_exp2) {
  LaneKeys r;
  lane_keys<C>(bins, Binades{e0, e1}, i, RowScale{most, ch, cl}, s_exp2, threadIdx.x & 31, r.k, r.w);
  return r;
}
template <int C>
struct ClusterKeys {
  const SampleShared& sh;
  uint32_t bins;
  Binades b;
  const RowScale& rs;
  __device__ __forceinline__ int n() const { return b.n(); }
  __device__ __forceinline__ uint32_t bits(int i, int j) const {
    bool neg;
    const uint32_t e = b.exponent(i, neg);
    return key_bits(e, neg, j);
  }
  __device__ __forceinline__ void lane_of(int i, int lane, uint32_t (&k)[4], uint64_t (&w)[4]) const {
    if (i >= sp::kTable) {
      const LaneKeys r = keys_not_kept<C>(bins, b.e0, b.e1, i, rs.most, rs.ch, rs.cl, sh.exp2);
#pragma unroll
      for (int x = 0; x < 4; x++) k[x] = r.k[x], w[x] = r.w[x];
      return;
    }
    const uint4 c = reinterpret_cast<const uint4*>(sh.keys[i])[lane];
    const ulonglong2 u = reinterpret_cast<const ulonglong2*>(sh.weight[i])[2 * lane],
                     v = reinterpret_cast<const ulonglong2*>(sh.weight[i])[2 * lane + 1];
    k[0] = c.x, k[1] = c.y, k[2] = c.z, k[3] = c.w;
    w[0] = u.x, w[1] = u.y, w[2] = v.x, w[3] = v.y;
  }
};

// The row kernel's counters: of positive keys, negative ones, zero.
struct RowKeys {
  const uint32_t* bins;
  const float2* exp2;
  RowScale rs;
  __device__ __forceinline__ int n() const { return sp::kRowBlocks; }
  __device__ __forceinline__ uint32_t bits(int i, int j) const {
    if (i == sp::kSpan) return 0;
    const bool neg = i > sp::kSpan;
    return key_bits(neg ? sp::kLeast + i - sp::kSpan - 1 : sp::kLeast + sp::kSpan - 1 - i, neg, j);
  }
  __device__ __forceinline__ void counts(int i, int lane, uint32_t (&k)[4]) const {
    if (i == sp::kSpan) {
      k[0] = lane == 0 ? bins[2 * sp::kRowKeys] : 0;
      k[1] = k[2] = k[3] = 0;
    } else if (i > sp::kSpan) {
      const uint4 u = *reinterpret_cast<const uint4*>(bins + sp::kRowKeys + (i - sp::kSpan - 1) * 128 + 4 * lane);
      k[0] = u.x, k[1] = u.y, k[2] = u.z, k[3] = u.w;
    } else {
      const uint4 u = *reinterpret_cast<const uint4*>(bins + (sp::kSpan - 1 - i) * 128 + 124 - 4 * lane);
      k[0] = u.w, k[1] = u.z, k[2] = u.y, k[3] = u.x;
    }
  }
  __device__ __forceinline__ void lane_of(int i, int lane, uint32_t (&k)[4], uint64_t (&w)[4]) const {
    counts(i, lane, k);
#pragma unroll
    for (int x = 0; x < 4; x++) {
      const uint64_t v = weight_here(bf2f((uint16_t)bits(i, 4 * lane + x)), rs, exp2).whole();
      w[x] = k[x] ? v : 0;
    }
  }
};

// By one warp: the first key at which the row's running count (or mass)
// reaches `goal` (at least goal, or more than it where `past`).  The caller knows
// that it does.
template <typename Keys>
__device__ __forceinline__ Place find(const Keys& keys, const uint32_t* count, const uint64_t* mass, uint64_t goal, bool by_mass, bool past) {
  const int lane = threadIdx.x & 31, n = keys.n();
  auto reached = [&](uint64_t c, uint64_t m) {
    const uint64_t x = by_mass ? m : c;
    return past ? x > goal : x >= goal;
  };
  Place p = {};
#pragma unroll 1
  for (int c = 0; c < n; c += 32) {
    const int i = min(c + lane, n - 1);
    const uint32_t f = __ballot_sync(0xffffffffu, reached(count[i], mass[i]));
    if (f) {
      p.i = min(c + __ffs(f) - 1, n - 1);
      break;
    }
  }
  uint64_t cb = p.i ? count[p.i - 1] : 0, mb = p.i ? mass[p.i - 1] : 0;
  uint32_t k[4], c = 0;
  uint64_t w[4], m = 0;
  keys.lane_of(p.i, lane, k, w);
#pragma unroll
  for (int x = 0; x < 4; x++) c += k[x], m += k[x] * w[x];
  cb += before_lane(c, lane);
  mb += before_lane(m, lane);
  const int at = max(__ffs(__ballot_sync(0xffffffffu, c > 0 && reached(cb + c, mb + m))) - 1, 0);
  int j = 0;
  uint64_t ww = 0;
#pragma unroll
  for (int x = 0; x < 4; x++) {  // the first of the lane's keys that reaches it
    const bool before = j == x && !(k[x] && reached(cb + k[x], mb + k[x] * w[x]));
    if (before && x < 3) cb += k[x], mb += k[x] * w[x], j = x + 1;
    if (j == x) ww = w[x];
  }
  p.j = 4 * at + __shfl_sync(0xffffffffu, j, at);
  p.count = __shfl_sync(0xffffffffu, cb, at);
  p.mass = __shfl_sync(0xffffffffu, mb, at);
  p.w = __shfl_sync(0xffffffffu, ww, at);
  return p;
}

struct RowSettings {
  float temperature, top_p, min_p, u;
  int top_k;
  __device__ __forceinline__ RowSettings(const sd_sampling& s, const float* us, int row) {
    temperature = s.temperature_rows ? s.temperature_rows[row] : s.temperature;
    top_p = s.top_p_rows ? s.top_p_rows[row] : s.top_p;
    min_p = s.min_p_rows ? s.min_p_rows[row] : s.min_p;
    top_k = s.top_k_rows ? s.top_k_rows[row] : s.top_k;
    u = us[row];
  }
  __device__ __forceinline__ RowScale scale(float most) const {  // log2(e) / temperature: the quotient and its remainder's
    constexpr float lh = (float)1.4426950408889634074, ll = (float)(1.4426950408889634074 - (double)lh);
    const float q = __fdiv_rn(lh, temperature);
    RowScale r = {most, temperature > 0.f ? 2.f * q : 0.f, 0.f};
    // (infinitely large or below 2^-126: every weight is 1, or all but the greatest's 0)
    if (q > 0.f && temperature >= 0x1p-126f) r.cl = 2.f * __fdiv_rn(__fadd_rn(__fmaf_rn(-q, temperature, lh), ll), temperature);
    if (temperature > 0.f && temperature < 0x1p-126f) r.ch = INFINITY;
    return r;
  }
};

struct Chosen {
  uint32_t key, r;   // the token's key and which of its occurrences it is
  uint64_t w, W;     // its weight, the sum of what is kept
  uint32_t N;        // how many are kept
};

// By one warp: the cuts and the token's key, from the binades' counts and sums
// (which become running ones).
template <typename Keys>
__device__ __forceinline__ Chosen walk(const Keys& keys, uint32_t* count, uint64_t* mass, const RowScale& rs, const float2* exp2,
                                       const RowSettings& set) {
  const int lane = threadIdx.x & 31;
  // a run of binades a lane
  const int n = keys.n(), each = (n + 31) / 32, i0 = min(n, lane * each), i1 = min(n, i0 + each);
  uint32_t c = 0;
  uint64_t m = 0;
#pragma unroll 1
  for (int i = i0; i < i1; i++) c += count[i], m += mass[i];
  uint32_t cb = before_lane(c, lane);
  uint64_t mb = before_lane(m, lane);
#pragma unroll 1
  for (int i = i0; i < i1; i++) {
    cb += count[i], mb += mass[i];
    count[i] = cb, mass[i] = mb;
  }
  __syncwarp();
  uint64_t N = count[n - 1], W = mass[n - 1];
  const uint64_t K = !(set.temperature > 0.f) ? 1 : set.top_k > 0 ? set.top_k : N;
  Place p = {};
  // top-k, min-p, top-p, the token: one search after the other
#pragma unroll 1
  for (int stage = 0; stage < 4; stage++) {
    if (stage == 1) {
      if (!(set.min_p > 0.f)) continue;
      const float least = fminf(set.min_p, 1.f);
      // the first binade whose last key weighs less
      int i = n;
#pragma unroll 1
      for (int b = 0; b < n && i == n; b += 32) {
        const bool below = b + lane < n && !weight_of(bf2f((uint16_t)keys.bits(min(b + lane, n - 1), 127)), rs, exp2).at_least(least);
        const uint32_t f = __ballot_sync(0xffffffffu, below);
        if (f) i = b + __ffs(f) - 1;
      }
      if (i == n) continue;
      uint32_t k[4], cc = 0;
      uint64_t w[4], mm = 0;
      keys.lane_of(i, lane, k, w);
#pragma unroll
      for (int x = 0; x < 4; x++)
        if (weight_of(bf2f((uint16_t)keys.bits(i, 4 * lane + x)), rs, exp2).at_least(least)) cc += k[x], mm += k[x] * w[x];
      cc = __reduce_add_sync(0xffffffffu, cc) + (i ? count[i - 1] : 0);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mm += __shfl_xor_sync(0xffffffffu, mm, o);
      mm += i ? mass[i - 1] : 0;
      if (cc < N) N = cc, W = mm;
      continue;
    }
    if ((stage == 0 && K >= N) || (stage == 2 && !(set.top_p < 1.f))) continue;
    const float u = set.u > 0.f ? fminf(set.u, 1.f - 0x1p-24f) : 0.f;
    uint64_t goal = K;
    if (stage) {
      goal = share_of(stage == 2 ? set.top_p : u, W, stage == 2);
      if (stage == 2 && goal == 0) goal = 1;
    }
    p = find(keys, count, mass, goal, stage > 0, stage == 3);
    if (stage == 0) {
      N = K;
      W = p.mass + (K - p.count) * p.w;
      continue;
    }
    const uint64_t r = (goal - p.mass + (stage == 2 ? p.w - 1 : 0)) / p.w;
    if (stage == 2) {
      if (p.count + r < N) N = p.count + r, W = p.mass + r * p.w;
    } else {
      p.count = r;
    }
  }
  return {keys.bits(p.i, p.j), (uint32_t)p.count, p.w, W, (uint32_t)N};
}

// The token's logarithm and the count (by one thread).
__device__ __forceinline__ void write_row(const SampleArgs& a, int row, const Chosen& ch, const RowScale& rs, const float2* exp2) {
  if (a.logprob) a.logprob[row] = 0.f - log1pf((float)(ch.W - ch.w) * 0x1p-44f / weight_of(bf2f((uint16_t)ch.key), rs, exp2).value());
  if (a.kept) a.kept[row] = (int32_t)ch.N;
}
__device__ __forceinline__ void write_empty(const SampleArgs& a, int row) {
  a.tokens[row] = -1;
  if (a.logprob) a.logprob[row] = -INFINITY;
  if (a.kept) a.kept[row] = 0;
}

__device__ __forceinline__ void tally(SampleShared& sh, uint32_t b, float& top, uint32_t& lo, uint32_t& hi) {
  const uint32_t mag = b & 0x7FFFu;
  if (mag > 0x7F80u || b == 0xFF80u) return;
  if (mag == 0) b = 0;  // -0 is 0
  atomicAdd(&sh.bins[b >> 1], b & 1 ? 0x10000u : 1u);
  top = fmaxf(top, __uint_as_float(b << 16));
  lo = min(lo, mag - 1);  // zero is the greatest
  hi = max(hi, mag);
}

// Eight tokens from t on, NaN where the row x of V tokens has none.
__device__ __noinline__ uint4 edge_vector(const uint16_t* x, int t, int V) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 8; k++) {
    const uint32_t e = t + k >= 0 && t + k < V ? x[t + k] : 0xFFFFu;
    w[k / 2] = k & 1 ? w[k / 2] | e << 16 : e;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A row as vectors of eight tokens on 16-byte addresses, its ends masked.
struct RowView {
  const uint16_t* x;
  const uint4* xv;
  int shift, V;  // tokens before x in its vector
  __device__ __forceinline__ RowView(const SampleArgs& a, int row) : x(a.logits + (int64_t)row * a.stride), V(a.V) {
    shift = (int)((reinterpret_cast<uintptr_t>(x) >> 1) & 7);
    xv = reinterpret_cast<const uint4*>(x - shift);
  }
  __device__ __forceinline__ int vectors() const { return (V + shift + 7) / 8; }
  __device__ __forceinline__ int token(int v, int k) const { return v * 8 + k - shift; }
  // vector v, NaN at and past `end`
  __device__ __forceinline__ void load(int v, int end, uint32_t (&w)[4]) const {
    uint4 u = make_uint4(0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu);
    if (v < end) {
      if (token(v, 0) >= 0 && token(v, 7) < V) u = xv[v];
      else u = edge_vector(x, token(v, 0), V);
    }
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  }
};
// The elements of a vector that are the key, as bits; -0 is 0.
__device__ __forceinline__ uint32_t matches(const uint32_t (&w)[4], uint32_t key) {
  const uint32_t both = key * 0x10001u, of = key == 0 ? 0x7FFF7FFFu : 0xFFFFFFFFu;
  uint32_t f = 0;
#pragma unroll
  for (int k = 0; k < 4; k++) {
    const uint32_t x = (w[k] & of) ^ both;  // bit 15 of a half below: it is zero
    const uint32_t z = ~(((x & 0x7FFF7FFFu) + 0x7FFF7FFFu) | x) & 0x80008000u;
    f |= z >> (15 - 2 * k);                 // elements 2 k at bit 2 k, 2 k + 1 at bit 16 + 2 k
  }
  return (f & 0x55u) | (f >> 15 & 0xAAu);
}
// By one warp: the token of occurrence nth of the key in vectors v0 .. end of a row, of
// which round i's by warp w are tot[i * WARPS + w].
template <int WARPS>
__device__ __forceinline__ void look_up(const SampleArgs& a, int row, const RowView& rv, int v0, int end, int rounds, const uint32_t* tot,
                                        uint32_t key, uint32_t nth) {
  const int lane = threadIdx.x & 31, n = rounds * WARPS;
  uint32_t run = 0;
#pragma unroll 1
  for (int c = 0; c < n; c += 32) {
    const uint32_t m = c + lane < n ? tot[c + lane] : 0, b = run + before_lane(m, lane);
    const uint32_t f = __ballot_sync(0xffffffffu, nth >= b && nth < b + m);
    run = __shfl_sync(0xffffffffu, b + m, 31);
    if (!f) continue;
    const int where = c + __ffs(f) - 1;
    const uint32_t left = nth - __shfl_sync(0xffffffffu, b, __ffs(f) - 1);
    const int v = v0 + (where / WARPS * WARPS + where % WARPS) * 32 + lane;
    uint32_t w[4];
    rv.load(v, end, w);
    uint32_t g = matches(w, key);
    const uint32_t h = __popc(g), before = before_lane(h, lane);
    if (left >= before && left < before + h) {
      for (uint32_t k = before; k < left; k++) g &= g - 1;
      a.tokens[row] = rv.token(v, __ffs(g) - 1);
    }
    return;
  }
}

// A cluster a row.  `only`: the rows that the row kernel left.
template <int C>
__global__ void __launch_bounds__(sp::kThreads, 1) k_sample(const __grid_constant__ SampleArgs a, bool only) {
  extern __shared__ __align__(16) uint8_t smem_sp[];
  SampleShared& sh = *reinterpret_cast<SampleShared*>(smem_sp);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster_rank();
  if (only) {  // none of this cluster's rows (which only it changes) is left: the rule
    pdl_wait();
    bool left = false;
    for (int64_t r = blockIdx.x / C + (int64_t)tid * (gridDim.x / C); r < a.rows; r += (int64_t)sp::kThreads * (gridDim.x / C))
      left |= a.tokens[r] == sp::kLater;
    if (!__syncthreads_or(left)) return;
  }
#pragma unroll 1
  for (int row = blockIdx.x / C; row < a.rows; row += gridDim.x / C) {
    if (only && a.tokens[row] != sp::kLater) continue;
    __syncthreads();
    // ---- count the slice
    const RowView rv(a, row);
    const int v0 = rank * (a.slice / 8), v1 = min(rv.vectors(), v0 + a.slice / 8);
    uint32_t held[sp::kHeld][4];  // all of a thread's loads in flight while the counters are cleared
#pragma unroll
    for (int i = 0; i < sp::kHeld; i++) rv.load(v0 + i * sp::kThreads + tid, v1, held[i]);
    const RowSettings set(a.s, a.u, row);
#pragma unroll
    for (int i = 0; i < 8; i++) reinterpret_cast<uint4*>(sh.bins)[tid + i * sp::kThreads] = make_uint4(0, 0, 0, 0);
    if (tid < 32) sh.exp2[tid] = make_float2(kExp2.hi[tid], kExp2.lo[tid]);
    __syncthreads();
    float top = -INFINITY;
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    auto tally4 = [&](const uint32_t (&w)[4]) {
#pragma unroll
      for (int k = 0; k < 4; k++) tally(sh, w[k] & 0xFFFF, top, lo, hi), tally(sh, w[k] >> 16, top, lo, hi);
    };
#pragma unroll
    for (int i = 0; i < sp::kHeld; i++) tally4(held[i]);
#pragma unroll 1
    for (int v = v0 + sp::kHeld * sp::kThreads + tid; v < v1; v += sp::kThreads) {
      uint32_t w[4];
      rv.load(v, v1, w);
      tally4(w);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) sh.top[warp] = top, sh.lo[warp] = lo, sh.hi[warp] = hi;
    __syncthreads();
    if (warp == 0) {
      top = sh.top[lane];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      lo = __reduce_min_sync(0xffffffffu, sh.lo[lane]);
      hi = __reduce_max_sync(0xffffffffu, sh.hi[lane]);
      if (lane == 0) sh.span[0] = __float_as_uint(top), sh.span[1] = lo, sh.span[2] = hi;
    }
    cluster_sync_all();

    // ---- the row's greatest logit and its binades
    const uint32_t bins = smem_u32(sh.bins), span = smem_u32(sh.span);
    top = -INFINITY, lo = 0xFFFFFFFFu, hi = 0;
#pragma unroll
    for (int k = 0; k < C; k++) {
      const uint32_t at = cluster_map(span, k);
      top = fmaxf(top, __uint_as_float(ld_cluster_u32(at)));
      lo = min(lo, ld_cluster_u32(at + 4));
      hi = max(hi, ld_cluster_u32(at + 8));
    }
    const bool none = top == -INFINITY;
    Binades bn;
    bn.e1 = hi >> 7;
    bn.e0 = min((int)((lo == 0xFFFFFFFFu ? 0u : lo + 1) >> 7), bn.e1);
    const RowScale rs = set.scale(top);

    // ---- each binade's keys, count and sum, into the first CTA
    if (!none) {
      const uint32_t mass0 = cluster_map(smem_u32(sh.mass), 0), count0 = cluster_map(smem_u32(sh.count), 0);
      const uint32_t keys0 = cluster_map(smem_u32(sh.keys), 0), weight0 = cluster_map(smem_u32(sh.weight), 0);
#pragma unroll 1
      for (int i = warp * C + rank; i < bn.n(); i += sp::kWarps * C) {
        uint32_t c[4], n = 0;
        uint64_t w[4], m = 0;
        lane_keys<C>(bins, bn, i, rs, sh.exp2, lane, c, w);
#pragma unroll
        for (int k = 0; k < 4; k++) n += c[k], m += c[k] * w[k];
        if (i < sp::kTable) {
          const uint32_t at = i * 128 + 4 * lane;
          st_cluster_u4(keys0 + 4 * at, c[0], c[1], c[2], c[3]);
          st_cluster_2u64(weight0 + 8 * at, w[0], w[1]);
          st_cluster_2u64(weight0 + 8 * at + 16, w[2], w[3]);
        }
        n = __reduce_add_sync(0xffffffffu, n);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
        if (lane == 0) st_cluster_u64(mass0 + 8 * i, m), st_cluster_u32(count0 + 4 * i, n);
      }
    }
    cluster_sync_all();

    // ---- the cuts and the token's key, by one warp
    if (rank == 0 && warp == 0) {
      if (!none) {
        const Chosen ch = walk(ClusterKeys<C>{sh, bins, bn, rs}, sh.count, sh.mass, rs, sh.exp2, set);
        // the CTA that holds the occurrence
        uint32_t mine = 0;
        if (lane < C) mine = ld_cluster_u32(cluster_map(bins + 4 * (ch.key >> 1), lane)) >> (ch.key & 1 ? 16 : 0) & 0xFFFF;
        const uint32_t before = before_lane(mine, lane);
        if (lane < C) {
          const uint32_t to = cluster_map(smem_u32(&sh.key), lane);
          st_cluster_u32(to, ch.key);
          st_cluster_u32(to + 4, ch.r >= before && ch.r < before + mine ? ch.r - before : 0xFFFFFFFFu);
        }
        if (lane == 0) write_row(a, row, ch, rs, sh.exp2);
      } else {
        if (lane < C) st_cluster_u32(cluster_map(smem_u32(&sh.nth), lane), 0xFFFFFFFFu);
        if (lane == 0) write_empty(a, row);
      }
    }
    cluster_sync_all();

    // ---- occurrence nth of the key in this slice
    const uint32_t key = sh.key, nth = sh.nth;
    if (nth == 0xFFFFFFFFu) continue;
    const int rounds = (v1 - v0 + sp::kThreads - 1) / sp::kThreads;  // at most 8
#pragma unroll
    for (int i = 0; i < sp::kHeld; i++) {
      if (i >= rounds) break;
      const uint32_t n = __reduce_add_sync(0xffffffffu, __popc(matches(held[i], key)));
      if (lane == 0) sh.tot[i * sp::kWarps + warp] = n;
    }
#pragma unroll 1
    for (int i = sp::kHeld; i < rounds; i++) {
      uint32_t w[4];
      rv.load(v0 + i * sp::kThreads + tid, v1, w);
      const uint32_t n = __reduce_add_sync(0xffffffffu, __popc(matches(w, key)));
      if (lane == 0) sh.tot[i * sp::kWarps + warp] = n;
    }
    __syncthreads();
    if (warp == 0) look_up<sp::kWarps>(a, row, rv, v0, v1, rounds, sh.tot, key, nth);
  }
}

struct RowShared {
  uint32_t bins[2 * sp::kRowKeys + 4];  // counters: positive keys, negative ones, zero
  uint64_t mass[sp::kRowBlocks + 1];
  uint32_t count[sp::kRowBlocks + 1];
  float2 exp2[32];
  uint32_t other, key, nth;
  uint32_t tot[8 * sp::kRowWarps];      // occurrences a round of vectors and warp
  uint32_t done[sp::kRowWarps];
};

// A CTA a row.
__global__ void __launch_bounds__(sp::kRowThreads, 2) k_sample_row(const __grid_constant__ SampleArgs a) {
  extern __shared__ __align__(16) uint8_t smem_sp[];
  RowShared& sh = *reinterpret_cast<RowShared*>(smem_sp);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, row = blockIdx.x;
  const RowView rv(a, row);
  const int end = rv.vectors();
  constexpr int U = 4;  // vectors of a thread in flight, twice
  uint32_t w[U][4];
#pragma unroll
  for (int i = 0; i < U; i++) rv.load(tid + i * sp::kRowThreads, end, w[i]);
  const RowSettings set(a.s, a.u, row);
  for (int i = tid; i < 2 * sp::kRowKeys / 4 + 1; i += sp::kRowThreads) reinterpret_cast<uint4*>(sh.bins)[i] = make_uint4(0, 0, 0, 0);
  if (tid < 32) sh.exp2[tid] = make_float2(kExp2.hi[tid], kExp2.lo[tid]);
  if (tid == 0) sh.other = 0;
  __syncthreads();
  bool other = false;  // a magnitude that has no counter
  auto count1 = [&](uint32_t b) {
    const uint32_t mag = b & 0x7FFFu, i = mag - (sp::kLeast << 7);
    if (i < (uint32_t)sp::kRowKeys) {
      atomicAdd(&sh.bins[i + (b >> 15) * sp::kRowKeys], 1u);
    } else if (mag == 0) {
      atomicAdd(&sh.bins[2 * sp::kRowKeys], 1u);
    } else if (mag <= 0x7F80u && b != 0xFF80u) {
      other = true;
    }
  };
  auto count8 = [&](const uint32_t (&w)[4]) {
    // bit 15 of a half: its magnitude has a counter
    constexpr uint32_t least = sp::kLeast << 7, past = least + sp::kRowKeys;
    uint32_t in = 0x80008000u;
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const uint32_t m = w[k] & 0x7FFF7FFFu;
      in &= (m + (0x8000u - least) * 0x10001u) & ~(m + (0x8000u - past) * 0x10001u);
    }
    if (in == 0x80008000u) {
      uint32_t* const at = sh.bins - least;
#pragma unroll
      for (int k = 0; k < 4; k++) {  // a negative key's counter: its bits less what lies between
        const uint32_t b = w[k] & 0xFFFFu, c = w[k] >> 16;
        atomicAdd(at + (int)(b - (b >> 15) * (0x8000u - sp::kRowKeys)), 1u);
        atomicAdd(at + (int)(c - (c >> 15) * (0x8000u - sp::kRowKeys)), 1u);
      }
    } else {
#pragma unroll 1
      for (int k = 0; k < 8; k++) count1((k < 4 ? k < 2 ? w[0] : w[1] : k < 6 ? w[2] : w[3]) >> 16 * (k & 1) & 0xFFFF);
    }
  };
#pragma unroll 1
  for (int v = tid; v < end; v += U * sp::kRowThreads) {
    uint32_t next[U][4];
#pragma unroll
    for (int i = 0; i < U; i++) rv.load(v + (U + i) * sp::kRowThreads, end, next[i]);
#pragma unroll
    for (int i = 0; i < U; i++) count8(w[i]);
#pragma unroll
    for (int i = 0; i < U; i++) {
#pragma unroll
      for (int k = 0; k < 4; k++) w[i][k] = next[i][k];
    }
  }
  if (__any_sync(0xffffffffu, other) && lane == 0) sh.other = 1;
  __syncthreads();
  if (sh.other) {
    if (tid == 0) a.tokens[row] = sp::kLater;
    return;
  }

  // ---- the binades' counts, the greatest logit, their sums
  RowKeys keys = {sh.bins, sh.exp2, {}};
  constexpr int kEach = (sp::kRowBlocks + sp::kRowWarps - 1) / sp::kRowWarps;
  uint32_t sums[kEach];
#pragma unroll
  for (int e = 0; e < kEach; e++) {
    uint32_t k[4];
    keys.counts(min(warp + e * sp::kRowWarps, sp::kRowBlocks - 1), lane, k);
    sums[e] = __reduce_add_sync(0xffffffffu, k[0] + k[1] + k[2] + k[3]);
  }
  if (lane == 0) {
#pragma unroll
    for (int e = 0; e < kEach; e++)
      if (warp + e * sp::kRowWarps < sp::kRowBlocks) sh.count[warp + e * sp::kRowWarps] = sums[e];
  }
  __syncthreads();
  int first = -1;
#pragma unroll
  for (int c = 0; c < sp::kRowBlocks; c += 32) {
    const uint32_t f = __ballot_sync(0xffffffffu, c + lane < sp::kRowBlocks && sh.count[c + lane] > 0);
    if (first < 0 && f) first = c + __ffs(f) - 1;
  }
  if (first < 0) {
    if (tid == 0) write_empty(a, row);
    return;
  }
  {
    uint32_t k[4];
    keys.counts(first, lane, k);
    const uint32_t j = __reduce_min_sync(0xffffffffu, k[0] ? 4 * lane : k[1] ? 4 * lane + 1 : k[2] ? 4 * lane + 2 : k[3] ? 4 * lane + 3 : 128);
    keys.rs = set.scale(bf2f((uint16_t)keys.bits(first, j)));
  }
#pragma unroll 1
  for (int i = warp; i < sp::kRowBlocks; i += sp::kRowWarps) {
    uint64_t m = 0;
    if (sh.count[i]) {
      uint32_t k[4];
      uint64_t x[4];
      keys.lane_of(i, lane, k, x);
#pragma unroll
      for (int e = 0; e < 4; e++) m += k[e] * x[e];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
    }
    if (lane == 0) sh.mass[i] = m;
  }
  __syncthreads();
  if (warp == 0) {
    const Chosen ch = walk(keys, sh.count, sh.mass, keys.rs, sh.exp2, set);
    if (lane == 0) {
      sh.key = ch.key, sh.nth = ch.r;
      write_row(a, row, ch, keys.rs, sh.exp2);
    }
  }
  __syncthreads();
  pdl_launch();
  const uint32_t key = sh.key, nth = sh.nth;
  const int rounds = (end + sp::kRowThreads - 1) / sp::kRowThreads;
  uint32_t before = 0;  // occurrences in the rounds done
#pragma unroll 1
  for (int i = 0; i < rounds; i += 2 * U) {
    uint32_t x[2 * U][4], all = 0;
#pragma unroll
    for (int j = 0; j < 2 * U; j++) rv.load((i + j) * sp::kRowThreads + tid, end, x[j]);
#pragma unroll
    for (int j = 0; j < 2 * U; j++) {
      const uint32_t n = __reduce_add_sync(0xffffffffu, __popc(matches(x[j], key)));
      if (lane == 0) sh.tot[j * sp::kRowWarps + warp] = n;  // none past the row's end
      all += n;
    }
    if (lane == 0) sh.done[warp] = all;
    __syncthreads();
    const uint32_t here = __reduce_add_sync(0xffffffffu, lane < sp::kRowWarps ? sh.done[lane] : 0u);
    if (nth < before + here) {
      if (warp == 0) look_up<sp::kRowWarps>(a, row, rv, i * sp::kRowThreads, end, 2 * U, sh.tot, key, nth - before);
      return;
    }
    before += here;
    __syncthreads();
  }
}

static int sample_bad(int code, const char* what) {
  set_error(std::string("sd_sample: ") + what);
  return code;
}

}  // namespace sdv

using namespace sdv;

extern "C" int sd_sample(const uint16_t* logits, int64_t row_stride, int32_t rows, int32_t vocab,
                         const sd_sampling* settings, const float* u, int32_t* tokens, float* logprob, int32_t* kept,
                         void* stream) {
  if (rows < 0 || vocab < 1) return sample_bad(SD_ERR_INVALID_ARG, "rows >= 0 and vocab >= 1 are needed");
  if (vocab > sp::kMaxVocab) return sample_bad(SD_ERR_UNSUPPORTED, "vocab must be at most 524160");
  if (!settings) return sample_bad(SD_ERR_INVALID_ARG, "null settings");
  const sd_sampling& s = *settings;
  if ((!s.temperature_rows && !(s.temperature >= 0.f && s.temperature <= 3e38f)) || (!s.top_k_rows && s.top_k < 0) ||
      (!s.top_p_rows && !(s.top_p > 0.f)) || (!s.min_p_rows && !(s.min_p >= 0.f && s.min_p <= 1.f)))
    return sample_bad(SD_ERR_INVALID_ARG, "temperature and top_k must not be negative, top_p must be positive, min_p in [0, 1]");
  if (rows == 0) return SD_OK;
  if (!logits || !u || !tokens) return sample_bad(SD_ERR_INVALID_ARG, "null argument");
  if (rows > 1 && row_stride < vocab) return sample_bad(SD_ERR_INVALID_ARG, "row_stride is shorter than a row");
  if ((uintptr_t)logits & 1) return sample_bad(SD_ERR_INVALID_ARG, "logits must be 2-byte aligned");
  const int vecs = (vocab + 7 + 7) / 8;  // a row may begin anywhere in its first vector
  auto slice = [&](int c) { return (vecs + c - 1) / c * 8; };
  // clusters of 1, 2, 4 and 8 CTAs that the card holds at once (of 8 fewer than its SMs /
  // 8: a cluster lies within one group of SMs)
  static int held[4] = {};
  static const cudaError_t set = []() {
    const void* kerns[4] = {(const void*)k_sample<1>, (const void*)k_sample<2>, (const void*)k_sample<4>, (const void*)k_sample<8>};
    cudaError_t e = cudaFuncSetAttribute(k_sample_row, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(RowShared));
    for (int i = 0; i < 4; i++) {
      if (e == cudaSuccess) e = cudaFuncSetAttribute(kerns[i], cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SampleShared));
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(1u << i), cfg.blockDim = dim3(sp::kThreads), cfg.dynamicSmemBytes = sizeof(SampleShared);
      cudaLaunchAttribute at = {};
      at.id = cudaLaunchAttributeClusterDimension;
      at.val.clusterDim.x = 1u << i, at.val.clusterDim.y = at.val.clusterDim.z = 1;
      cfg.attrs = &at, cfg.numAttrs = 1;
      if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&held[i], kerns[i], &cfg);
    }
    return e;
  }();
  SD_CK(set);
  auto at_once = [&](int c) { return held[c == 1 ? 0 : c == 2 ? 1 : c == 4 ? 2 : 3]; };
  int C = 1;
  while (slice(C) > sp::kSlice) C *= 2;
  // few rows: more CTAs a row while each still has 4096 tokens and every row its cluster
  while (C < sp::kMaxCluster && rows <= at_once(2 * C) && vocab >= 4096 * 2 * C) C *= 2;
  const SampleArgs a = {logits, row_stride, rows, vocab, slice(C), s, u, tokens, logprob, kept};
  cudaStream_t st = (cudaStream_t)stream;
  // More rows than clusters at once, or a row of 16384 and not four CTAs for each: a CTA a row,
  // two an SM.  151936 tokens: 8 rows 20 us by clusters of 8, 34 a CTA each, 32 rows 22 (by
  // 4) and 34, 64 rows 41 and 34, 256 rows 142 and 51; 32000 tokens: 32 rows 17.4 (by 4)
  // and 16.5, 64 rows 18.7 (by 2) and 16.3, 128 rows 20.7 (by 1) and 16.5.
  const bool many = rows > at_once(C) || (C < 4 && vocab >= 4096 * 4);
  if (many) {
    k_sample_row<<<rows, sp::kRowThreads, sizeof(RowShared), st>>>(a);
    SD_CK(cudaGetLastError());
  }
  auto kern = C == 1 ? k_sample<1> : C == 2 ? k_sample<2> : C == 4 ? k_sample<4> : k_sample<8>;
  const int clusters = many ? std::min(rows, 32) : rows;
  SD_CK(launch_cluster(kern, dim3((unsigned)(clusters * C)), dim3(sp::kThreads), sizeof(SampleShared), st, many, C, a, many));
  return SD_OK;
}
