// Causal attention over packed prompts on the tensor cores (tcgen05 + TMEM).
//
//   o_i = sum_j exp(s_ij - lse_i) v_j,  s_ij = q_i . k_j scale over the keys j that row
//   i sees,
// in one pass over the keys with a row's reference and running sum.  The rows of a kv
// head's query heads are packed, token by token, into tiles of 128 (T = 128 / G tokens
// of G heads), so that K and V are read once for the group and a single token fills G
// rows.  A unit is a kv head and 2 T tokens (two tiles, WIDE) or up to T (one); its
// steps are 128 keys, the last ones first: a row meets its own and the nearest keys at
// once, which with slopes are the greatest scores.  Warps:
//  * 0..3 and 4..7: softmax, a thread a row: 128 scores from TMEM, their
//    exponentials, P (bf16) back over them; then the outputs.  A wide unit
//    gives each of the two groups a tile of rows, a narrow one alternate steps of the
//    same rows, joined through shared memory.  A row's weights are 2^(score - reference),
//    the reference kBias above the greatest score of the first half step in which the
//    row sees a key; it stays, and only where the weights would come to 1/2 in all is it
//    raised and O rescaled in TMEM (looking for the maximum in every step: 177 us for
//    166 on 8 prompts of up to 2048).  So O never passes the greatest value of the row's
//    keys, and fp32 holds it down to the bias.  P is bf16, as V is: a second term for what
//    the rounding leaves would make three products of two (568 us more for one prompt
//    of 16384 at the full rate); an output is off by 0.0019 to 0.0023 of its norm, where
//    its own rounding alone gives 0.0016.  One body of code serves both halves of a step
//    and all lengths (written out twice, 8 prompts took a fifth longer, the window with
//    caps a third).
//  * 8, 9: the products of one group each: S = Q K^T and O += P V, those of one group
//    while the other is in its softmax.  TMEM: [S 128][S 128][O D][O D].
//  * 10: walks the CTA's units, says what each is (PaDesc), and loads Q, K and V by TMA.
//  * 11: in steps where some row does not see some key, looks for infinities and NaNs
//    in V (P is 0 there, and 0 times those is not) and takes them out of the operand;
//    the rows that do see them get them back at the end.
// The steps are dealt evenly over the CTAs, by the host (it has the lengths): a
// unit may be split over its keys; its parts are joined by a second kernel.
//
// What bounds it: per group a round of scores (512 cycles of products at D = 128), the
// softmax of 128 scores a thread, and the second half's product, one after the other;
// two groups in turn make a step of two tiles in about 2600 cycles, of which 2048 are
// products.  A softmax warp's instructions count (a step's 64 weights take 540 cycles
// at 2.5 instructions each), not the exponential unit (ncu: 39%), and so does fetching
// them: all of the loop stays small.  Where scores have options and heads are 64, that
// chain waits for itself (issue 45%, tensor pipe 16%).  One GB300: 16384 rows, 32 query and
// 8 kv heads of 128: 1360 us, 1620 TFLOP/s (0.84 of the measured cuBLAS burst, 0.93 of
// its sustained rate); 8 prompts of up to 2048: 147 us; 512 rows over 33280 keys, 40
// heads: 272 us; 16 single tokens over 1.5 to 8k keys: 69 us, 5.0 TB/s; 5 prompts of up to
// 3001, 16 heads of 64, cap, slopes and window: 138 us.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <vector>

#include "gemm.cuh"
#include "kv4_attn.cuh"
#include "tcgen05.cuh"

namespace sdv {

namespace pa {
constexpr int kThreads = 384, kMma = 8, kLoad = 10;
constexpr int kKeys = 128;       // of a step
constexpr int kMaxCta = 160;
constexpr int kNK = 2, kNV = 2;  // stages of K and of V
constexpr int kNU = 4;           // units being described
constexpr float kMost = 0.5f;    // of a row's weights so far
// Of a reference over a score: a value of 2^-126 has 8 bits left (O is held in multiples
// of 2^-149).  8 prompts of up to 2048 take 151 us with 11, 148 with 13, 144 with 15 and
// 143 with 17; one of 16384 1473, 1377, 1347 and 1347.
constexpr float kBias = 15.f;
constexpr float kExact = 0x1p20f;  // offsets from references up to here are good to 2^-3
constexpr int kXs = 20;          // floats of a row being exchanged (16 used)
}  // namespace pa

// Where a CTA's share begins: step of the unit (request, kv head, token block).
struct PaAt {
  int r, h, i, step;
};

struct PaArgs {
  CUtensorMap qmap, kmap, vmap;
  PaAt at[pa::kMaxCta + 1];  // [grid + 1]: a share ends where the next begins
  Kv4Score s;
  const uint16_t* v;
  int64_t kv_stride;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int R, hq, hkv, G, T, U;   // T: tokens of a tile, U: of a unit (T or 2 T)
  uint16_t* out;
  float* lse;
  float* part;
  int32_t* status;
  uint32_t limit;  // of a wait, in ns
  uint32_t loads;  // steps' values that a CTA loads at most: all, but for sd_debug_prompt_wait
  // cap tanh(x scale / cap) log2(e) = x (k0 + k1 x^2 + ... + k4 x^8) while |x| <= series
  float k0, k1, k2, k3, k4, series;
};

// Joins of split units: [first CTA, parts].
struct PaJoins {
  PaAt at[pa::kMaxCta];  // step: parts
  int cta[pa::kMaxCta];
  int n;
};

template <int D>
struct PaShape {
  static constexpr int kTile = 128 * D * 2, kStep = pa::kKeys * D * 2;
  static constexpr int off_k = 2 * kTile, off_v = off_k + pa::kNK * kStep;
  static constexpr int off_x = kTile;  // [128][kXs] floats: narrow units leave Q's second tile free
  static constexpr int off_o = off_v + pa::kNV * kStep;            // [8 warps][32 rows][64 dims] bf16
  static constexpr int off_ml = off_o + 8 * 4096;
  static constexpr int off_bar = off_ml + 128 * 8;
  static constexpr int off_ctl = off_bar + 64 * 8;                 // PaCtl
  static constexpr int smem = off_ctl + 512;
  static constexpr int kPart = 256 * (D + 2);  // floats of a part: [row][D], then [row] (reference, sum)
};

// A unit, or a share of its steps, as the CTA's warps need it.  Steps are counted from
// the unit's first.
struct PaDesc {
  int n;               // steps of the share; 0: no row sees a key, -1: the end
  int wide, tc;        // two tiles; tokens
  int h, k0, hi;       // kv head; the request's first key; step u has the keys from 128 (hi - u) on
  int tok, p0;         // row of the first token, its position
  int ua;              // first step of the share
  int part;            // -1: the unit is whole; else the slot of its part
  int m0, m1;          // steps from m0 up to m1: every row sees every key
  int x[2], y[2];      // steps x, x + 1 (narrow: x + 2), ... below y are a group's
  int g0[2], g1[2];    // as m0, m1, for the rows of a group's tile
};
struct PaCtl {
  PaDesc unit[pa::kNU];
  int abort, turn;     // turn: 1 while a group's products are being issued
  int late;            // as abort, of what is waited for at the end
  uint32_t tmem;
  int bad[8];          // [unit with steps, mod 8]: infinities or NaNs were taken out of V
};
static_assert(sizeof(PaCtl) <= 512, "PaShape::smem");

// A unit's rows and steps.
struct PaUnit {
  int r, h, i;
  int m, n, q0, k0;    // rows and keys of the request, their first
  int nu;              // units a kv head
  int tok, tc;         // first token, tokens
  int p0;              // position of the first
  int hi, steps;       // number (key / 128) of step 0, which is the last; steps (0: no row sees a key)
  bool wide;
  __device__ __forceinline__ void request(const PaArgs& a) {
    q0 = a.cu_q[r], m = a.cu_q[r + 1] - q0;
    k0 = a.cu_k[r], n = a.cu_k[r + 1] - k0;
    nu = (m + a.U - 1) / a.U;
  }
  __device__ __forceinline__ void unit(const PaArgs& a) {
    tok = i * a.U;
    tc = min(a.U, m - tok);
    wide = tc > a.T;
    p0 = n - m + tok;
    const int p1 = p0 + tc - 1;
    hi = p1 < 0 ? 0 : p1 / pa::kKeys;
    steps = p1 < 0 ? 0 : hi + 1 - first(a, p0);
  }
  // the number of the first key that a row at position p sees, in steps
  static __device__ __forceinline__ int first(const PaArgs& a, int p) {
    return a.s.window > 0 && p >= 0 ? max(p - a.s.window + 1, 0) / pa::kKeys : 0;
  }
  // steps [x, y) in which rows of positions f .. l all see every key
  __device__ __forceinline__ void seen(const PaArgs& a, int f, int l, int& x, int& y) const {
    x = hi + 1 - (f >= 0 ? (int)(((int64_t)f + 1) / pa::kKeys) : 0);
    y = hi + 1 - (a.s.window > 0 && l >= 0 ? (int)(((int64_t)max(l - a.s.window + 1, 0) + pa::kKeys - 1) / pa::kKeys) : 0);
  }
  // steps [x, y) of those from ua to ub in which a tile of positions f .. l has keys
  __device__ __forceinline__ void range(const PaArgs& a, int f, int l, int ua, int ub, int& x, int& y) const {
    x = l < 0 ? ub : max(ua, hi - l / pa::kKeys);
    y = max(x, min(ub, hi + 1 - first(a, f)));
  }
};

// A CTA's walk over its units.
struct PaWalk : PaUnit {
  int ua, ub;
  PaAt end;
  bool fresh;
  __device__ __forceinline__ PaWalk(const PaArgs& a) {
    const PaAt b = a.at[blockIdx.x];
    end = a.at[blockIdx.x + 1];
    r = b.r, h = b.h, i = b.i, ua = b.step;
    fresh = true;
  }
  __device__ __forceinline__ bool next(const PaArgs& a) {
    if (!fresh) {
      ua = 0;
      if (++i == nu) {
        i = 0;
        if (++h == a.hkv) {
          h = 0;
          do r++;
          while (r < end.r && a.cu_q[r + 1] == a.cu_q[r]);
        }
      }
    }
    if (r > end.r || (r == end.r && (h > end.h || (h == end.h && (i > end.i || (i == end.i && ua >= end.step)))))) return false;
    if (r >= a.R) return false;
    if (fresh || i == 0) request(a);
    fresh = false;
    unit(a);
    ub = r == end.r && h == end.h && i == end.i ? end.step : max(1, steps);
    return true;
  }
  __device__ __forceinline__ void describe(const PaArgs& a, PaDesc& d) const {
    d.n = steps ? ub - ua : 0;
    d.wide = wide, d.tc = tc;
    d.h = h, d.k0 = k0, d.hi = hi;
    d.tok = q0 + tok, d.p0 = p0, d.ua = ua;
    d.part = ua == 0 && ub == max(1, steps) ? -1 : 2 * (int)blockIdx.x + (ua == 0);
    seen(a, p0, p0 + tc - 1, d.m0, d.m1);
    for (int t = 0; t < 2; t++) {
      const int f = p0 + (wide ? t * a.T : 0), l = p0 + (wide && t == 0 ? a.T : tc) - 1;
      seen(a, f, l, d.g0[t], d.g1[t]);
      if (wide) {
        range(a, f, l, ua, ub, d.x[t], d.y[t]);
      } else {
        d.x[t] = ua + t;
        d.y[t] = ub;
      }
    }
  }
};

// 64 consecutive 32-bit columns of this thread's TMEM lane: asked for, and waited for
// (the registers are tied to the wait, so that no use moves above it).
__device__ __forceinline__ void pa_tmem_ld(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void pa_wait_ld(uint32_t (&r)[64]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]), "+r"(r[32]), "+r"(r[33]), "+r"(r[34]), "+r"(r[35]), "+r"(r[36]), "+r"(r[37]), "+r"(r[38]), "+r"(r[39]), "+r"(r[40]), "+r"(r[41]), "+r"(r[42]), "+r"(r[43]), "+r"(r[44]), "+r"(r[45]), "+r"(r[46]), "+r"(r[47]), "+r"(r[48]), "+r"(r[49]), "+r"(r[50]), "+r"(r[51]), "+r"(r[52]), "+r"(r[53]), "+r"(r[54]), "+r"(r[55]), "+r"(r[56]), "+r"(r[57]), "+r"(r[58]), "+r"(r[59]), "+r"(r[60]), "+r"(r[61]), "+r"(r[62]), "+r"(r[63])
               :
               : "memory");
}
__device__ __forceinline__ float pa_max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
template <int N>
__device__ __forceinline__ void pa_tmem_st(uint32_t taddr, const uint32_t (&r)[N]);
template <>
__device__ __forceinline__ void pa_tmem_st(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
               "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
               : "memory");
}
__device__ __forceinline__ uint32_t pa_bf16x2(float lo, float hi) {
  uint32_t y;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
  return y;
}
__device__ __forceinline__ void pa_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// D (tmem) (+)= A (tmem) * B (smem).
__device__ __forceinline__ void pa_umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma3d_g2s(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// B operand with its N side (dims) contiguous, 128-byte swizzle: rows of 64 dims, 8
// keys 1024 bytes, panels of 64 dims 16384 bytes apart.
__device__ __forceinline__ uint64_t pa_sdesc_v(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(16384 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ uint32_t pa_clock() {  // ns, mod 2^32
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}

// A bounded wait in few instructions (all of the kernel's code has to stay in the
// instruction cache): past the limit it sets *abort, which ends every wait.  What a warp
// does after a wait that gave up stays within its buffers and its unit's rows: it goes by
// a PaDesc that was written, and no other is written from then on.
__device__ __forceinline__ void pa_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t limit) {
  if (mbar_try_wait(bar, parity)) return;
  const uint32_t t0 = pa_clock();
#pragma unroll 1
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); i++) {
    if (i % 64) continue;  // a try suspends the warp for a while by itself
    if (*abort) return;
    if (pa_clock() - t0 > limit) *abort = 1;
  }
}

// What a softmax thread keeps of its row over a unit.
struct PaRow {
  float ref, l;  // reference (base 2), sum of 2^(score - ref)
  bool done;     // the group had steps
  bool live;     // the lane has a row
};

// What a call's scores have: nothing, slopes, a cap (and slopes or none).
constexpr int kPlain = 0, kSlopes = 1, kCapped = 2;

// 64 scores of a row, from key c0 of a step on: scale, cap and slope in base 2 (none:
// q.k), and -inf for the keys that it does not see (kb: the first one's number; see0 ..
// see1: the keys it sees).
template <int MODE>
__device__ __forceinline__ void pa_scores(const PaArgs& a, float (&x)[64], int kb, int see0, int see1, bool masked,
                                          float slope) {
  if (MODE == kCapped) {
    // tanh's Taylor series to x^9 where every score of the warp is below 0.3 of the cap
    // (off by 1.6e-8 there), six multiply-adds a score: they are what bounds capped calls
#pragma unroll
    for (int d = 0; d < 64; d += 32) {
      float top = 0.f;
#pragma unroll
      for (int c = d; c < d + 32; c += 2) top = pa_max3(top, fabsf(x[c]), fabsf(x[c + 1]));
      if (__any_sync(0xffffffffu, !(top <= a.series))) {
        kv4_cap(a.s, reinterpret_cast<float (&)[32]>(x[d]));
        continue;
      }
#pragma unroll
      for (int c = d; c < d + 32; c += 2) {
        const uint64_t z = f2pack(x[c], x[c + 1]), u = f2mul(z, z);
        uint64_t q = f2fma(u, f2pack(a.k4, a.k4), f2pack(a.k3, a.k3));
        q = f2fma(q, u, f2pack(a.k2, a.k2));
        q = f2fma(q, u, f2pack(a.k1, a.k1));
        q = f2fma(q, u, f2pack(a.k0, a.k0));
        f2unpack(f2mul(q, z), x[c], x[c + 1]);
      }
    }
  }
  if (MODE == kSlopes) {  // the scale ahead of the slope: one over the other may pass fp32
    const float f = a.s.scale * kLog2e;
#pragma unroll
    for (int c = 0; c < 64; c += 2) f2unpack(f2mul(f2pack(x[c], x[c + 1]), f2pack(f, f)), x[c], x[c + 1]);
  }
  if (MODE == kSlopes || (MODE == kCapped && a.s.slopes)) {
#pragma unroll
    for (int c = 0; c < 64; c++) x[c] = fmaf(slope, (float)c, x[c]);
  }
  if (masked) {
    // sixteens of which every row of the warp sees all are passed over
    const int a0 = see0 - kb, a1 = see1 - kb;
    const int w0 = __reduce_max_sync(0xffffffffu, a0), w1 = __reduce_min_sync(0xffffffffu, a1);
#pragma unroll
    for (int d = 0; d < 64; d += 16) {
      if (w0 <= d && w1 >= d + 15) continue;
#pragma unroll
      for (int c = d; c < d + 16; c++)
        if (c < a0 || c > a1) x[c] = -INFINITY;
    }
  }
}
__device__ __forceinline__ float pa_max(const float (&x)[64]) {
  float t4[4];
#pragma unroll
  for (int e = 0; e < 4; e++) t4[e] = pa_max3(x[e], x[e + 4], x[e + 8]);
#pragma unroll
  for (int c = 12; c < 60; c += 8) {
#pragma unroll
    for (int e = 0; e < 4; e++) t4[e] = pa_max3(t4[e], x[c + e], x[c + 4 + e]);
  }
  return fmaxf(pa_max3(t4[0], x[60], x[61]), fmaxf(pa_max3(t4[1], x[62], x[63]), fmaxf(t4[2], t4[3])));
}
// 64 weights 2^(x f + off) of a row as bf16 pairs into TMEM; their sum.
__device__ __forceinline__ float pa_weights(const float (&x)[64], float f, float off, uint32_t taddr) {
  const uint64_t ff = f2pack(f, f), oo = f2pack(off, off);
  uint64_t l2[2] = {0, 0};
#pragma unroll
  for (int c0 = 0; c0 < 64; c0 += 32) {
    uint32_t p[16];
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      float p0, p1;
      f2unpack(f2fma(f2pack(x[c0 + c], x[c0 + c + 1]), ff, oo), p0, p1);
      p0 = ex2(p0);
      p1 = ex2(p1);
      l2[c >> 1 & 1] = f2add(l2[c >> 1 & 1], f2pack(p0, p1));
      p[c / 2] = pa_bf16x2(p0, p1);
    }
    pa_tmem_st(taddr + c0 / 2, p);
  }
  float l0, l1;
  f2unpack(f2add(l2[0], l2[1]), l0, l1);
  return l0 + l1;
}

// The reference raised to `top` where that is greater, O (where it holds anything) and
// the sum with it.
template <int D>
__device__ __forceinline__ void pa_grow(PaRow& w, uint32_t to, float top, bool held) {
  const bool grows = top > w.ref;
  const float al = grows ? ex2(w.ref - top) : 1.f;
  if (grows) w.ref = top;
  w.l *= al;
  if (held) {
#pragma unroll 1
    for (int c = 0; c < D; c += 16) {
      float o[16];
      tmem_ld16(to + c, o);
      uint32_t y[16];
#pragma unroll
      for (int k = 0; k < 16; k++) y[k] = __float_as_uint(o[k] * al);
      pa_tmem_st(to + c, y);
    }
  }
}

// One step: scores from TMEM, P back in two halves, said by half(0) and half(1).  kb:
// first key; see0 .. see1: the keys that the row sees; masked: some row of the tile
// does not see some key; scores are f x + slope2 c + base, c a key's number in the
// step; first(): waits for the product of the first half.  O is at
// rest until half(0): its last product's commit came before these scores'.
template <int D, int MODE, typename Half, typename First>
__device__ __forceinline__ void pa_step(const PaArgs& a, PaRow& w, uint32_t ts, uint32_t to, int kb, int see0, int see1,
                                        bool masked, float f, float slope2, float base, Half half, First first) {
  auto far = [&](float l) { return w.live && !(w.l + l < pa::kMost) && w.l == w.l; };  // too much, or the first NaN
#pragma unroll 1
  for (int h = 0; h < 2; h++, base += 64.f * slope2) {
    uint32_t r[64];
    float (&x)[64] = reinterpret_cast<float (&)[64]>(r);
    pa_tmem_ld(ts + 64 * h, r);
    pa_wait_ld(r);
    if (MODE != kPlain || masked) pa_scores<MODE>(a, x, kb + 64 * h, see0, see1, masked, slope2);
    // A row's reference goes by the greatest score of the first keys that it sees (nothing
    // is held of it before).  Where it, or base, passes 2^20 its last place shows in the
    // exponent, and a weight could be anything: such scores are rounded first, so that
    // the greatest weighs 2^-kBias, or 1 where the bias is less than a last place.
    auto large = [&]() { return !(fmaxf(fabsf(w.ref), fabsf(base)) <= pa::kExact); };  // or no reference yet
    float l = 0.f, fx = f, bx = base;  // a score is fx x + bx
    auto reference = [&]() { w.ref = fmaxf(fmaf(pa_max(x), fx, bx), -INFINITY) + pa::kBias; };  // no NaN
    auto round = [&]() {
#pragma unroll
      for (int c = 0; c < 64; c++) x[c] = fmaf(x[c], fx, bx);
      fx = 1.f, bx = 0.f;
    };
    auto weights = [&]() { l = pa_weights(x, fx, w.ref == -INFINITY ? 0.f : bx - w.ref, ts + 32 * h); };
    auto raise = [&]() {
      if (h == 1) first();
      // by the greatest score, and by what has come together (of any row within 2^4 of the
      // limit, so that a warp seldom comes here)
      const float top = fmaf(pa_max(x), fx, bx) + pa::kBias;
      pa_grow<D>(w, to, w.l + l >= pa::kMost / 16 ? fmaxf(top, w.ref + 10.f) : top, h == 1 || w.done);
      if (!(l == l)) w.l = l;
    };
    // At most two passes: the second is under a reference that holds the weights.  Without
    // options the usual pass has a body of its own (one prompt of 16384: 1345 us, 1430
    // without); with them the instructions fetched count more (5 ragged prompts with cap,
    // slopes and a window: 164 us with it, 138 without).
    if (MODE == kPlain) {
      bool done = false;
      if (!__any_sync(0xffffffffu, w.live && large())) {
        l = pa_weights(x, f, base - w.ref, ts + 32 * h);
        done = !__any_sync(0xffffffffu, far(l));
      } else if (w.ref == -INFINITY) {
        reference();
      }
      if (__builtin_expect(!done, 0)) {
        bool rounded = false;
#pragma unroll 1
        for (int again = 0;; again++) {
          if (!rounded && large()) round(), rounded = true;
          weights();
          if (again == 1 || !__any_sync(0xffffffffu, far(l))) break;
          raise();
        }
      }
    } else {
#pragma unroll 1
      for (int again = 0;; again++) {
        if (__any_sync(0xffffffffu, w.live && large())) {
          if (w.ref == -INFINITY) reference();
          if (large()) round();  // what is rounded stays as it is
        }
        weights();
        if (again == 1 || !__any_sync(0xffffffffu, far(l))) break;
        raise();
      }
    }
    w.l += l;
    pa_wait_st();
    half(h);
  }
  w.done = true;
}

template <int D, int MODE>
__global__ void __launch_bounds__(pa::kThreads, 1) k_prompt_attn(const __grid_constant__ PaArgs a) {
  using S = PaShape<D>;
  extern __shared__ __align__(1024) uint8_t sm[];  // the only shared memory, so that it begins on a swizzle's boundary
  if (smem_u32(sm) & 1023) {
    set_status(a.status, SD_ERR_CUDA);
    return;
  }
  uint64_t* const u_full = reinterpret_cast<uint64_t*>(sm + S::off_bar);  // [kNU] unit described
  uint64_t* const u_empty = u_full + pa::kNU;      // [kNU] unit done (8 softmax warps, 2 products', 1 looking at V)
  uint64_t* const q_full = u_empty + pa::kNU;
  uint64_t* const q_empty = q_full + 1;            // products with Q done (2 commits), exchange done (8 warps)
  uint64_t* const k_full = q_empty + 1;            // [kNK]
  uint64_t* const k_empty = k_full + pa::kNK;      // [kNK] products done (2)
  uint64_t* const v_full = k_empty + pa::kNK;      // [kNV]
  uint64_t* const v_empty = v_full + pa::kNV;      // [kNV] products done (2), looked at
  uint64_t* const v_ok = v_empty + pa::kNV;        // [kNV] looked at
  uint64_t* const s_full = v_ok + pa::kNV;         // [t] scores ready, the products before them done (commit)
  uint64_t* const p_full = s_full + 2;             // [t][half] weights written (4 warps)
  uint64_t* const h_full = p_full + 4;             // [t] the product of P's first half done (commit)
  uint64_t* const o_full = h_full + 2;             // [t] a unit's last product done (commit)
  uint64_t* const o_empty = o_full + 2;            // [t] outputs read (4 warps)
  uint64_t* const x_full = o_empty + 2;            // groups that share rows meet (8 warps)
  uint64_t* const t_done = x_full + 1;             // [t] all of a group's products done (commit)
  PaCtl& ctl = *reinterpret_cast<PaCtl*>(sm + S::off_ctl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch();

  if (warp == pa::kMma) {
    tmem_alloc(&ctl.tmem, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < pa::kNU; i++) mbar_init(&u_full[i], 1), mbar_init(&u_empty[i], 11);
    mbar_init(q_full, 1), mbar_init(q_empty, 10);
    for (int i = 0; i < pa::kNK; i++) mbar_init(&k_full[i], 1), mbar_init(&k_empty[i], 2);
    for (int i = 0; i < pa::kNV; i++) mbar_init(&v_full[i], 1), mbar_init(&v_empty[i], 3), mbar_init(&v_ok[i], 1);
    for (int t = 0; t < 2; t++) {
      mbar_init(&s_full[t], 1), mbar_init(&h_full[t], 1), mbar_init(&o_full[t], 1), mbar_init(&o_empty[t], 4);
      mbar_init(&p_full[2 * t], 4), mbar_init(&p_full[2 * t + 1], 4);
    }
    mbar_init(x_full, 8), mbar_init(&t_done[0], 1), mbar_init(&t_done[1], 1);
    ctl.abort = ctl.turn = ctl.late = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = ctl.tmem;
  auto wait = [&](uint64_t* bar, uint32_t parity) { pa_wait(smem_u32(bar), parity & 1, &ctl.abort, a.limit); };
  auto aborted = [&]() { return *(volatile int*)&ctl.abort != 0; };
  // One group's products at a time: those of both, interleaved, would end together,
  // and the softmax of both would run together, with the tensor cores idle.
  auto turn = [&]() {
    const uint32_t t0 = pa_clock();
#pragma unroll 1
    while (atomicCAS(&ctl.turn, 0, 1) != 0) {
      if (aborted()) return;
      if (pa_clock() - t0 > a.limit) *(volatile int*)&ctl.abort = 1;
    }
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(72));
    if (warp == pa::kLoad) {
      if (elect_one()) {
        PaWalk w(a);
        uint32_t nk = 0, nv = 0, nq = 0;
        bool on = true;
        // after a wait that gave up nothing more is described or loaded: a stage's next copy
        // would begin while the one before it may be under way
        auto free = [&](uint64_t* bar, uint32_t parity) {
          wait(bar, parity);
          return on = !aborted();
        };
#pragma unroll 1
        for (uint32_t i = 0; on; i++) {
          const bool more = w.next(a);
          PaDesc& d = ctl.unit[i % pa::kNU];
          if (!free(&u_empty[i % pa::kNU], (i / pa::kNU & 1) ^ 1)) break;
          if (more) w.describe(a, d);
          else d.n = -1;
          mbar_arrive(&u_full[i % pa::kNU]);
          if (!more) break;
          if (w.steps == 0) continue;  // no row sees a key: the softmax warps write the rows
          const int n = w.ub - w.ua, key0 = w.k0 + (w.hi - w.ua) * pa::kKeys;
          auto load_k = [&](int u) {
            const uint32_t st = nk % pa::kNK;
            if (!free(&k_empty[st], (nk / pa::kNK & 1) ^ 1)) return;
            mbar_arrive_expect_tx(&k_full[st], S::kStep);
#pragma unroll
            for (int c = 0; c < D; c += 64)
              tma3d_g2s(sm + S::off_k + st * S::kStep + c * 256, &a.kmap, c, w.h, key0 - u * pa::kKeys, &k_full[st]);
            nk++;
          };
          load_k(0);
          if (!on || !free(q_empty, (nq & 1) ^ 1)) break;
          const int tiles = w.wide ? 2 : 1;
          mbar_arrive_expect_tx(q_full, tiles * (D / 64) * 128 * a.G * a.T);
          for (int t = 0; t < tiles; t++)
            for (int c = 0; c < D; c += 64)
              tma3d_g2s(sm + t * S::kTile + c * 256, &a.qmap, c, w.h * a.G, w.q0 + w.tok + t * a.T, q_full);
          nq++;
#pragma unroll 1
          for (int u = 0; u < n && on; u++) {
            if (u + 1 < n) load_k(u + 1);
            const uint32_t st = nv % pa::kNV;
            on = on && nv < a.loads;
            if (!on || !free(&v_empty[st], (nv / pa::kNV & 1) ^ 1)) break;
            mbar_arrive_expect_tx(&v_full[st], S::kStep);
#pragma unroll
            for (int c = 0; c < D; c += 64)
              tma3d_g2s(sm + S::off_v + st * S::kStep + c * 256, &a.vmap, c, w.h, key0 - u * pa::kKeys, &v_full[st]);
            nv++;
          }
        }
        // the CTA ends with no copy and no product under way, whatever its warps did: the
        // last phases of K's and V's stages and of Q, and both groups' commits
        static_assert(pa::kNK == 2 && pa::kNV == 2, "two stages each");
#pragma unroll 1
        for (uint32_t e = 0; e < 7; e++) {
          uint64_t* const bar = e < 2 ? &k_full[e] : e < 4 ? &v_full[e - 2] : e == 4 ? q_full : &t_done[e - 5];
          const uint32_t n = e < 2 ? nk + 1 - e : e < 4 ? nv + 3 - e : e == 4 ? 2 * nq : 2;  // twice the phases begun
          if (n > 1) pa_wait(smem_u32(bar), (n / 2 - 1) & 1, &ctl.late, (uint32_t)kWaitLimitNs);
        }
      }
      __syncwarp();
    } else if (warp < pa::kLoad) {
      if (elect_one()) {  // one lane throughout
        const int t = warp - pa::kMma;
        const uint32_t id0 = (1u << 4) | (1u << 7) | (1u << 10) | (8u << 24);  // fp32 += bf16 bf16, M = 128
        const uint32_t ids = id0 | ((uint32_t)(pa::kKeys / 8) << 17), idv = id0 | (1u << 16) | ((uint32_t)(D / 8) << 17);
        const uint64_t kd = sdesc_sw128(smem_u32(sm + S::off_k)), vd = pa_sdesc_v(smem_u32(sm + S::off_v));
        const uint32_t ts = tm + t * 128, to = tm + 256 + t * 128;
        uint32_t nk = 0, nv = 0, units = 0, pp = 0, po = 1;  // stages taken, units; parities of p_full and o_empty
#pragma unroll 1
        for (uint32_t i = 0;; i++) {
          const PaDesc& d = ctl.unit[i % pa::kNU];
          wait(&u_full[i % pa::kNU], i / pa::kNU);
          const int n = d.n;
          if (aborted()) break;
          if (n <= 0) {
            if (n < 0) break;
            mbar_arrive(&u_empty[i % pa::kNU]);
            continue;
          }
          // the group's steps: x, x + by, ... below y
          const int by = d.wide ? 1 : 2, x = d.x[t] - d.ua, y = d.y[t] - d.ua, m0 = d.m0 - d.ua, m1 = d.m1 - d.ua;
          const uint64_t qd = sdesc_sw128(smem_u32(sm + (d.wide ? t : 0) * S::kTile));
          // A wide unit's stages are released by both groups, those that one of them has no use
          // for too; a narrow unit's by the one group that uses them, in the other's name as
          // well.  A wait for a phase is one only while the phase before it is known to be
          // over, and may not come two phases late: no group may lose sight of a stage.  A
          // narrow unit of several steps keeps both in sight: its Q is released after its
          // outputs, so the next unit's is not there before all of its stages were used.  One
          // of a single step releases Q once K is used, ahead of its V: the group without a
          // step waits for that V, and releases it, itself.
          const bool both = by == 1 || n == 1;  // V is released by both groups
          int k = 0, v = 0;  // steps whose K (wide units') and V (both groups') are taken
          auto pass_k = [&](int u) {
#pragma unroll 1
            for (; by == 1 && k < u; k++) {
              wait(&k_full[(nk + k) % pa::kNK], (nk + k) / pa::kNK);
              mbar_arrive(&k_empty[(nk + k) % pa::kNK]);
            }
          };
          auto pass_v = [&](int u) {
#pragma unroll 1
            for (; both && v < u; v++) {
              wait(&v_full[(nv + v) % pa::kNV], (nv + v) / pa::kNV);
              mbar_arrive(&v_empty[(nv + v) % pa::kNV]);
            }
          };
          auto scores = [&](int u) {  // of step u, whose K is there
            const uint32_t st = (nk + u) % pa::kNK;
            const uint64_t kk = kd + st * (S::kStep >> 4);
#pragma unroll
            for (int c = 0; c < D / 16; c++)
              umma_bf16(ts, qd + (c >> 2) * (16384 >> 4) + (c & 3) * 2, kk + (c >> 2) * (16384 >> 4) + (c & 3) * 2, ids, c > 0);
            umma_commit(&s_full[t]);
            umma_commit(&k_empty[st]);
            if (by == 2) mbar_arrive(&k_empty[st]);
            if (u + by >= y) umma_commit(q_empty);
            k++;
          };
          wait(q_full, units);
          // Step u's values after its P, and the scores of the next; u = x - by begins.
#pragma unroll 1
          for (int u = x - by; u < y; u += by) {
            if (x >= y || aborted()) break;
            const bool more = u + by < y;
            // K and V are waited for ahead of P, while the softmax runs: between P and the
            // next scores there is nothing but the products
            if (more) {
              pass_k(u + by);
              wait(&k_full[(nk + u + by) % pa::kNK], (nk + u + by) / pa::kNK);
            }
            const uint32_t vs = (nv + u) % pa::kNV;
            if (u >= x) {
              pass_v(u);
              wait(&v_full[vs], (nv + u) / pa::kNV);
              if (u < m0 || u >= m1) wait(&v_ok[vs], (nv + u) / pa::kNV);
              if (u == x) {
                wait(&o_empty[t], po);
                po ^= 1;
              }
              const uint64_t vv = vd + vs * (S::kStep >> 4);
#pragma unroll
              for (int h = 0; h < 2; h++) {
                wait(&p_full[2 * t + h], pp);
                if (h == 0) turn();
                tc_fence_after();
#pragma unroll
                for (int c = 4 * h; c < 4 * h + 4; c++)
                  pa_umma_ts(to, ts + 8 * c, vv + c * (2048 >> 4), idv, u > x || c > 0);
                if (h == 0) umma_commit(&h_full[t]);
              }
              pp ^= 1;
            } else {
              turn();
              tc_fence_after();
            }
            if (more) scores(u + by);
            else umma_commit(&o_full[t]);
            if (u >= x) {
              umma_commit(&v_empty[vs]);
              if (!both) mbar_arrive(&v_empty[vs]);
              v++;
            }
            atomicExch(&ctl.turn, 0);
          }
          if (x >= y) mbar_arrive(q_empty);
          pass_k(n);
          pass_v(n);
          mbar_arrive(&u_empty[i % pa::kNU]);
          nk += n, nv += n;
          units++;
        }
        umma_commit(&t_done[t]);
      }
      __syncwarp();
    } else {
      // ----------------------------------------------- looking at values --
      uint32_t nv = 0, units = 0;
#pragma unroll 1
      for (uint32_t i = 0;; i++) {
        const PaDesc& d = ctl.unit[i % pa::kNU];
        wait(&u_full[i % pa::kNU], i / pa::kNU);
        const int n = d.n, m0 = d.m0 - d.ua, m1 = d.m1 - d.ua;
        if (__any_sync(0xffffffffu, aborted() || n < 0)) break;
        if (n > 0) {
          if (lane == 0) ctl.bad[units & 7] = 0;
#pragma unroll 1
          for (int u = 0; u < n; u++, nv++) {
            const uint32_t st = nv % pa::kNV;
            wait(&v_full[st], nv / pa::kNV);
            if (u < m0 || u >= m1) {
              uint4* const v = reinterpret_cast<uint4*>(sm + S::off_v + st * S::kStep);
              uint32_t odd = 0;  // bit 15 of a half word: its exponent is all ones
#pragma unroll 8
              for (int e = lane; e < S::kStep / 16; e += 32) {
                const uint4 z = v[e];
                odd |= ((z.x & 0x7F807F80u) + 0x00800080u) | ((z.y & 0x7F807F80u) + 0x00800080u) |
                       ((z.z & 0x7F807F80u) + 0x00800080u) | ((z.w & 0x7F807F80u) + 0x00800080u);
              }
              if (__any_sync(0xffffffffu, odd & 0x80008000u)) {
                if (lane == 0) ctl.bad[units & 7] = 1;
                uint32_t* const vw = reinterpret_cast<uint32_t*>(v);
#pragma unroll 1
                for (int e = lane; e < S::kStep / 4; e += 32) {
                  const uint32_t z = vw[e], o = ((z & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
                  if (o) vw[e] = z & ~((o >> 15) * 0xFFFFu);
                }
              }
              fence_async_smem();
            }
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&v_ok[st]);
              mbar_arrive(&v_empty[st]);
            }
          }
          units++;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&u_empty[i % pa::kNU]);
      }
    }
  } else {
    // ---------------------------------------------------------- softmax --
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(216));
    const int t = warp >> 2, idx = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t ts = tm + t * 128 + lanes, to = tm + 256 + t * 128 + lanes;
    const float f = MODE == kPlain ? a.s.scale * kLog2e : 1.f;  // base 2 from q.k, or from what pa_scores gives
    const int tok_of = idx / a.G;
    uint32_t some = 0, sp = 0, hp = 0, op = 0, xp = 0;  // units with steps; parities of s_full, h_full, o_full and x_full
    // not a named barrier: after a wait that gave up the warps may differ in their units
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(x_full);
      while (!mbar_try_wait(smem_u32(x_full), xp) && !aborted()) {
      }
      xp ^= 1;
    };
#pragma unroll 1
    for (uint32_t i = 0;; i++) {
      const PaDesc& d = ctl.unit[i % pa::kNU];
      wait(&u_full[i % pa::kNU], i / pa::kNU);
      const int n = d.n;
      if (__any_sync(0xffffffffu, aborted() || n < 0)) break;
      // the row's token in the unit; rows past the last token follow it, and are not written
      const int tok = min((d.wide ? t * a.T : 0) + tok_of, d.tc - 1);
      const int p = d.p0 + tok;
      const int see0 = a.s.window > 0 && p >= 0 ? max(p - a.s.window + 1, 0) : 0;
      const bool pair = !d.wide && n > 1;              // the groups share the rows
      const bool live = (d.wide ? t * a.T : 0) + tok_of < d.tc && tok_of < a.T;
      PaRow row = {-INFINITY, 0.f, false, live};
      if (n > 0) {
        wait(q_full, some);  // no group is a unit ahead of the others' barriers
        if (!pair && lane == 0) mbar_arrive(q_empty);  // nothing to exchange
        const float slope2 = MODE != kPlain && a.s.slopes ? a.s.slopes[d.h * a.G + idx % a.G] * kLog2e : 0.f;
        const int by = d.wide ? 1 : 2, y = d.y[t], g0 = d.g0[t], g1 = d.g1[t];
        int kb = (d.hi - d.x[t]) * pa::kKeys;
#pragma unroll 1
        for (int u = d.x[t]; u < y; u += by, kb -= by * pa::kKeys) {
          wait(&s_full[t], sp);
          sp ^= 1;
          tc_fence_after();
          pa_step<D, MODE>(a, row, ts, to, kb, see0, p, u < g0 || u >= g1, f, slope2, MODE != kPlain ? slope2 * (float)(kb - p) : 0.f, [&](int h) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[2 * t + h]);
          }, [&]() {
            wait(&h_full[t], hp);
            tc_fence_after();
          });
          hp ^= 1;
        }
      }
      // while the last product runs: sums and factors
      const bool whole = d.part < 0;
      const int64_t at = (int64_t)(d.tok + tok) * a.hq + d.h * a.G + idx % a.G;  // the row of out
      float* const part = a.part + (int64_t)d.part * S::kPart;
      // (reference, sum) of the row and the outputs' factors
      float M = row.ref, L = row.l, mine = 1.f, other = 0.f;
      if (pair) {
        float2* const s_ml = reinterpret_cast<float2*>(sm + S::off_ml);
        if (t == 1) s_ml[idx] = make_float2(row.ref, row.l);
        meet();
        if (t == 0) {
          const float2 ml = s_ml[idx];
          M = fmaxf(row.ref, ml.x);
          const float Ms = M == -INFINITY ? 0.f : M;
          mine = row.done ? ex2(row.ref - Ms) : 0.f;
          other = ml.x == -INFINITY ? 0.f : ex2(ml.x - Ms);
          L = mine * row.l + other * ml.y;
          if (!(ml.y == ml.y)) L = ml.y, other = ml.y;  // a NaN among the other's scores
        }
      }
      const bool writes = d.wide || t == 0;  // a narrow unit's rows are the first group's to write
      const float inv = L == 0.f ? 0.f : 1.f / L;
      if (writes && live) {
        if (whole) {
          if (a.lse) a.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * (1.f / kLog2e);
        } else {
          __stcg(reinterpret_cast<float2*>(part + 256 * D) + t * 128 + idx, make_float2(M, L));
        }
      }
      // What a row's 64 dims from c on come to goes out through shared memory (pieces of
      // 16 bytes, their order turned by the row), so that eight lanes write a row's 128
      // bytes: a lane a row took 4000 cycles a unit.
      uint4* const so = reinterpret_cast<uint4*>(sm + S::off_o + warp * 4096);
      auto put = [&](int piece, const float* o) {
        so[lane * 8 + (piece ^ (lane & 7))] = make_uint4(pa_bf16x2(o[0] * inv, o[1] * inv), pa_bf16x2(o[2] * inv, o[3] * inv),
                                                         pa_bf16x2(o[4] * inv, o[5] * inv), pa_bf16x2(o[6] * inv, o[7] * inv));
      };
      auto write = [&](int c) {
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const int r = e * 4 + (lane >> 3), to_row = __shfl_sync(0xffffffffu, live ? (int)at : -1, r);
          if (to_row >= 0)
            *reinterpret_cast<uint4*>(a.out + (int64_t)to_row * D + c + (lane & 7) * 8) = so[r * 8 + ((lane & 7) ^ (r & 7))];
        }
        __syncwarp();
      };
      const bool some_sum = row.done && row.l != 0.f;
      bool bad = false;
      if (row.done) {
        wait(&o_full[t], op);
        op ^= 1;
        tc_fence_after();
        bad = *(volatile int*)&ctl.bad[some & 7];
      }
      if (whole && !pair && row.done && !bad) {
#pragma unroll 1
        for (int c = 0; c < D; c += 64) {
          uint32_t r[64];
          pa_tmem_ld(to + c, r);
          pa_wait_ld(r);
          float (&o)[64] = reinterpret_cast<float (&)[64]>(r);
          if (!some_sum) {
#pragma unroll
            for (int e = 0; e < 64; e++) o[e] = 0.f;
          }
#pragma unroll
          for (int e = 0; e < 8; e++) put(e, o + 8 * e);
          write(c);
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float o[16];
          if (row.done) tmem_ld16(to + c, o);
#pragma unroll
          for (int e = 0; e < 16; e++) o[e] = some_sum ? o[e] : 0.f;
          if (bad && live) {
            // infinities and NaNs that were taken out of V and that the row sees
#pragma unroll 1
            for (int u = d.x[t]; u < d.y[t]; u += d.wide ? 1 : 2) {
              if (u >= d.m0 && u < d.m1) continue;
              const int kb = (d.hi - u) * pa::kKeys;
#pragma unroll 1
              for (int key = max(kb, see0); key <= min(kb + pa::kKeys - 1, p); key++) {
                const uint16_t* v = a.v + (int64_t)(d.k0 + key) * a.kv_stride + d.h * D + c;
#pragma unroll
                for (int e = 0; e < 16; e++)
                  if ((v[e] & 0x7F80) == 0x7F80) o[e] += bf2f(v[e]);
              }
            }
          }
          if (pair) {
            float4* const xr = reinterpret_cast<float4*>(sm + S::off_x) + idx * (pa::kXs / 4);
            if (t == 1) {
#pragma unroll
              for (int e = 0; e < 4; e++) xr[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
            meet();
            if (t == 0) {
#pragma unroll
              for (int e = 0; e < 4; e++) {
                const float4 v = xr[e];
                o[4 * e] = fmaf(other, v.x, mine * o[4 * e]);
                o[4 * e + 1] = fmaf(other, v.y, mine * o[4 * e + 1]);
                o[4 * e + 2] = fmaf(other, v.z, mine * o[4 * e + 2]);
                o[4 * e + 3] = fmaf(other, v.w, mine * o[4 * e + 3]);
              }
            }
            meet();
          }
          if (!writes) continue;
          if (whole) {
            put(c / 8 & 7, o);
            put((c / 8 & 7) + 1, o + 8);
            if (c % 64 == 48) write(c - 48);
          } else if (live) {
            float4* const dst = reinterpret_cast<float4*>(part + (int64_t)(t * 128 + idx) * D + c);
#pragma unroll
            for (int e = 0; e < 4; e++) __stcg(dst + e, make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
          }
        }
      }
      tc_fence_before();
      if (pair) fence_async_smem();  // Q's second tile may be loaded where the exchange was
      __syncwarp();
      if (lane == 0) {
        if (row.done) mbar_arrive(&o_empty[t]);
        if (pair) mbar_arrive(q_empty);
        mbar_arrive(&u_empty[i % pa::kNU]);
      }
      some += n > 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == pa::kMma) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
    if ((ctl.abort | ctl.late) && lane == 0) set_status(a.status, SD_TIMEOUT_AT(40));
  }
}

// Joins the parts of the units that CTAs share, a warp a row, in CTA order (so a call
// gives the same bits every time): o = sum 2^(ref_c - ref) o_c / sum 2^(ref_c - ref) l_c.
// Bound by the latency of the parts' loads, four parts of a row in flight: 12.7
// us for the 40 MB of 151 split units with a cold L2 (they were written just before), 4.5
// to 10 for fewer; with a pass of its own for the maximum 16.9 and 5.3 to 12.9.
template <int D>
__global__ void __launch_bounds__(256) k_prompt_join(const __grid_constant__ PaJoins jn, const int32_t* cu_q, int hq, int G, int T,
                                                     int U, const float* parts, uint16_t* out, float* lse) {
  const PaAt b = jn.at[blockIdx.x];
  const int lane = threadIdx.x & 31, row = blockIdx.y * 8 + (threadIdx.x >> 5);  // tile * 128 + row of it
  const int q0 = cu_q[b.r], m = cu_q[b.r + 1] - q0, tc = min(U, m - b.i * U);
  const int idx = row & 127, tk = idx / G, tok = (row >> 7) * T + tk;
  if (tk >= T || tok >= tc) return;
  const int head = b.h * G + idx - tk * G;
  const int c0 = jn.cta[blockIdx.x], n = b.step;
  auto part_of = [&](int p) { return parts + (int64_t)(p == 0 ? 2 * c0 + 1 : 2 * (c0 + p)) * PaShape<D>::kPart; };
  pdl_wait();  // up to here only what the first kernel does not write
  // a part's weights come to less than 1/2: those of n parts are scaled so that they all do
  const float share = (float)(32 - __clz(n - 1));
  float M = -INFINITY, L = 0.f;
  constexpr int kF = D / 32;
  float acc[kF] = {};
  for (int c = 0; c < n; c += 4) {
    float2 ml[4];
    float v[4][kF];
#pragma unroll
    for (int k = 0; k < 4; k++) {
      ml[k] = make_float2(-INFINITY, 0.f);
      if (c + k >= n) continue;
      const float* pc = part_of(c + k);
      ml[k] = __ldcg(reinterpret_cast<const float2*>(pc + 256 * D) + row);
      if constexpr (kF == 4) {
        const float4 u = __ldcg(reinterpret_cast<const float4*>(pc + (int64_t)row * D) + lane);
        v[k][0] = u.x, v[k][1] = u.y, v[k][2] = u.z, v[k][3] = u.w;
      } else {
        const float2 u = __ldcg(reinterpret_cast<const float2*>(pc + (int64_t)row * D) + lane);
        v[k][0] = u.x, v[k][1] = u.y;
      }
    }
    float top = M;
#pragma unroll
    for (int k = 0; k < 4; k++) top = fmaxf(top, ml[k].x);
    const float Ms = top == -INFINITY ? 0.f : top, al = ex2(M - Ms);
    M = top;
    L *= al;
#pragma unroll
    for (int q = 0; q < kF; q++) acc[q] *= al;
#pragma unroll
    for (int k = 0; k < 4; k++)
      if (!(ml[k].y == 0.f)) {
        const float f = ex2(ml[k].x - Ms - share);
        L = fmaf(f, ml[k].y, L);
#pragma unroll
        for (int q = 0; q < kF; q++) acc[q] = fmaf(f, v[k][q], acc[q]);
      }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int64_t at = (int64_t)(q0 + b.i * U + tok) * hq + head;
  uint32_t* dst = reinterpret_cast<uint32_t*>(out + at * D) + lane * (kF / 2);
#pragma unroll
  for (int q = 0; q < kF; q += 2) dst[q / 2] = pa_bf16x2(acc[q] * inv, acc[q + 1] * inv);
  if (lane == 0 && lse) lse[at] = L == 0.f ? -INFINITY : (M + (log2f(L) + share)) * (1.f / kLog2e);
}

// ------------------------------------------------------------------ host --

// How a call's units are dealt over at most `ctas` CTAs: where each share begins,
// and the units that are split.
struct PaPlan {
  int ctas = 0, U = 0;
  std::vector<PaAt> at;    // [ctas + 1]
  std::vector<PaAt> join;  // step: parts
  std::vector<int> first;  // CTA of a join's first part
};

static int steps_of(int64_t p0, int64_t p1, int window) {
  if (p1 < 0) return 0;
  const int64_t lo = window > 0 ? std::max<int64_t>(p0 - window + 1, 0) / pa::kKeys : 0;
  return (int)(p1 / pa::kKeys + 1 - lo);
}

// A wide step costs 4, a narrow one 3, a unit's beginning and end kUnit.  (Narrow steps
// at 2: 512 rows after 32768 keys, twelve of them in a narrow unit, 292 us against 248.)
constexpr int kUnit = 8, kPiece = 4;

static void pa_plan(PaPlan& pl, const int32_t* cu_q, const int32_t* cu_k, int R, int hkv, int T, int window, int ctas) {
  auto m_of = [&](int r) { return cu_q[r + 1] - cu_q[r]; };
  // Few rows: a tile a unit, its keys shared by both groups, so that more CTAs have a unit's
  // beginning and end (32 heads of 128: 512 rows 11.9 us for 13.0, 64 rows over 8192
  // keys 23.4 for 24.4; over long contexts K and V are read more often, 512 rows over
  // 8192 keys 63 for 59).
  int64_t wide_units = 0;
  for (int r = 0; r < R; r++) wide_units += (int64_t)hkv * ((m_of(r) + 2 * T - 1) / (2 * T));
  pl.U = wide_units * 2 <= ctas ? T : 2 * T;
  const int U = pl.U;
  struct Unit {
    int steps, cost;  // of the unit; a step's
  };
  std::vector<Unit> units;           // of a kv head, request after request
  std::vector<int64_t> cost0;        // before each unit, within its request and kv head
  std::vector<int> begin(R + 1);
  std::vector<int64_t> head_cost(R);
  int64_t total = 0, pieces = 0;
  for (int r = 0; r < R; r++) {
    begin[r] = (int)units.size();
    const int m = m_of(r), past = cu_k[r + 1] - cu_k[r] - m;
    int64_t c = 0;
    for (int t = 0; t < m; t += U) {
      const int tc = std::min(U, m - t);
      const Unit u = {std::max(1, steps_of((int64_t)past + t, (int64_t)past + t + tc - 1, window)), tc > T ? 4 : 3};
      units.push_back(u);
      cost0.push_back(c);
      c += kUnit + (int64_t)u.steps * u.cost;
      pieces += (int64_t)hkv * ((u.steps + kPiece - 1) / kPiece);
    }
    head_cost[r] = c;
    total += c * hkv;
  }
  begin[R] = (int)units.size();
  auto add = [&](int r, int h, int i, int step) {
    pl.at.push_back({r, h, i, step});
  };
  if (pieces <= ctas) {
    // little work: every unit in even pieces of about kPiece steps, a CTA each
    for (int r = 0; r < R; r++)
      for (int h = 0; h < hkv; h++)
        for (int i = 0; i < begin[r + 1] - begin[r]; i++) {
          const int n = units[begin[r] + i].steps, k = (n + kPiece - 1) / kPiece;
          for (int x = 0; x < k; x++) add(r, h, i, (int)((int64_t)n * x / k));
        }
  } else {
    int r = 0;
    int64_t before = 0;  // cost of the requests before r
    for (int c = 0; c < ctas; c++) {
      const int64_t want = total * c / ctas;
      while (r + 1 < R && want >= before + head_cost[r] * hkv) before += head_cost[r] * hkv, r++;
      if (begin[r + 1] == begin[r]) continue;
      int h = (int)std::min<int64_t>((want - before) / head_cost[r], hkv - 1);
      const int64_t in = want - before - head_cost[r] * h;
      const int nu = begin[r + 1] - begin[r];
      int i = (int)(std::upper_bound(cost0.begin() + begin[r], cost0.begin() + begin[r + 1], in) - (cost0.begin() + begin[r])) - 1;
      const Unit& u = units[begin[r] + i];
      int step = (int)((in - cost0[begin[r] + i] - kUnit / 2) / u.cost);
      // no part of less than three steps
      if (step < 3) step = 0;
      if (step > u.steps - 3) {
        step = 0;
        if (in - cost0[begin[r] + i] >= kUnit && ++i == nu) {
          i = 0;
          if (++h == hkv) {
            h = 0;
            int q = r + 1;
            while (q < R && begin[q + 1] == begin[q]) q++;
            if (q == R) break;
            if (!pl.at.empty() && pl.at.back().r == q && pl.at.back().h == 0 && pl.at.back().i == 0) continue;
            add(q, 0, 0, 0);
            continue;
          }
        }
      }
      const PaAt x = {r, h, i, step};
      if (!pl.at.empty()) {
        const PaAt& y = pl.at.back();
        const bool after = x.r != y.r ? x.r > y.r : x.h != y.h ? x.h > y.h : x.i != y.i ? x.i > y.i : x.step > y.step;
        if (!after) continue;
      }
      pl.at.push_back(x);
    }
  }
  pl.ctas = (int)pl.at.size();
  add(R, 0, 0, 0);
  for (int c = 1; c < pl.ctas; c++) {
    if (pl.at[c].step == 0) continue;
    const PaAt& x = pl.at[c];
    if (!pl.join.empty() && pl.join.back().r == x.r && pl.join.back().h == x.h && pl.join.back().i == x.i) {
      pl.join.back().step++;
    } else {
      pl.join.push_back({x.r, x.h, x.i, 2});
      pl.first.push_back(c - 1);
    }
  }
}

static int pa_map(CUtensorMap* map, const uint16_t* p, int D, int64_t heads, int64_t rows, int64_t stride, int box_heads,
                  int box_rows, const char* who) {
  auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!fn) {
    set_error("cuTensorMapEncodeTiled unavailable");
    return SD_ERR_CUDA;
  }
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows}, es[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(p), dims, strides, box, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error(std::string(who) + ": cuTensorMapEncodeTiled failed: " + std::to_string((int)r));
    return SD_ERR_CUDA;
  }
  return SD_OK;
}

template <int D>
static int pa_launch(PaArgs& a, const PaPlan& pl, cudaStream_t st) {
  constexpr int smem = PaShape<D>::smem;
  static const cudaError_t set[3] = {
      cudaFuncSetAttribute(k_prompt_attn<D, kPlain>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
      cudaFuncSetAttribute(k_prompt_attn<D, kSlopes>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
      cudaFuncSetAttribute(k_prompt_attn<D, kCapped>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)};
  const int mode = a.s.cap > 0.f ? kCapped : a.s.slopes ? kSlopes : kPlain;
  SD_CK(set[mode]);
  auto kern = mode == kCapped ? k_prompt_attn<D, kCapped> : mode == kSlopes ? k_prompt_attn<D, kSlopes> : k_prompt_attn<D, kPlain>;
  kern<<<(unsigned)pl.ctas, pa::kThreads, smem, st>>>(a);
  SD_CK(cudaGetLastError());
  if (!pl.join.empty()) {
    PaJoins j;
    j.n = (int)pl.join.size();
    std::copy(pl.join.begin(), pl.join.end(), j.at);
    std::copy(pl.first.begin(), pl.first.end(), j.cta);
    const dim3 grid((unsigned)j.n, a.U > a.T ? 32 : 16);
    SD_CK(launch(k_prompt_join<D>, grid, dim3(256), 0, st, true, j, a.cu_q, a.hq, a.G, a.T, a.U, (const float*)a.part, a.out, a.lse));
  }
  return SD_OK;
}

}  // namespace sdv

using namespace sdv;

// Of the calls to come (sd_debug_prompt_wait).
static std::atomic<uint32_t> pa_limit{(uint32_t)kWaitLimitNs};
static std::atomic<uint32_t> pa_loads{UINT32_MAX};

extern "C" int sd_debug_prompt_wait(int64_t limit_ns, int64_t loads) {
  if (limit_ns < 0 || limit_ns > (int64_t)kWaitLimitNs || loads < 0) {
    set_error("sd_debug_prompt_wait: a limit of 0 .. 2 s and loads >= 0 are needed");
    return SD_ERR_INVALID_ARG;
  }
  pa_limit = (uint32_t)(limit_ns ? limit_ns : (int64_t)kWaitLimitNs);
  pa_loads = limit_ns ? (uint32_t)std::min<int64_t>(loads, UINT32_MAX) : UINT32_MAX;
  return SD_OK;
}

static int pa_ctas() { return std::min(num_sms(), pa::kMaxCta); }

extern "C" size_t sd_prompt_attn_workspace(int32_t head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  return (size_t)2 * pa_ctas() * (head_dim == 128 ? PaShape<128>::kPart : PaShape<64>::kPart) * sizeof(float);
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
  PaArgs a = {};
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
  auto meets = [&](const uint16_t* x, int64_t n, int64_t stride, int heads) {  // out's rows and n of another tensor
    const uintptr_t x0 = (uintptr_t)x, x1 = x0 + 2 * ((uintptr_t)(n - 1) * stride + (uintptr_t)heads * head_dim);
    const uintptr_t o0 = (uintptr_t)out, o1 = o0 + 2 * (uintptr_t)rows * n_q_heads * head_dim;
    return n > 0 && x0 < o1 && o0 < x1;
  };
  if (meets(q, rows, q_stride, n_q_heads) || meets(k, keys, kv_stride, n_kv_heads) || meets(v, keys, kv_stride, n_kv_heads))
    return kv4_bad(SD_ERR_INVALID_ARG, who, "out overlaps q, k or v");
  if ((int64_t)rows * n_q_heads > 0x7FFFFFFF) return kv4_bad(SD_ERR_UNSUPPORTED, who, "more than 2^31 rows and heads");
  a.v = v, a.kv_stride = kv_stride;
  a.hq = n_q_heads, a.hkv = n_kv_heads, a.G = n_q_heads / n_kv_heads, a.R = R;
  a.T = 128 / a.G;
  a.cu_q = cu_q, a.cu_k = cu_k, a.out = out, a.lse = lse, a.part = (float*)workspace, a.status = status;
  a.limit = pa_limit, a.loads = pa_loads;
  if (a.s.cap > 0.f) {
    const double in = (double)a.s.scale / a.s.cap, out = (double)a.s.cap * 1.4426950408889634;
    a.k0 = (float)(out * in);
    a.k1 = (float)(out * in * in * in * (-1.0 / 3.0));
    a.k2 = (float)(out * std::pow(in, 5) * (2.0 / 15.0));
    a.k3 = (float)(out * std::pow(in, 7) * (-17.0 / 315.0));
    a.k4 = (float)(out * std::pow(in, 9) * (62.0 / 2835.0));
    a.series = (float)(0.3 / in);
    // coefficients outside fp32's normal range leave the general form
    if (!(std::fabs(a.k4) > 1e-37f && a.k0 < 1e37f && a.series < 1e37f)) a.series = -1.f;
  }
  PaPlan pl;
  try {
    pa_plan(pl, cu_q_host, cu_k_host, R, n_kv_heads, a.T, a.s.window, pa_ctas());
  } catch (const std::exception&) {
    return kv4_bad(SD_ERR_OOM, who, "out of host memory");
  }
  a.U = pl.U;
  std::copy(pl.at.begin(), pl.at.end(), a.at);
  if (int rc = pa_map(&a.qmap, q, head_dim, n_q_heads, rows, q_stride, a.G, a.T, who)) return rc;
  // no keys: the maps are not read
  if (int rc = pa_map(&a.kmap, keys ? k : q, head_dim, keys ? n_kv_heads : n_q_heads, keys ? keys : rows, keys ? kv_stride : q_stride, 1, pa::kKeys, who))
    return rc;
  if (int rc = pa_map(&a.vmap, keys ? v : q, head_dim, keys ? n_kv_heads : n_q_heads, keys ? keys : rows, keys ? kv_stride : q_stride, 1, pa::kKeys, who))
    return rc;
  return head_dim == 128 ? pa_launch<128>(a, pl, (cudaStream_t)stream) : pa_launch<64>(a, pl, (cudaStream_t)stream);
}
