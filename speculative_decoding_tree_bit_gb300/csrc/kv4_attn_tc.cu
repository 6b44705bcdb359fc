// Attention over the 4-bit cache on the tensor cores (tcgen05 + TMEM), for
// many rows a kv head: trees of many nodes, wide head groups.
//
// S = Q K^T and O += P V with two tiles t of up to 128 query rows, per tile of
// 64 keys (two records).  Tensor memory of a tile: [S or P 64][S or P 64][O D]:
// P replaces its S, and the next key tile's S is there before this one's P is,
// so the softmax warps never wait for a product.  Warps, each role walking the
// CTA's units on its own:
//  * 16: records into a ring of eight, one bulk copy each;
//  * 0..3 and 4..7: nibbles to fp16 operands, K's and V's.
//    K's codes as they are (subnormal code 2^-24; the key's scale and middle
//    are applied to its score, as in the warp kernel); V's as values, s code + (m
//    - 8 s) in one fp16 multiply-add per pair after a power of two, 2^-E for all
//    keys of the unit (11 bits of the value and of m - 8 s, against the output's
//    8).  A unit whose values differ in size by more than 2^6 is taken apart: each
//    key has an E of its own, which its weight makes up for.  The rows' own keys
//    are a tile of 64 in the same form, bf16 to fp16 after a power of two, per key
//    for K;
//  * 17: the products;
//  * 8..15: softmax, a thread per row: the scores of 64 keys from TMEM, maximum,
//    exponentials, P back.  A row's reference, its greatest score + E, may lag by
//    2^6 before O is rescaled in TMEM (fp16 P: exponentials are taken 2^9 up, at
//    most 2^15).  So weights down to 2^-17 of the row's greatest p |v| keep their 11
//    bits, down to 2^-28 count, and nothing that a row does not see moves its
//    weights or values.  (A factor per key in every unit, not in those taken apart
//    alone: 412 us where the tree of 64 below took 362.)
// (18 and 19 do nothing: they complete a warpgroup.  Registers a scheduler:
// 5 warps x 96 = 2 x 72 decoding + 2 x 144 softmax + 48, or 80 and 136, 64 and 152.)
// WIDE: the first rows of a segment are tile 0's, the others tile 1's, up to
// 256.  Not WIDE (at most 128 rows a segment): both tiles hold the same rows and
// take alternate key tiles.  With at most 64 (32) rows a tile holds them twice
// (four times), a copy in other lanes taking half (a quarter) of the keys and
// leaving P 0 in the others': the products cost the same, the softmax is shared
// by all schedulers, each of which reaches only its quarter of the lanes.  The
// copies' partial sums are added in shared memory at a segment's end; the parts
// of a segment that spans CTAs are joined by a second kernel, in a fixed order.
//
// Measured: a tree of 64 with 40 query and 8 kv heads over 131072 keys, D = 128
// (WIDE, two segments of 160 rows a kv head): 366 us, 470 TFLOP/s; with every
// unit taken apart 603.  The 160 rows are split 96 / 64, so that the schedulers
// have 2, 2, 1 and 0 softmax warps, and the products run 512 rows for 320; bound
// by the two schedulers' softmax warps, which wait for tensor memory and their own
// chains (one score buffer a tile took 438 us where two took 397; four softmax
// warps, 500).  Not WIDE, 8 requests of 128 rows over 16000 keys: 187 us.
#include <algorithm>
#include <type_traits>

#include "kv4_attn.cuh"
#include "kv4_rows.cuh"
#include "tcgen05.cuh"

namespace sdv {

namespace kt {
constexpr int kSoft = 8, kLoad = 16, kMma = 17, kThreads = 20 * 32, kSoftThreads = 256;
constexpr int kRaw = 8;
constexpr int kRows = 256;  // of a segment, at most
constexpr int kJoins = 4;   // segments of a (request, kv head), at most: 64 rows x 16 heads
constexpr int kUp = -5;       // V operands are values times 2^(kUp - E), below 2^kUp: s 2^(24 + kUp - E) fits fp16
constexpr int kApart = 6;     // the keys of a unit share one E while their magnitudes are within 2^6
constexpr float kBase = 9.f;  // P is 2^kBase at the reference, 2^15 at most
}  // namespace kt

template <int D, bool WIDE, bool BIAS = false>
struct TcShape {
  static constexpr int NS = WIDE ? 3 : 4;                            // operand stages
  static constexpr int kStage = kv4_rec(D) + 128;
  static constexpr int kOp = 64 * D * 2;                             // 64 keys, fp16
  static constexpr int kQ = 128 * D * 2;                             // a tile of queries, fp16
  static constexpr int kX = 36;                                      // floats of a row being added up
  static constexpr int off_q = NS * 2 * kOp;                         // [WIDE ? 2 : 1]; shared with [2 t][128][kX] floats
  static constexpr int kQs = (WIDE ? 2 : 1) * kQ;
  static constexpr int off_raw = off_q + (kQs > 256 * kX * 4 ? kQs : 256 * kX * 4);  // [kRaw][kStage]
  static constexpr int off_sc = off_raw + kt::kRaw * kStage;         // [NS][32] key pairs: (m / s - 8) twice, s twice
  static constexpr int off_pos = off_sc + NS * 64 * 8;               // [NS][64]
  static constexpr int off_e = off_pos + NS * 64 * 4;                // [NS][64] E of a key, in units taken apart
  static constexpr int off_info = off_e + NS * 64 * 4;               // [NS] (keys held + kTcOwn + kTcApart, masks of either half, E)
  static constexpr int off_bar = off_info + NS * 16;
  static constexpr int off_ok = off_bar + (2 * kt::kRaw + 2 * NS + 14) * 8;
  static constexpr int off_vmax = off_ok + kt::kRaw * 4;             // [4] (greatest, least magnitude)
  static constexpr int off_ml = off_vmax + 32;                       // [2 t][128] (reference, sum)
  static constexpr int off_inv = off_ml + 256 * 8;                   // [kRows] 1 / sum
  static constexpr int smem = off_inv + kt::kRows * 4 + 1024;
  // Registers of the decoding warps; the softmax warps have 216 less these.  Each
  // form's best of 64, 72 and 80 (96 rows over 65536 keys: 107, 107, 104 us; with
  // a cap 116, 123, 123; 320 rows over 131072 keys 388, 362, 397).
  static constexpr int kDecodeRegs = WIDE ? 72 : BIAS ? 64 : 80;
  static constexpr int kPart = kt::kRows * (D + 2);                  // floats of a part: [rows][D], then [rows] (max, sum)
};

// N consecutive 32-bit columns of this thread's TMEM lane, waited for.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; i++) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; i++) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[64]) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 64; i++) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};\n\ttcgen05.wait::st.sync.aligned;" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};\n\ttcgen05.wait::st.sync.aligned;" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};\n\ttcgen05.wait::st.sync.aligned;" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
      : "memory");
}
// D (tmem) (+)= A (smem) * B (smem)^T, or A (tmem) * B (smem), fp16.
__device__ __forceinline__ void umma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  umma_bf16(d, a, b, idesc, accumulate);  // the operands' type is in the descriptor
}
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// B operand with its N side contiguous, 128-byte swizzle: rows of 64 values, 8
// rows 1024 bytes, panels of 64 values 8192 bytes apart.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(8192 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ uint32_t h2dup(float x) { return pack_f16x2(x, x); }
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t y;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(a), "r"(b), "r"(c));
  return y;
}
// Exponent e of |x| < 2^(e+1); -127 of 0 and subnormals.
__device__ __forceinline__ int expo(uint32_t bits) { return (int)(bits >> 23 & 255) - 127; }

// A bound on the magnitudes of a row with scale s and middle m, as bits.
__device__ __forceinline__ uint32_t kv4_magnitude(float s, float m) { return __float_as_uint(fmaf(8.f, s, fabsf(m))); }
// E of values of magnitude at most |x| (bits), which lie below 2^E; past 2^121 the
// operands have to be finite, no more.
__device__ __forceinline__ int tc_exponent(uint32_t bits) { return min(max(expo(bits) + 1, -90), 121); }

// A CTA's walk over its segments, by whole warps.
template <bool BIAS>
struct TcWalk {
  int r, s, seg, ua, ub;
  Kv4Req rq;
  __device__ __forceinline__ TcWalk(const Kv4AttnArgs& a, const Kv4Share& sh) : r(sh.r0), s(sh.s0), seg(sh.seg0) {
    rq = kv4_req<kt::kRows, 2, BIAS>(a, r);
    ua = sh.u0 - seg;
    ub = min(rq.nu, sh.u1 - seg);
  }
  __device__ __forceinline__ bool next(const Kv4AttnArgs& a, const Kv4Share& sh) {
    seg += rq.nu;
    if (seg >= sh.u1) return false;
    if (++s == a.c.hkv * rq.nc) {
      s = 0;
      do rq = kv4_req<kt::kRows, 2, BIAS>(a, ++r);
      while (rq.nc == 0);
    }
    ua = 0;
    ub = min(rq.nu, sh.u1 - seg);
    return true;
  }
  __device__ __forceinline__ int head() const { return s / rq.nc; }
  __device__ __forceinline__ int groups_end() const { return (rq.ctx + kKvGroup - 1) / kKvGroup; }
  // groups of 32 keys of unit u
  __device__ __forceinline__ int groups(const Kv4AttnArgs& a, int u) const {
    if (u < rq.no) return a.k_new ? (rq.m + 31) / 32 : 1;
    return min(2, groups_end() - (rq.g0 + 2 * (u - rq.no)));
  }
};

// Joins the parts of segments that span CTAs, a warp a row.  The last of a
// segment's CTAs could do it and save the launch, but with many parts a
// segment it leaves the other CTAs idle: 96 / 256 rows over 2000 keys 31 / 52
// us against 24 / 28 with this kernel, over 65536 keys 113 / 206 against 96 /
// 132; eight such requests of 2000 keys, one or two parts each, 49 / 70
// against 49 / 67.
template <int D, bool WIDE>
__global__ void __launch_bounds__(256) k_kv4_join(Kv4AttnArgs a, int rows) {
  pdl_wait();
  const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);  // (row, query head)
  if (i >= (int64_t)rows * a.hq) return;
  const int lane = threadIdx.x & 31;
  const int e = (int)(i / a.hq), hq = (int)(i - (int64_t)e * a.hq), h = hq / a.G;
  const int r = request_of(a.cu, a.R, e);
  const Kv4Req rq = kv4_req_rows<kt::kRows>(a, r);
  if (rq.m == 0) return;
  const int rho = (hq - h * a.G) * rq.m + e - rq.n0;
  const int run = TcRowsOf<WIDE>(a.G * rq.m, rq.nc, 0).run, rc = rho / run, row = rho - rc * run;
  const int4 jn = a.joins[((int64_t)r * a.c.hkv + h) * kt::kJoins + rc];  // (first CTA, parts, first slot, -)
  if (jn.y == 0) return;  // whole in one CTA, which wrote it
  auto part_of = [&](int p) { return a.part + (int64_t)(p == 0 ? jn.z : 2 * (jn.x + p)) * TcShape<D, WIDE>::kPart; };
  float M = -INFINITY, L = 0.f;
  for (int p = lane; p < jn.y; p += 32) M = fmaxf(M, __ldcg(part_of(p) + kt::kRows * D + 2 * row));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float Ms = M == -INFINITY ? 0.f : M;
  constexpr int kF = D / 32;  // dims of a lane
  float acc[kF] = {};
  for (int c = 0; c < jn.y; c += 8) {
    float2 ml[8];
    float v[8][kF];
#pragma unroll
    for (int k = 0; k < 8; k++) {
      const float* pc = part_of(min(c + k, jn.y - 1));
      ml[k] = __ldcg(reinterpret_cast<const float2*>(pc + kt::kRows * D) + row);
      if constexpr (kF == 4) {
        const float4 u = __ldcg(reinterpret_cast<const float4*>(pc + row * D) + lane);
        v[k][0] = u.x, v[k][1] = u.y, v[k][2] = u.z, v[k][3] = u.w;
      } else {
        const float2 u = __ldcg(reinterpret_cast<const float2*>(pc + row * D) + lane);
        v[k][0] = u.x, v[k][1] = u.y;
      }
    }
#pragma unroll
    for (int k = 0; k < 8; k++)
      if (c + k < jn.y) {
        const float f = ex2(ml[k].x - Ms);
        L = fmaf(f, ml[k].y, L);
#pragma unroll
        for (int q = 0; q < kF; q++) acc[q] = fmaf(f, v[k][q], acc[q]);
      }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  uint32_t* out = reinterpret_cast<uint32_t*>(a.out + i * D) + lane * (kF / 2);
#pragma unroll
  for (int q = 0; q < kF; q += 2) out[q / 2] = pack_bf16x2(acc[q] * inv, acc[q + 1] * inv);
  if (lane == 0 && a.lse) a.lse[i] = L == 0.f ? -INFINITY : (M + log2f(L)) * (1.f / kLog2e);
}

// A softmax thread's row in a segment, and what its loop leaves.
struct TcRow {
  float qsf, fac, slope;   // sum of q, factor of a score, slope
  int qpos, start, key0;   // position, document start, the copy's first key of a tile
  uint64_t anc;
  bool live;               // the warp has rows
  float ref, l;            // the greatest score + E, give or take 6; the sum of 2^(kBase + x - ref)
  bool any;
};

constexpr int kTcOwn = 256, kTcApart = 512;  // s_info: the rows' own keys; each key has its E in s_e

// The scores of a tile's keys key0 .. key0 + N - 1 from TMEM (times 1 / fac without
// options), -inf where the row does not see the key.
template <bool BIAS, int N>
__device__ __forceinline__ void tc_scores(const Kv4AttnArgs& a, const TcRow& w, uint32_t tmem, int key0, const int4& info,
                                          const float2* s_sc, const int* s_pos, float (&x)[N]) {
  tmem_ld(tmem + key0, x);
  const ulonglong2* sc = reinterpret_cast<const ulonglong2*>(s_sc + key0);
  const uint64_t qq = f2pack(w.qsf, w.qsf);
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const ulonglong2 v = sc[c / 2];
    f2unpack(f2mul(f2fma(v.x, qq, f2pack(x[c], x[c + 1])), v.y), x[c], x[c + 1]);
  }
  if (BIAS) {
#pragma unroll
    for (int c = 0; c < N; c += 2) f2unpack(f2mul(f2pack(x[c], x[c + 1]), f2pack(w.fac, w.fac)), x[c], x[c + 1]);
    const int* kp = s_pos + key0;
    kv4_cap(a.s, x);
    kv4_bias(a.s, x, w.slope, w.qpos, w.start, [&](int c) { return kp[c]; });
  }
  if ((info.x & ~kTcApart) != 64) {  // not every key is held, or the rows' own keys
    const uint64_t held = (uint64_t)(uint32_t)info.z << 32 | (uint32_t)info.y;
    const uint64_t see = (info.x & kTcOwn ? held & w.anc : held) >> key0;
#pragma unroll
    for (int c = 0; c < N; c++)
      if (!(see >> c & 1)) x[c] = -INFINITY;
  }
}

// O times al, a row's own factor, in TMEM.  The product before may still be adding
// to O (the one before that was done before these scores).
template <int D>
__device__ __forceinline__ void tc_rescale(uint32_t tb, float al, uint64_t* o_full, uint32_t parity, int* s_abort, int32_t* status) {
  if (!kv4_wait(o_full, parity, s_abort)) set_status(status, SD_TIMEOUT_AT(35));
  tc_fence_after();
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    float o[16];
    tmem_ld(tb + 128 + c, o);
    uint32_t y[16];
#pragma unroll
    for (int k = 0; k < 16; k++) y[k] = __float_as_uint(o[k] * al);
    tmem_st(tb + 128 + c, y);
  }
}

// One unit whose values differ too much in size for one E: each key has its own.
// Rare, so 16 keys at a time and the scores twice; P takes the place of scores
// that are already read.
template <int D, bool BIAS>
__device__ __forceinline__ void tc_apart(const Kv4AttnArgs& a, TcRow& w, uint32_t tb, uint32_t buf, int nk, const int4& info,
                                         const float2* s_sc, const int* s_pos, const float* s_e, uint64_t* o_full,
                                         uint32_t parity, int* s_abort) {
  const float f = BIAS ? 1.f : w.fac;
  float top = -INFINITY;
#pragma unroll 1
  for (int c0 = w.key0; c0 < w.key0 + nk; c0 += 16) {
    float x[16];
    tc_scores<BIAS>(a, w, tb + buf, c0, info, s_sc, s_pos, x);
#pragma unroll
    for (int c = 0; c < 16; c++) top = fmaxf(top, fmaf(x[c], f, s_e[c0 + c]));
  }
  const bool grows = top > w.ref + 6.f || (w.ref == -INFINITY && top > w.ref);
  if (__any_sync(0xffffffffu, grows)) {
    const float al = grows ? ex2(w.ref - top) : 1.f;
    if (grows) w.ref = top;
    w.l *= al;
    if (w.any) tc_rescale<D>(tb, al, o_full, parity, s_abort, a.status);
  }
  const float off = kt::kBase - (w.ref == -INFINITY ? 0.f : w.ref);
#pragma unroll 1
  for (int c0 = w.key0; c0 < w.key0 + nk; c0 += 16) {
    float x[16];
    tc_scores<BIAS>(a, w, tb + buf, c0, info, s_sc, s_pos, x);
    uint32_t p[8];
#pragma unroll
    for (int c = 0; c < 16; c += 2) {
      const float e0 = s_e[c0 + c], e1 = s_e[c0 + c + 1];
      const float p0 = ex2(fmaf(x[c], f, off + e0)), p1 = ex2(fmaf(x[c + 1], f, off + e1));
      w.l = fmaf(p0, ex2(-e0), fmaf(p1, ex2(-e1), w.l));
      p[c / 2] = pack_f16x2(p0, p1);
    }
    tmem_st(tb + buf + c0 / 2, p);
  }
  const uint32_t none[8] = {};
#pragma unroll 1
  for (int c = 0; c < 64; c += 16)
    if (c < w.key0 || c >= w.key0 + nk) tmem_st(tb + buf + c / 2, none);
}

// The softmax of a segment's units of tile t, NC keys of each (the copy's share).
template <int D, bool BIAS, bool WIDE, int NC>
__device__ __forceinline__ void tc_softmax(const Kv4AttnArgs& a, TcRow& w, uint32_t tb, int i0, int n, uint32_t op0,
                                           uint32_t& par, uint64_t* s_full, uint64_t* op_full, uint64_t* p_full,
                                           uint64_t* o_full, const float2* s_sc, const int* s_pos, const float* s_e,
                                           const int4* s_info, int* s_abort) {
  constexpr int NS = TcShape<D, WIDE>::NS, step = WIDE ? 1 : 2;
  const int lane = threadIdx.x & 31;
  const float f = BIAS ? 1.f : w.fac;  // > 0
#pragma unroll 1
  for (int i = i0; i < n;) {
#pragma unroll 1
    for (; i < n; i += step) {
      const uint32_t st = (op0 + i) % NS;
      const int b = WIDE ? i & 1 : i >> 1 & 1;
      const uint32_t buf = b * 64;  // first TMEM column of the unit's scores
      if (!kv4_wait(s_full + b, par >> b & 1, s_abort)) set_status(a.status, SD_TIMEOUT_AT(33));
      par ^= 1u << b;
      if (!kv4_wait(&op_full[st], (op0 + i) / NS & 1, s_abort)) set_status(a.status, SD_TIMEOUT_AT(34));
      tc_fence_after();
      const int4 info = s_info[st];
      if (info.x & kTcApart) break;
      if (w.live) {
        float x[NC];
        tc_scores<BIAS>(a, w, tb + buf, w.key0, info, s_sc + st * 64, s_pos + st * 64, x);
        float t4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < NC; c++) t4[c & 3] = fmaxf(t4[c & 3], x[c]);
        const float E = __int_as_float(info.w);
        const float top = fmaf(fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])), f, E);
        const bool grows = top > w.ref + 6.f || (w.ref == -INFINITY && top > w.ref);
        if (__any_sync(0xffffffffu, grows)) {
          const float al = grows ? ex2(w.ref - top) : 1.f;
          if (grows) w.ref = top;
          w.l *= al;
          if (w.any) tc_rescale<D>(tb, al, o_full + (b ^ 1), par >> (b ^ 1) & 1 ^ 1, s_abort, a.status);
        }
        const float off = kt::kBase + E - (w.ref == -INFINITY ? 0.f : w.ref);
        uint32_t p[NC / 2];
        uint64_t l4[2] = {0, 0};
        const uint64_t ff = f2pack(f, f), oo = f2pack(off, off);
#pragma unroll
        for (int c = 0; c < NC; c += 2) {
          float p0, p1;
          f2unpack(f2fma(f2pack(x[c], x[c + 1]), ff, oo), p0, p1);
          p0 = ex2(p0);
          p1 = ex2(p1);
          l4[c >> 1 & 1] = f2add(l4[c >> 1 & 1], f2pack(p0, p1));
          p[c / 2] = pack_f16x2(p0, p1);
        }
        {
          float l0, l1;
          f2unpack(f2add(l4[0], l4[1]), l0, l1);
          w.l = fmaf(l0 + l1, ex2(-E), w.l);
        }
        if constexpr (NC == 64) {
          tmem_st(tb + buf, p);
        } else {
          uint32_t y[32];
#pragma unroll
          for (int c = 0; c < 32; c++) y[c] = c / (NC / 2) * NC == w.key0 ? p[c % (NC / 2)] : 0u;
          tmem_st(tb + buf, y);
        }
      }
      w.any = true;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full + b);
    }
    if (i >= n) break;
    const uint32_t st = (op0 + i) % NS;
    const int b = WIDE ? i & 1 : i >> 1 & 1;
    if (w.live)
      tc_apart<D, BIAS>(a, w, tb, b * 64, NC, s_info[st], s_sc + st * 64, s_pos + st * 64, s_e + st * 64, o_full + (b ^ 1),
                        par >> (b ^ 1) & 1 ^ 1, s_abort);
    w.any = true;
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(p_full + b);
    i += step;
  }
}

template <int D, bool BIAS, bool WIDE>
__global__ void __launch_bounds__(kt::kThreads, 1) k_kv4_attn_tc(const __grid_constant__ Kv4AttnArgs a) {
  using S = TcShape<D, WIDE, BIAS>;
  constexpr int NS = S::NS;
  extern __shared__ uint8_t smem_tc[];
  uint8_t* const sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_tc) + 1023) & ~uintptr_t(1023));
  uint8_t* const raw = sm + S::off_raw;
  float2* const s_sc = reinterpret_cast<float2*>(sm + S::off_sc);
  int* const s_pos = reinterpret_cast<int*>(sm + S::off_pos);
  float* const s_e = reinterpret_cast<float*>(sm + S::off_e);
  int4* const s_info = reinterpret_cast<int4*>(sm + S::off_info);
  uint64_t* const raw_full = reinterpret_cast<uint64_t*>(sm + S::off_bar);  // record landed
  uint64_t* const raw_empty = raw_full + kt::kRaw;   // record decoded (8 warps)
  uint64_t* const op_full = raw_empty + kt::kRaw;    // operands, scales written (8 warps)
  uint64_t* const op_empty = op_full + NS;           // products done with them (commit)
  uint64_t* const q_full = op_empty + NS;            // [t] queries in TMEM (4 warps)
  uint64_t* const s_full = q_full + 2;               // [t][buffer] scores ready (commit)
  uint64_t* const p_full = s_full + 4;               // [t][buffer] weights written (4 warps)
  uint64_t* const o_full = p_full + 4;               // [t][buffer] the product with V done (commit)
  int* const s_ok = reinterpret_cast<int*>(sm + S::off_ok);
  uint2* const s_vmax = reinterpret_cast<uint2*>(sm + S::off_vmax);
  float2* const s_ml = reinterpret_cast<float2*>(sm + S::off_ml);
  float* const s_inv = reinterpret_cast<float*>(sm + S::off_inv);
  float* const s_x = reinterpret_cast<float*>(sm + S::off_q);
  __shared__ int s_abort;
  __shared__ uint32_t s_tmem;
  __shared__ Kv4Share sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch();

  if (warp == kt::kSoft) kv4_share<kt::kRows, 2, BIAS>(a, 4, sh);
  if (warp == kt::kMma) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < kt::kRaw; i++) mbar_init(&raw_full[i], 1), mbar_init(&raw_empty[i], 8);
    for (int i = 0; i < NS; i++) mbar_init(&op_full[i], 8), mbar_init(&op_empty[i], 1);
    for (int t = 0; t < 2; t++) {
      mbar_init(&q_full[t], 4);
      for (int b = 0; b < 2; b++)
        mbar_init(&s_full[2 * t + b], 1), mbar_init(&p_full[2 * t + b], 4), mbar_init(&o_full[2 * t + b], 1);
    }
    s_abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = s_tmem;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!kv4_wait(bar, parity & 1, &s_abort)) set_status(a.status, SD_TIMEOUT_AT(32));
  };

  if (sh.u0 >= sh.u1) {
    // no work for this CTA
  } else if (warp >= kt::kLoad) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(48));
    if (warp == kt::kLoad) {
      TcWalk<BIAS> w(a, sh);
      uint32_t n = 0;
      do {
        const int h = w.head(), c0 = max(w.ua, w.rq.no);
        const int ga = w.rq.g0 + 2 * (c0 - w.rq.no), gb = w.ub > c0 ? min(w.groups_end(), w.rq.g0 + 2 * (w.ub - w.rq.no)) : ga;
        for (int base = ga; base < gb; base += 32) {
          const uint8_t* addr = base + lane < gb ? a.c.record(D, w.r, h, base + lane) : nullptr;
          for (int i = 0; i < 32 && base + i < gb; i++, n++) {
            const uint8_t* rec = reinterpret_cast<const uint8_t*>(
                __shfl_sync(0xffffffffu, (unsigned long long)reinterpret_cast<uintptr_t>(addr), i));
            const int slot = n % kt::kRaw;
            wait(&raw_empty[slot], (n / kt::kRaw & 1) ^ 1);
            if (lane == 0) {
              s_ok[slot] = rec != nullptr;
              if (rec) {
                uint8_t* dst = raw + slot * S::kStage;
                mbar_arrive_expect_tx(&raw_full[slot], kv4_rec(D) + (BIAS ? 128 : 0));
                bulk_g2s(dst, rec, kv4_rec(D), &raw_full[slot]);
                if (BIAS) bulk_g2s(dst + kv4_rec(D), a.c.pos + a.c.slot0(w.r, h) + (base + i) * kKvGroup, 128, &raw_full[slot]);
              } else {
                set_status(a.status, SD_ERR_CAPACITY);
                mbar_arrive(&raw_full[slot]);
              }
            }
            __syncwarp();
          }
        }
      } while (w.next(a, sh));
    } else if (warp == kt::kMma) {
      {
        // the whole warp walks and waits; one lane, elected, issues: so the
        // compiler keeps the operands in uniform registers (33 cycles a
        // product of 64 columns, against 45 and more under lane == 0)
        TcWalk<BIAS> w(a, sh);
        const uint32_t id0 = (1u << 4) | (8u << 24);  // fp32 += fp16 fp16, M = 128
        const uint32_t idv = id0 | (1u << 16) | ((uint32_t)(D / 8) << 17);
        const uint64_t kop = sdesc_sw128(smem_u32(sm)), vop = sdesc_mn(smem_u32(sm) + S::kOp),
                       qop = sdesc_sw128(smem_u32(sm + S::off_q));
        uint32_t op0 = 0, np = 0, segs = 0;  // np: parity of each p_full
        do {
          const int n = w.ub - w.ua;
          // scores of tile t and unit i into buffer b
          auto scores = [&](int t, int i, int b) {
            const uint32_t st = (op0 + i) % NS;
            const uint64_t kd = kop + st * (2 * S::kOp >> 4), qd = qop + (WIDE ? t : 0) * (S::kQ >> 4);
            const uint32_t id = id0 | ((uint32_t)(w.groups(a, w.ua + i) * 4) << 17), d = tm + t * 256 + b * 64;
            wait(&op_full[st], (op0 + i) / NS);
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int x = 0; x < D / 16; x++)
                umma_f16_ss(d, qd + (x >> 2) * (16384 >> 4) + (x & 3) * 2, kd + (x >> 2) * (8192 >> 4) + (x & 3) * 2, id, x > 0);
              umma_commit(&s_full[2 * t + b]);
            }
            __syncwarp();
          };
          auto values = [&](int t, int i, int b, bool first, bool release) {
            const uint32_t st = (op0 + i) % NS;
            const uint64_t vd = vop + st * (2 * S::kOp >> 4);
            const bool two = w.groups(a, w.ua + i) == 2;
            const uint32_t o = tm + t * 256 + 128, p = tm + t * 256 + b * 64;
            wait(&p_full[2 * t + b], np >> (2 * t + b));
            np ^= 1u << (2 * t + b);
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int x = 0; x < 4; x++)
                if (x < 2 || two) umma_f16_ts(o, p + 8 * x, vd + x * (2048 >> 4), idv, !first || x > 0);
              umma_commit(&o_full[2 * t + b]);
              if (release) umma_commit(&op_empty[st]);
            }
            __syncwarp();
          };
          wait(&q_full[0], segs);
          if (WIDE) wait(&q_full[1], segs);
          tc_fence_after();
          if (WIDE) {
            for (int i = 0; i < min(n, 2); i++) scores(0, i, i), scores(1, i, i);
            for (int i = 0; i < n; i++) {
              values(0, i, i & 1, i == 0, false);
              values(1, i, i & 1, i == 0, true);
              if (i + 2 < n) scores(0, i + 2, i & 1), scores(1, i + 2, i & 1);
            }
          } else {
            for (int i = 0; i < min(n, 3); i++) scores(i & 1, i, i >> 1);
            for (int i = 0; i < n; i++) {
              values(i & 1, i, i >> 1 & 1, i < 2, true);
              if (i + 3 < n) scores((i + 3) & 1, i + 3, (i + 3) >> 1 & 1);
            }
          }
          op0 += n;
          segs++;
        } while (w.next(a, sh));
      }
      __syncwarp();
    }
  } else if (warp < kt::kSoft) {
      // ------------------------------------------------------- operands --
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kDecodeRegs));
      TcWalk<BIAS> w(a, sh);
      const bool is_k = warp < 4;
      const int dt = tid & 127, dw = warp & 3;
      // eight lanes take four rows' neighbouring 16-byte pieces: two phases a
      // read, none shared a write
      const int row = 16 * (dw & 1) + 4 * (lane >> 3) + (lane >> 1 & 3);
      const int cg = (D == 128 ? 2 * (dw >> 1) : 0) + (lane & 1);
      const bool mine = D == 128 || dw < 2;
      const uint32_t at0 = (is_k ? 0 : S::kOp) + (cg >> 1) * 8192 + row * 128;
      uint32_t op = 0, nraw = 0;
      do {
        const int h = w.head();
        auto put_info = [&](int st, bool apart, int keys, int lo, int hi, int E) {  // what the softmax warps need of a unit
          s_info[st] = make_int4(keys + (apart ? kTcApart : 0), lo, hi, __float_as_int((float)E));
        };
        for (int u = w.ua; u < w.ub; u++, op++) {
          const int st = op % NS;
          uint8_t* const dst = sm + st * 2 * S::kOp;
          if (u >= w.rq.no) {
            const int ga = w.rq.g0 + 2 * (u - w.rq.no), ng = w.groups(a, u);
            // everything this thread needs of the records, then their slots are free
            int lim[2] = {0, 0};
            uint32_t sm0[2] = {0, 0}, ksm = 0, ksv = 0, most = 0, other = 0;
            uint4 x[2];
            int kpos = 0;
#pragma unroll
            for (int gi = 0; gi < 2; gi++) {
              if (gi >= ng) continue;
              const uint32_t slot = (nraw + gi) % kt::kRaw;
              wait(&raw_full[slot], (nraw + gi) / kt::kRaw);
              const uint8_t* rec = raw + slot * S::kStage;
              lim[gi] = s_ok[slot] ? max(0, min(kKvGroup, w.rq.ctx - (ga + gi) * kKvGroup)) : 0;
              if (is_k) {
                if (mine) x[gi] = *reinterpret_cast<const uint4*>(rec + row * (D / 2) + cg * 16);
                if (dw == gi) {
                  ksm = *reinterpret_cast<const uint32_t*>(rec + 16 * D + lane * 4);
                  ksv = *reinterpret_cast<const uint32_t*>(rec + kv4_half(D) + 16 * D + lane * 4);
                  if (BIAS) kpos = *reinterpret_cast<const int*>(rec + kv4_rec(D) + lane * 4);
                }
              } else {
                const uint8_t* v = rec + kv4_half(D);
                if (mine) x[gi] = *reinterpret_cast<const uint4*>(v + row * (D / 2) + (D == 128 ? cg ^ (row & 2) : cg) * 16);
                sm0[gi] = *reinterpret_cast<const uint32_t*>(v + 16 * D + row * 4);
                const uint32_t vw = *reinterpret_cast<const uint32_t*>(v + 16 * D + lane * 4);
                const uint32_t big = kv4_magnitude(__uint_as_float(vw << 16), __uint_as_float(vw & 0xFFFF0000u));
                other = most;
                most = lane < lim[gi] && big <= 0x7F800000u ? min(big, 0x7F7FFFFFu) : 0;  // NaN does not count
              }
            }
            __syncwarp();
            if (lane == 0)
              for (int gi = 0; gi < ng; gi++) mbar_arrive(&raw_empty[(nraw + gi) % kt::kRaw]);
            nraw += ng;
            wait(&op_empty[st], (op / NS & 1) ^ 1);
            if (is_k) {
              if (dw < 2) {
                float2 sc = make_float2(0.f, 0.f);
                if (lane < (dw ? lim[1] : lim[0])) {
                  const float s = __uint_as_float(ksm << 16), m = __uint_as_float(ksm & 0xFFFF0000u);
                  // a row of one value has s = 0 and every code 8: any s will do
                  sc.y = s == 0.f ? fmaxf(fabsf(m) * 0.0625f, 1e-30f) : s;
                  sc.x = m / sc.y - 8.f;
                  if (!(fabsf(__uint_as_float(ksv << 16)) <= 3.4e38f)) sc.x = __int_as_float(0x7FC00000);  // V held as NaN
                  if (BIAS) s_pos[st * 64 + dt] = kpos;
                }
                float* const p = reinterpret_cast<float*>(s_sc + st * 64) + (dt >> 1) * 4 + (dt & 1);
                p[0] = sc.x;
                p[2] = sc.y;
              }
#pragma unroll
              for (int gi = 0; gi < 2; gi++) {
                if (gi >= ng || !mine) break;
                const uint32_t xs[4] = {x[gi].x, x[gi].y, x[gi].z, x[gi].w};
#pragma unroll
                for (int j = 0; j < 4; j++)
                  *reinterpret_cast<uint4*>(dst + at0 + gi * 4096 + ((((cg & 1) * 4 + j) ^ (row & 7)) << 4)) =
                      make_uint4(codes2<0>(xs[j]), codes2<1>(xs[j]), codes2<2>(xs[j]), codes2<3>(xs[j]));
              }
            } else {
              // one E for the unit's keys, or one a key; magnitudes of 0 do not count
              const uint32_t top = __reduce_max_sync(0xffffffffu, max(most, other));
              const uint32_t far = max(top, (uint32_t)kt::kApart << 23) - ((uint32_t)kt::kApart << 23);
              const bool apart = __any_sync(0xffffffffu, (most && most < far) || (other && other < far));
              const int E = tc_exponent(top);
              if (dt == 64) put_info(st, apart, lim[0] + lim[1], lim[0] == 32 ? -1 : (1 << lim[0]) - 1,
                                     lim[1] == 32 ? -1 : (1 << lim[1]) - 1, E);
              if (apart && dw < 2) s_e[st * 64 + dt] = (float)tc_exponent(dw == ng - 1 ? most : ng == 2 ? other : 0u);
#pragma unroll
              for (int gi = 0; gi < 2; gi++) {
                if (gi >= ng || !mine) break;
                float s = __uint_as_float(sm0[gi] << 16), m = __uint_as_float(sm0[gi] & 0xFFFF0000u);
                if (row >= lim[gi] || !(s <= 3.4e38f)) s = m = 0.f;  // not held, or NaN: its scores say so
                s = fminf(s, 3e35f);  // below 2^118: s 2^(24 + kUp - E) is finite
                const int e = apart ? tc_exponent(kv4_magnitude(s, m)) : E;
                const uint32_t me = h2dup(s * pow2i(24 + kt::kUp - e)), mo = h2dup(s * pow2i(20 + kt::kUp - e)),
                               cc = h2dup(fmaf(-8.f, s, m) * pow2i(kt::kUp - e));
                const uint32_t xs[4] = {x[gi].x, x[gi].y, x[gi].z, x[gi].w};
#pragma unroll
                for (int j = 0; j < 4; j++)
                  *reinterpret_cast<uint4*>(dst + at0 + gi * 4096 + ((((cg & 1) * 4 + j) ^ (row & 7)) << 4)) =
                      make_uint4(hfma2(codes2<0>(xs[j]), me, cc), hfma2(codes2<1>(xs[j]), mo, cc),
                                 hfma2(codes2<2>(xs[j]), me, cc), hfma2(codes2<3>(xs[j]), mo, cc));
              }
            }
          } else {
            // the rows' own keys (or values): two threads a row
            wait(&op_empty[st], (op / NS & 1) ^ 1);
            const int j = dt >> 1, half = dt & 1, m = a.k_new ? w.rq.m : 0;
            const bool in = j < m;
            const int64_t off = (int64_t)(w.rq.n0 + j) * a.kv_stride + h * D + half * (D / 2);
            // greatest magnitude of a row, as bits: at 0x7F800000 and above, a
            // NaN or an infinity
            auto row_max = [&](const uint16_t* src) {
              uint32_t big = 0;
#pragma unroll
              for (int i = 0; i < D / 16; i++) {
                const uint4 v = in ? *reinterpret_cast<const uint4*>(src + off + 8 * i) : make_uint4(0, 0, 0, 0);
                const uint32_t vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; k++) big = max(big, max(vs[k] << 16 & 0x7FFF0000u, vs[k] & 0x7FFF0000u));
              }
              return max(big, __shfl_xor_sync(0xffffffffu, big, 1));
            };
            // even and odd dims times up and up4, as the nibbles' order has them
            auto store = [&](const uint16_t* src, float up, float up4, bool zero) {
              uint8_t* const d = dst + (is_k ? 0 : S::kOp) + j * 128;
#pragma unroll
              for (int i = 0; i < D / 16; i++) {
                const uint4 v = in ? *reinterpret_cast<const uint4*>(src + off + 8 * i) : make_uint4(0, 0, 0, 0);
                const uint32_t vs[4] = {v.x, v.y, v.z, v.w};
                float f[8];
#pragma unroll
                for (int k = 0; k < 4; k++) {
                  f[2 * k] = zero ? 0.f : __uint_as_float(vs[k] << 16) * up;
                  f[2 * k + 1] = zero ? 0.f : __uint_as_float(vs[k] & 0xFFFF0000u) * up4;
                }
                const int c = half * (D / 16) + i;  // 16-byte piece of the row
                *reinterpret_cast<uint4*>(d + (c >> 3) * 8192 + (((c & 7) ^ (j & 7)) << 4)) =
                    make_uint4(pack_f16x2(f[0], f[4]), pack_f16x2(f[1], f[5]), pack_f16x2(f[2], f[6]), pack_f16x2(f[3], f[7]));
              }
            };
            if (is_k) {
              const uint32_t vbig = a.k_new ? row_max(a.v_new) : 0;
              const bool odd = vbig >= 0x7F800000u;
              const int e = min(max(10 - expo(a.k_new ? row_max(a.k_new) : 0), -100), 100);  // the greatest below 2^11; odd dims 2^4 up
              store(a.k_new, pow2i(e), pow2i(e + 4), false);
              if (half == 0) {
                float* const p = reinterpret_cast<float*>(s_sc + st * 64) + (j >> 1) * 4 + (j & 1);
                p[0] = odd ? __int_as_float(0x7FC00000) : 0.f;  // rows that see such a value are NaN
                p[2] = pow2i(-24 - e);
                if (BIAS && in) s_pos[st * 64 + j] = a.row_pos ? a.row_pos[w.rq.n0 + j] : w.rq.ctx + j;
              }
            } else {
              uint32_t big = a.k_new ? row_max(a.v_new) : 0;
              const bool odd = big >= 0x7F800000u;
              if (odd) big = 0;
              const uint32_t most = __reduce_max_sync(0xffffffffu, big), least = __reduce_min_sync(0xffffffffu, big - 1u);
              if (lane == 0) s_vmax[dw] = make_uint2(most, least);
              bar_sync(1, 128);
              uint2 v = s_vmax[0];
#pragma unroll
              for (int i = 1; i < 4; i++) v = make_uint2(max(v.x, s_vmax[i].x), min(v.y, s_vmax[i].y));
              bar_sync(1, 128);
              const int E = tc_exponent(v.x);
              const bool apart = v.x && v.y + 1u + ((uint32_t)kt::kApart << 23) < v.x;
              const int e = apart ? tc_exponent(big) : E;
              if (apart && half == 0) s_e[st * 64 + j] = (float)e;
              store(a.v_new, pow2i(kt::kUp - e), pow2i(kt::kUp - e), odd);
              if (dt == 64) put_info(st, apart, m + kTcOwn, m >= 32 ? -1 : (1 << m) - 1,
                                     m >= 64 ? -1 : m > 32 ? (1 << (m - 32)) - 1 : 0, E);
            }
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&op_full[st]);
        }
      } while (w.next(a, sh));
  } else {
      // -------------------------------------------------------- softmax --
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(216 - S::kDecodeRegs));
      TcWalk<BIAS> w(a, sh);
      const int t = (warp - kt::kSoft) >> 2, st256 = tid - kt::kSoft * 32;
      const int idx = (warp & 3) * 32 + lane;                                // TMEM lane
      const uint32_t tb = tm + t * 256 + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes
      const float scale = BIAS ? 1.f : a.s.scale * kLog2e;
      uint32_t op0 = 0, par = 0;  // par: parity of the units done in either buffer
      do {
        const int h = w.head(), rc = w.s - h * w.rq.nc, n = w.ub - w.ua;
        const TcRowsOf<WIDE> rw(a.G * w.rq.m, w.rq.nc, rc);
        const int span = 128 / rw.copies;  // lanes of a copy
        TcRow x;
        {
          const int ridx = idx % span;
          const bool ok = ridx < rw.of(t);
          x.live = (ridx & ~31) < rw.of(t);
          x.key0 = idx / span * (64 / rw.copies);
          const int rho = rw.row(t, ridx), gq = rho / w.rq.m, node = rho - gq * w.rq.m;
          const int hq = h * a.G + gq;
          x.start = BIAS && a.s.start ? a.s.start[w.r] : INT32_MIN;
          x.slope = BIAS && a.s.slopes ? a.s.slopes[hq] : 0.f;
          x.qpos = a.row_pos ? a.row_pos[w.rq.n0 + node] : w.rq.ctx + node;
          x.anc = a.anc ? a.anc[w.rq.n0 + node] : (2ull << node) - 1;
          x.ref = -INFINITY;
          x.l = 0.f;
          x.any = false;
          const uint4* src = reinterpret_cast<const uint4*>(a.q + (int64_t)(w.rq.n0 + node) * a.q_stride + hq * D);
          uint4 v[D / 8];
#pragma unroll
          for (int i = 0; i < D / 8; i++) v[i] = ok ? src[i] : make_uint4(0, 0, 0, 0);
          float qs = 0.f, big = 0.f;
#pragma unroll
          for (int i = 0; i < D / 8; i++) {
            const uint32_t vs[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int k = 0; k < 4; k++) {
              const float f0 = __uint_as_float(vs[k] << 16), f1 = __uint_as_float(vs[k] & 0xFFFF0000u);
              qs += f0 + f1;
              big = fmaxf(big, fmaxf(fabsf(f0), fabsf(f1)));
            }
          }
          const int e = min(max(14 - expo(__float_as_uint(big)), -100), 100);
          const float up = pow2i(e), up4 = pow2i(e - 4);
          x.qsf = qs * pow2i(e - 24);
          x.fac = pow2i(24 - e) * scale;
          if (WIDE || t == 0) {
            uint8_t* const qt = sm + S::off_q + (WIDE ? t : 0) * S::kQ + idx * 128;
#pragma unroll
            for (int c = 0; c < D / 8; c++) {
              const uint32_t vs[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
              float f[8];
#pragma unroll
              for (int k = 0; k < 4; k++) {
                f[2 * k] = __uint_as_float(vs[k] << 16) * up;
                f[2 * k + 1] = __uint_as_float(vs[k] & 0xFFFF0000u) * up4;
              }
              *reinterpret_cast<uint4*>(qt + (c >> 3) * 16384 + (((c & 7) ^ (idx & 7)) << 4)) =
                  make_uint4(pack_f16x2(f[0], f[4]), pack_f16x2(f[1], f[5]), pack_f16x2(f[2], f[6]), pack_f16x2(f[3], f[7]));
            }
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0 && (WIDE || t == 0)) mbar_arrive(&q_full[t]);

        {
          auto run = [&](auto nc) {
            tc_softmax<D, BIAS, WIDE, decltype(nc)::value>(a, x, tb, WIDE ? 0 : t, n, op0, par, &s_full[2 * t], op_full, &p_full[2 * t],
                                                           &o_full[2 * t], s_sc, s_pos, s_e, s_info, &s_abort);
          };
          if (WIDE || rw.copies == 1) run(std::integral_constant<int, 64>());
          else if (rw.copies == 2) run(std::integral_constant<int, 32>());
          else run(std::integral_constant<int, 16>());
        }
        if (x.any) {
          // the last two products may be under way
          for (int b = 0; b < 2; b++) wait(&o_full[2 * t + b], (par >> b) ^ 1);
          tc_fence_after();
        }
        // Add up the copies, 32 dims at a time, and write the rows: the outputs
        // where the CTA has the whole segment, else a part.
        const bool whole = w.ua == 0 && w.ub == w.rq.nu;
        const int slot = 2 * blockIdx.x + (w.seg + w.ua > sh.u0 ? 1 : 0);
        float* part = a.part + (int64_t)slot * S::kPart;
        s_ml[t * 128 + idx] = x.live ? make_float2(x.ref, x.l) : make_float2(-INFINITY, 0.f);
        bar_sync(2, kt::kSoftThreads);
        auto lane_of = [&](int row, int j) {  // copy j of a row: [t][lane]
          if (WIDE) return row < rw.split ? row : 128 + row - rw.split;
          return j / rw.copies * 128 + j % rw.copies * span + row;
        };
        const int nsub = WIDE ? 1 : 2 * rw.copies;
        float f;  // of this thread's O: its weight in the row's sum
        {
          const int ridx = idx % span, row = ridx + (WIDE && t ? rw.split : 0);
          float M = -INFINITY, L = 0.f;
          if (ridx < rw.of(t)) {
#pragma unroll
            for (int j = 0; j < 8; j++)
              if (j < nsub) M = fmaxf(M, s_ml[lane_of(row, j)].x);
          }
          const float Ms = M == -INFINITY ? 0.f : M;
          f = x.any ? ex2(x.ref - Ms) * pow2i(-kt::kUp) : 0.f;
          if (ridx < rw.of(t) && (WIDE || idx + t * 128 == row)) {  // one thread a row
#pragma unroll
            for (int j = 0; j < 8; j++)
              if (j < nsub) {
                const float2 ml = s_ml[lane_of(row, j)];
                L = fmaf(ex2(ml.x - Ms), ml.y, L);
              }
            if (whole) {
              if (a.lse) {
                const int rho = rw.base + row, gq = rho / w.rq.m;
                a.lse[(int64_t)(w.rq.n0 + rho - gq * w.rq.m) * a.hq + h * a.G + gq] =
                    L == 0.f ? -INFINITY : (M - kt::kBase + log2f(L)) * (1.f / kLog2e);
              }
            } else {
              __stcg(reinterpret_cast<float2*>(part + kt::kRows * D) + row, make_float2(M - kt::kBase, L));
            }
            s_inv[row] = L == 0.f ? 0.f : 1.f / L;
          }
        }
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          if (x.live) {
            float* dst = s_x + (t * 128 + idx) * S::kX;
            float o[32];
            if (x.any) tmem_ld(tb + 128 + c, o);
#pragma unroll
            for (int e = 0; e < 32; e++) o[e] = x.any ? o[e] * f : 0.f;
#pragma unroll
            for (int e = 0; e < 32; e += 8) {  // columns hold dims 0 4 1 5 2 6 3 7 of each eight
              *reinterpret_cast<float4*>(dst + e) = make_float4(o[e], o[e + 2], o[e + 4], o[e + 6]);
              *reinterpret_cast<float4*>(dst + e + 4) = make_float4(o[e + 1], o[e + 3], o[e + 5], o[e + 7]);
            }
          }
          bar_sync(2, kt::kSoftThreads);
          for (int i = st256; i < rw.rows * 8; i += kt::kSoftThreads) {
            const int row = i >> 3, x4 = i & 7, d = c + x4 * 4;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int j = 0; j < 8; j++)
              if (j < nsub) {
                const float4 v = *reinterpret_cast<const float4*>(s_x + lane_of(row, j) * S::kX + x4 * 4);
                acc.x += v.x;
                acc.y += v.y;
                acc.z += v.z;
                acc.w += v.w;
              }
            if (whole) {
              const float inv = s_inv[row];
              const int rho = rw.base + row, gq = rho / w.rq.m;
              const int64_t at = (int64_t)(w.rq.n0 + rho - gq * w.rq.m) * a.hq + h * a.G + gq;
              *reinterpret_cast<uint2*>(a.out + at * D + d) =
                  make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
            } else {
              __stcg(reinterpret_cast<float4*>(part + row * D + d), acc);
            }
          }
          bar_sync(2, kt::kSoftThreads);
        }
        tc_fence_before();
        if (st256 == 0 && w.ua == 0) {
          const int last = sh.cta_of(w.seg + w.rq.nu - 1);
          a.joins[((int64_t)w.r * a.c.hkv + h) * kt::kJoins + rc] =
              make_int4(blockIdx.x, whole ? 0 : last - (int)blockIdx.x + 1, slot, 0);
        }
        op0 += n;
      } while (w.next(a, sh));
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kt::kMma) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
  }
}

// [joins of each (request, kv head)] [2 grid parts]
static size_t joins_bytes(int R, int hkv) { return ((size_t)R * hkv * kt::kJoins * sizeof(int4) + 255) / 256 * 256; }
size_t kv4_tc_workspace(int R, int hkv, int head_dim) {
  return joins_bytes(R, hkv) + (size_t)2 * num_sms() * kt::kRows * (head_dim + 2) * sizeof(float);
}

template <int D, bool WIDE>
static int launch_tc(Kv4AttnArgs a, int rows, int64_t units, bool bias, cudaStream_t st) {
  constexpr int smem = TcShape<D, WIDE>::smem;
  static const cudaError_t set[2] = {
      cudaFuncSetAttribute(k_kv4_attn_tc<D, false, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
      cudaFuncSetAttribute(k_kv4_attn_tc<D, true, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)};
  SD_CK(set[bias]);
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(num_sms(), units));
  a.joins = reinterpret_cast<int4*>(a.part);
  a.part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(a.part) + joins_bytes(a.R, a.c.hkv));
  (bias ? k_kv4_attn_tc<D, true, WIDE> : k_kv4_attn_tc<D, false, WIDE>)<<<(unsigned)grid, kt::kThreads, smem, st>>>(a);
  SD_CK(cudaGetLastError());
  SD_CK(launch(k_kv4_join<D, WIDE>, dim3((unsigned)(((int64_t)rows * a.hq + 7) / 8)), dim3(256), 0, st, true, a, rows));
  return SD_OK;
}

int kv4_launch_attn_tc(const Kv4AttnArgs& a, int head_dim, int rows, int most, int64_t units, bool bias,
                       cudaStream_t st) {
  if (head_dim == 128)
    return most > 128 ? launch_tc<128, true>(a, rows, units, bias, st) : launch_tc<128, false>(a, rows, units, bias, st);
  return most > 128 ? launch_tc<64, true>(a, rows, units, bias, st) : launch_tc<64, false>(a, rows, units, bias, st);
}

}  // namespace sdv
