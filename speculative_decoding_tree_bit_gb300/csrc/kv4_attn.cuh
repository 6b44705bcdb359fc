// Attention over the 4-bit cache: what its kernels share.
#pragma once

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
  int32_t* tickets;  // [grid], zero between calls (warp kernel)
  float* part;       // [2 grid][rows of a tile][D + 2]
  int4* joins;       // [R][hkv][kJoins]: where a segment's parts lie (tensor-core kernel)
};

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Scores in base 2 from q.k: scale and cap, pairs at a time.  cap tanh(x / cap):
// by tanh's Taylor series to x^9 while every x of the warp is below 0.3 (off by
// 1.6e-8 there; scores far below the cap are the rule), else as 1 - 2 / (1 +
// e^2x), off by 1.2e-7 of the cap.  One branch for all N values, by whole warps.
template <int N>
__device__ __forceinline__ void kv4_cap(const Kv4Score& s, float (&t)[N]) {
  if (s.cap > 0.f) {
    const float in = __fdividef(s.scale, s.cap), out = s.cap * kLog2e;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      f2unpack(f2mul(f2pack(t[i], t[i + 1]), f2pack(in, in)), t[i], t[i + 1]);
      top = fmaxf(top, fmaxf(fabsf(t[i]), fabsf(t[i + 1])));
    }
    auto series = [&](int i, float& a, float& b) {
      const uint64_t x = f2pack(t[i], t[i + 1]), u = f2mul(x, x), z = f2mul(x, f2pack(out, out));
      uint64_t q = f2fma(u, f2pack(62.f / 2835.f, 62.f / 2835.f), f2pack(-17.f / 315.f, -17.f / 315.f));
      q = f2fma(q, u, f2pack(2.f / 15.f, 2.f / 15.f));
      q = f2fma(q, u, f2pack(-1.f / 3.f, -1.f / 3.f));
      f2unpack(f2fma(f2mul(q, u), z, z), a, b);
    };
    if (!__any_sync(0xffffffffu, top >= 0.3f)) {
#pragma unroll
      for (int i = 0; i < N; i += 2) series(i, t[i], t[i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        float w[2];
        series(i, w[0], w[1]);
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const float y = fmaf(-2.f * out, __fdividef(1.f, 1.f + ex2(2.f * kLog2e * t[i + e])), out);
          t[i + e] = fabsf(t[i + e]) < 0.3f ? w[e] : y;
        }
      }
    }
  } else {
    const float f = s.scale * kLog2e;
#pragma unroll
    for (int i = 0; i < N; i += 2) f2unpack(f2mul(f2pack(t[i], t[i + 1]), f2pack(f, f)), t[i], t[i + 1]);
  }
}

// A row's slope and masks over N keys; pos(i): position of key i.
template <int N, typename Pos>
__device__ __forceinline__ void kv4_bias(const Kv4Score& s, float (&t)[N], float slope, int q_pos, int start, Pos pos) {
  if (s.slopes) {
#pragma unroll
    for (int i = 0; i < N; i++) t[i] = fmaf(slope * kLog2e, (float)(pos(i) - q_pos), t[i]);
  }
  if (s.window > 0 || s.start) {
    const int64_t since = (int64_t)q_pos - (s.window > 0 ? s.window : INT32_MAX);
    const int first = (int)max(since + 1, (int64_t)start);  // the least position seen
#pragma unroll
    for (int i = 0; i < N; i++)
      if (pos(i) < first) t[i] = -INFINITY;
  }
}

// A bounded wait that looks at the clock and at the other warps' abort flag
// only every so many tries: a try suspends the warp for a while by itself, and
// reading the clock costs more than a wake-up.
__device__ __forceinline__ bool kv4_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint32_t addr = smem_u32(bar);
  for (int i = 0; i < 64; i++)
    if (mbar_try_wait(addr, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (;;) {
    for (int i = 0; i < 64; i++)
      if (mbar_try_wait(addr, parity)) return true;
    if (*abort) return false;
    if (globaltimer() - t0 > kWaitLimitNs) {
      *abort = 1;
      return false;
    }
  }
}

// 8x8 transpose of 16-bit values across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// The four nibbles of each 16-bit half of w as fp16 pairs, from two words (w
// and w >> 8) and two masks: nibble i even lies at bits 0..3 and reads as the
// subnormal code 2^-24, i odd at bits 4..7 and reads as code 2^-20.
template <int I>
__device__ __forceinline__ uint32_t codes2(uint32_t w) {
  return (I < 2 ? w : w >> 8) & (I & 1 ? 0x00F000F0u : 0x000F000Fu);
}
// (code - 8) 2^-9 of the same pair: one fused multiply-add, exact.
template <int I>
__device__ __forceinline__ uint32_t centred2(uint32_t w) {
  uint32_t y;
  // 2^15 or 2^11, and -8 2^-9
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(codes2<I>(w)), "r"(I & 1 ? 0x68006800u : 0x78007800u), "r"(0xA400A400u));
  return y;
}
__device__ __forceinline__ void mma_f16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t y;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
  return y;
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// What a call's requests hold, as the attention kernels split them: a request
// is hkv x nc segments (kv head, tile of RT rows) of nu units each: the rows'
// own keys in `no` runs of 32 GU, then the groups of 32 cached slots from group
// g0 on, GU a unit; at least one unit, so that a row that sees nothing is
// written too.
struct Kv4Req {
  int n0, m, ctx, g0, no, nu, nc;
};

// A request's rows alone: n0, m and nc.
template <int RT>
__device__ __forceinline__ Kv4Req kv4_req_rows(const Kv4AttnArgs& a, int r) {
  Kv4Req q = {};
  q.n0 = a.cu[r];
  q.m = min(max(a.cu[r + 1] - q.n0, 0), 64);
  q.nc = (a.G * q.m + RT - 1) / RT;
  return q;
}

// BIAS: the call has scoring options.  LANE: by a lane for a request of its
// own, else by a whole warp for one.
template <int RT, int GU, bool BIAS, bool LANE = false>
__device__ __forceinline__ Kv4Req kv4_req(const Kv4AttnArgs& a, int r) {
  Kv4Req q = kv4_req_rows<RT>(a, r);
  int ctx = a.c.ctx_len[r];
  if (ctx < 0 || ctx > a.c.cap) {
    set_status(a.status, SD_ERR_CAPACITY);
    ctx = ctx < 0 ? 0 : (int)a.c.cap;
  }
  q.ctx = ctx;
  int first = 0;
  if (BIAS && (a.s.window > 0 || a.s.start)) {
    const int p0 = a.row_pos && q.m ? a.row_pos[q.n0] : ctx;
    first = LANE ? kv4_first_lane(a.c, a.s, r, ctx, p0) : kv4_first(a.c, a.s, r, ctx, p0);
  }
  q.g0 = first / kKvGroup;
  q.no = a.k_new ? (q.m + 32 * GU - 1) / (32 * GU) : 0;
  q.nu = q.no + (ctx > first ? ((ctx - 1) / kKvGroup - q.g0 + GU) / GU : 0);
  if (q.nu == 0) q.no = q.nu = 1;  // an empty run
  return q;
}

// A CTA's share of a call's units: U over C CTAs, the first `more` of them one
// more than `each`; [u0, u1), beginning in segment s0 (first unit seg0) of
// request r0.
struct Kv4Share {
  int r0, s0, seg0, u0, u1, each, more;
  Kv4Req rq;  // of request r0
  __device__ __forceinline__ int first(int c) const { return c * each + min(c, more); }
  __device__ __forceinline__ int cta_of(int u) const {
    const int big = more * (each + 1);
    return u < big ? u / (each + 1) : more + (u - big) / each;
  }
};

// By one warp, into shared memory.  With less work than 2 `width` units a CTA,
// a CTA takes whole segments, or even parts of one of about `width` units, so
// that fewer parts are joined; else every CTA takes its part.  Measured with
// the warp kernel (width 4 units a warp, against 1): one request of 2000
// keys, 8 / 32 rows a kv head: 14 / 20 us against 18 / 31; a tree of 16 over
// 2048 keys with its own keys: 29 against 27.
template <int RT, int GU, bool BIAS>
__device__ __forceinline__ void kv4_share(const Kv4AttnArgs& a, int width, Kv4Share& sh) {
  const int lane = threadIdx.x & 31;
  int U = 0, segs = 0, lo = 0;
  Kv4Req rq = {};
  for (int base = 0; base < a.R; base += 32) {
    rq = {};
    if (base + lane < a.R) rq = kv4_req<RT, GU, BIAS, true>(a, base + lane);
    const int n = a.c.hkv * rq.nc * rq.nu;
    int run = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += v;
    }
    lo = U + run - n;
    U += __shfl_sync(0xffffffffu, run, 31);
    segs += __reduce_add_sync(0xffffffffu, a.c.hkv * rq.nc);
  }
  int C = gridDim.x;
  if (U < C * width * 2) C = min(C, segs * ((U + segs * width - 1) / max(1, segs * width)));
  C = max(C, 1);
  const int each = U / C, more = U - each * C;
  const int u0 = (int)blockIdx.x < C ? (int)blockIdx.x * each + min((int)blockIdx.x, more) : U;
  const int u1 = (int)blockIdx.x < C ? u0 + each + ((int)blockIdx.x < more) : U;
  if (u0 < u1) {
    int before = 0;
    for (int base = 0; base < a.R; base += 32) {
      if (a.R > 32) {
        rq = {};
        if (base + lane < a.R) rq = kv4_req<RT, GU, BIAS, true>(a, base + lane);
        const int n = a.c.hkv * rq.nc * rq.nu;
        int run = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, run, o);
          if (lane >= o) run += v;
        }
        lo = before + run - n;
        before += __shfl_sync(0xffffffffu, run, 31);
      }
      if (u0 >= lo && u0 < lo + a.c.hkv * rq.nc * rq.nu) {
        sh.r0 = base + lane;
        sh.rq = rq;
        sh.s0 = (u0 - lo) / rq.nu;
        sh.seg0 = lo + (u0 - lo) / rq.nu * rq.nu;
      }
      if (before > u0) break;
    }
  }
  if (lane == 0) {
    sh.u0 = u0;
    sh.u1 = u1;
    sh.each = each;
    sh.more = more;
  }
}

// Many rows a kv head (kv4_attn_tc.cu).
size_t kv4_tc_workspace(int R, int hkv, int head_dim);
int kv4_launch_attn_tc(const Kv4AttnArgs& a, int head_dim, int rows, int most, int64_t units, bool bias,
                       cudaStream_t st);

}  // namespace sdv
