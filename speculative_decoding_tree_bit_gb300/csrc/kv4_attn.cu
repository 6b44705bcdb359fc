// Attention over the 4-bit cache, and the weight its keys collect.
#include <algorithm>

#include "kv4_attn.cuh"

namespace sdv {

// ------------------------------------------------ attention, warp MMA --
//
// Scores and outputs are computed transposed, S^T = K Q^T and O^T = V^T P^T,
// with mma.m16n8k16: the codes are the 16-row A side, the query rows the
// 8-wide B side, so that the few rows of a decode step (the heads of a group)
// fill half or all of a tile.
//
// What bounds it is not the bytes alone but the integer pipe, at 2 cycles a
// warp instruction, that makes operands of the nibbles: 4 bits of a 16-bit
// lane are read in place as an fp16 subnormal (code 2^-24, or 2^-20 for the
// odd nibbles, whose 2^-4 is in the queries), so eight codes cost four masks
// and one shift.  K's codes enter as they are, 0..15: score = s (c.q) +
// (m - 8 s) sum(q).  V's are centred by a fused multiply-add on the other pipe
// (a sum over many keys would lose what the offset 8 sum(p s) cancels):
// output = sum (p s)(c - 8) + sum p m.  Queries are bf16, exact in fp16 after
// a power of two that brings a row's greatest value below 2^15 (values
// 2^-27 of it and less lose bits).  A weight p s enters as one fp16 term
// with 11 bits, 2^-12 of its value against the 2^-9 of the output's own
// rounding.  p's reference follows the row's scores plus the exponents of the
// values that it sees (a unit's greatest for all of its keys where they are
// within 2^6), so weights down to 2^-16 of the row's greatest keep their bits,
// down to 2^-26 count, and no value that a row does not see moves them.  The
// rows' own keys and values are bf16 products, their weights two bf16 terms.
//
// A warp works on its own: it takes every W-th unit of the CTA's segment, and
// keeps a ring of two 32-slot records, one bulk copy each, filled a unit
// ahead; the next segment's first two are on their way while a segment is
// joined.  Running maxima are per warp; the warps' parts are joined in shared
// memory at the segment's end, the CTAs' parts of a segment in global memory
// by the last CTA to finish, in CTA order (the same bits every time).  The
// segments' units are dealt evenly over the CTAs, whatever the requests'
// lengths; two CTAs an SM, so that one works while the other joins.
//
// Measured, 32 query and 8 kv heads, D = 128: 32 tokens over 1500 to 8192 keys 50
// us, 3.4 TB/s (the ALU pipe 51% busy, issue 53%); 32 chains of 8 rows over 1024
// to 4096 keys with a cap 90 us, 106 TFLOP/s (two tiles of rows a warp, six warps;
// four tiles, four warps: 135 where two took 110); a tree of 16 over 2048 keys 25
// us, most of it latency.

constexpr int kMaxCtas = 512;
constexpr float kUnset = 3e38f;  // a row's reference before it sees a key

template <int D, int NT, int W>
struct AttnShape {
  static constexpr int RT = 8 * NT;
  static constexpr int kStage = kv4_rec(D) + 128;
  static constexpr int kPairs = D / 2 + 2;                       // float pairs of a row of a warp's output
  static constexpr int off_o = W * 2 * kStage;                   // [W][RT][kPairs] float pairs
  static constexpr int off_q = off_o + W * RT * kPairs * 8;           // [NT][D/32][32] uint4: fp16 queries, two k-steps each
  static constexpr int off_qb = off_q + NT * (D / 16) * 32 * 8;  // the same, bf16
  static constexpr int off_anc = off_qb + NT * (D / 16) * 32 * 8;  // [RT] u64
  static constexpr int off_bar = off_anc + RT * 8;               // [W][2]
  static constexpr int off_ml = off_bar + W * 2 * 8;             // [2][W][RT]
  static constexpr int off_row = off_ml + 2 * W * RT * 4;        // qsum, factor, slope, pos, L [RT] each
  static constexpr int off_ok = off_row + 5 * RT * 4;            // [W][2]
  static constexpr int smem = off_ok + W * 2 * 4;
};

// A segment to join at a CTA's end: n parts (0: none) from CTA c0 on.
struct Kv4Join {
  int seg, n, c0, n0, m, h, rc;
};

template <int D, int NT, int W, bool BIAS>
__global__ void __launch_bounds__(W * 32, 2) k_kv4_attn(const __grid_constant__ Kv4AttnArgs a) {
  using S = AttnShape<D, NT, W>;
  constexpr int RT = S::RT;
  constexpr int KK = D / 16;  // k-steps of a score, and 16-dim tiles of an output
  extern __shared__ __align__(128) uint8_t sm[];
  float* s_o = reinterpret_cast<float*>(sm + S::off_o);
  uint4* s_q = reinterpret_cast<uint4*>(sm + S::off_q);
  uint4* s_qb = reinterpret_cast<uint4*>(sm + S::off_qb);
  uint64_t* s_anc = reinterpret_cast<uint64_t*>(sm + S::off_anc);
  uint64_t* s_bar = reinterpret_cast<uint64_t*>(sm + S::off_bar);
  float* s_m = reinterpret_cast<float*>(sm + S::off_ml);
  float* s_l = s_m + W * RT;
  float* s_qs = reinterpret_cast<float*>(sm + S::off_row);
  float* s_fac = s_qs + RT;
  float* s_slope = s_fac + RT;
  int* s_pos = reinterpret_cast<int*>(s_slope + RT);
  float* s_L = reinterpret_cast<float*>(s_pos + RT);
  int* s_ok = reinterpret_cast<int*>(sm + S::off_ok);
  __shared__ int s_abort;
  __shared__ Kv4Share sh;
  __shared__ Kv4Join s_join[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;

  if (warp == 0) kv4_share<RT, 1, BIAS>(a, 4 * W, sh);  // at least four units a warp while there is less than that a CTA
  if (tid == 0) {
    s_abort = 0;
    s_join[0] = s_join[1] = Kv4Join{};
  }
  if (lane == 0) {
    mbar_init(&s_bar[warp * 2], 1);
    mbar_init(&s_bar[warp * 2 + 1], 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (sh.u0 >= sh.u1) return;

  uint64_t* const bar = s_bar + warp * 2;
  uint8_t* const ring = sm + warp * 2 * S::kStage;
  uint32_t used = 0;  // records this warp has taken from its ring

  // the segment at hand: unit range [ua, ub), of which the units from no on are
  // records.  A lane holds the address of every 32nd of the warp's records.
  int r = sh.r0, s = sh.s0, seg = sh.seg0;
  const int u0 = sh.u0, u1 = sh.u1;
  Kv4Req rq = BIAS && NT == 1 ? sh.rq : kv4_req<RT, 1, BIAS>(a, r);  // short calls wait for the window's check once
  int ua = u0 - seg, ub = min(rq.nu, u1 - seg);
  const uint8_t* addr;
  auto first_record = [&]() {  // the first of the segment's records that falls to this warp
    return ua + warp + (rq.no - ua - warp > 0 ? (rq.no - ua - warp + W - 1) / W * W : 0);
  };
  auto look_up = [&](int u) {  // u: the warp's unit that lane 0 stands for
    const int x = u + lane * W;
    addr = x < ub ? a.c.record(D, r, s / rq.nc, rq.g0 + x - rq.no) : nullptr;
  };
  auto issue = [&](int u, int k, int stage) {  // k: the lane that holds unit u's address
    const uint8_t* rec = reinterpret_cast<const uint8_t*>(
        __shfl_sync(0xffffffffu, (unsigned long long)reinterpret_cast<uintptr_t>(addr), k));
    if (lane == 0) {
      s_ok[warp * 2 + stage] = rec != nullptr;
      if (rec) {
        uint8_t* dst = ring + stage * S::kStage;
        mbar_arrive_expect_tx(&bar[stage], kv4_rec(D) + (BIAS ? 128 : 0));
        bulk_g2s(dst, rec, kv4_rec(D), &bar[stage]);
        if (BIAS) bulk_g2s(dst + kv4_rec(D), a.c.pos + a.c.slot0(r, s / rq.nc) + (rq.g0 + u - rq.no) * kKvGroup, 128, &bar[stage]);
      } else {
        set_status(a.status, SD_ERR_CAPACITY);
        mbar_arrive(&bar[stage]);
      }
    }
    __syncwarp();
  };
  auto begin = [&]() {
    const int u = first_record();
    if (u < ub) {
      look_up(u);
      issue(u, 0, used & 1);
      if (u + W < ub) issue(u + W, 1, (used + 1) & 1);
    }
  };
  const int e0 = q >> 1;  // which of a key pair this lane reads first (bank spread)
  const uint32_t sel_lo = e0 ? 0x1054u : 0x5410u, sel_hi = e0 ? 0x3276u : 0x7632u;
  const float sc2 = BIAS ? 1.f : a.s.scale * kLog2e;

  for (bool first = true;; first = false) {
    const int h = s / rq.nc, rc = s - h * rq.nc;
    const int rows = min(RT, a.G * rq.m - rc * RT);
    const int start = BIAS && a.s.start ? a.s.start[r] : INT32_MIN;

    // the own rows' lines on their way to the L2 while the queries are read
    if (a.k_new && ua < rq.no)
      for (int i = tid; i < rq.m * (D / 64); i += W * 32) {
        const int64_t at = (int64_t)(rq.n0 + i / (D / 64)) * a.kv_stride + h * D + i % (D / 64) * 64;
        prefetch_l2(a.k_new + at);
        prefetch_l2(a.v_new + at);
      }
    // the tile's query rows as B fragments; dims are taken in the order the
    // codes' nibbles give them
    if (first && tid / 32 * 32 >= RT * (D / 8)) begin();
    for (int i = tid; i < RT * (D / 8); i += W * 32) {
      const int row = i / (D / 8), oct = i % (D / 8);
      const int rho = rc * RT + row;
      const bool ok = row < rows;
      const int node = ok ? rho % rq.m : 0, hq = h * a.G + (ok ? rho / rq.m : 0);
      uint4 x = make_uint4(0, 0, 0, 0);
      if (ok) x = *reinterpret_cast<const uint4*>(a.q + (int64_t)(rq.n0 + node) * a.q_stride + hq * D + oct * 8);
      uint64_t anc = ok ? (2ull << node) - 1 : 0;
      int pos = rq.ctx + node;
      float slope = 0.f;
      if (oct == 0) {
        if (ok && a.anc) anc = a.anc[rq.n0 + node];
        if (BIAS && a.row_pos) pos = a.row_pos[rq.n0 + node];
        if (BIAS && a.s.slopes) slope = a.s.slopes[hq];
      }
      if (first && i == tid) begin();  // behind the queries' own loads
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
      float f[8], qs = 0.f, big = 0.f;
#pragma unroll
      for (int k = 0; k < 8; k++) {
        f[k] = bf2f((uint16_t)(xs[k >> 1] >> (16 * (k & 1))));
        qs += f[k];
        big = fmaxf(big, fabsf(f[k]));
      }
#pragma unroll
      for (int o = D / 16; o > 0; o >>= 1) {
        qs += __shfl_xor_sync(0xffffffffu, qs, o);
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      }
      // 2^e brings the row's greatest value into [2^14, 2^15)
      const int e = min(max(14 + 127 - (int)(__float_as_uint(big) >> 23), -100), 100);
      const float up = pow2i(e), up4 = pow2i(e - 4);
      const int ql = oct / (D / 32), j = oct % (D / 32);
      const int at = ((row >> 3) * (KK / 2) + j) * 32 + 4 * (row & 7) + ql;
      s_q[at] = make_uint4(pack_f16x2(f[0] * up, f[4] * up), pack_f16x2(f[1] * up4, f[5] * up4),
                           pack_f16x2(f[2] * up, f[6] * up), pack_f16x2(f[3] * up4, f[7] * up4));
      s_qb[at] = make_uint4(prmt(x.x, x.z, 0x5410), prmt(x.x, x.z, 0x7632), prmt(x.y, x.w, 0x5410),
                            prmt(x.y, x.w, 0x7632));
      if (oct == 0) {
        s_qs[row] = qs * sc2;
        s_fac[row] = pow2i(24 - e) * sc2;
        s_slope[row] = slope;
        s_pos[row] = pos;
        s_anc[row] = anc;
      }
    }
    __syncthreads();
    // Of a lane's two rows: l, mv, o are sums of p = 2^(x + ref), p m and p s (c -
    // 8) 2^-9 over the keys so far, x their scores.  11 - ref is the greatest x
    // + E so far, give or take: a value row's magnitudes lie below 2^(E + 1).  One
    // reference for all three, so that p s fits fp16 and only what a row sees moves it
    float o[NT][KK][4];
    uint64_t l[NT], mv[NT], fac[NT], qs[NT], ref[NT];
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
#pragma unroll
      for (int t = 0; t < KK; t++) o[nt][t][0] = o[nt][t][1] = o[nt][t][2] = o[nt][t][3] = 0.f;
      ref[nt] = f2pack(kUnset, kUnset);
      l[nt] = mv[nt] = 0;
      fac[nt] = f2pack(s_fac[nt * 8 + 2 * q], s_fac[nt * 8 + 2 * q + 1]);
      qs[nt] = f2pack(s_qs[nt * 8 + 2 * q], s_qs[nt * 8 + 2 * q + 1]);
    }

    float sc[2][NT][4];  // scores (base 2) of keys 16 i + g, 16 i + g + 8
    // p s < 2^(x + E + ref - 2) has to stay below 2^15: a lane's greatest x + E
    // past 17 - ref, anywhere in the warp, rescales what it has so far
    auto over = [&](const float (&top)[NT][2], float ev) {
      bool any = false;
#pragma unroll
      for (int nt = 0; nt < NT; nt++) {
        float r0, r1;
        f2unpack(ref[nt], r0, r1);
        any |= top[nt][0] + r0 > 17.f - ev || top[nt][1] + r1 > 17.f - ev;
      }
      return __any_sync(0xffffffffu, any) != 0;
    };
    auto grow = [&](const float (&top)[NT][2]) {  // top: a lane's greatest x + E
#pragma unroll
      for (int nt = 0; nt < NT; nt++) {
        float al[2], r[2];
        f2unpack(ref[nt], r[0], r[1]);
#pragma unroll
        for (int e = 0; e < 2; e++) {
          float t = top[nt][e];
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
          const float rn = fminf(r[e], 11.f - t);
          al[e] = ex2(rn - r[e]);
          r[e] = rn;
        }
        const uint64_t al2 = f2pack(al[0], al[1]);
        ref[nt] = f2pack(r[0], r[1]);
        l[nt] = f2mul(l[nt], al2);
        mv[nt] = f2mul(mv[nt], al2);
#pragma unroll
        for (int t = 0; t < KK; t++) {
          o[nt][t][0] *= al[0];
          o[nt][t][1] *= al[1];
          o[nt][t][2] *= al[0];
          o[nt][t][3] *= al[1];
        }
      }
    };
    auto exponent = [](float x) { return fmaxf((float)((int)(__float_as_uint(x) >> 23) - 127), -90.f); };  // of x >= 0

    // the rows' own keys, in runs of 32, 16 at a time
    for (int u = ua + warp; u < min(ub, rq.no); u += W)
#pragma unroll 1
      for (int j0 = u * 32; j0 < min(u * 32 + 32, a.k_new ? rq.m : 0); j0 += 16) {
        float so[NT][4];  // scores, then weights, of keys g and g + 8
        const int ja = j0 + g, jb = ja + 8;
#pragma unroll
        for (int nt = 0; nt < NT; nt++) so[nt][0] = so[nt][1] = so[nt][2] = so[nt][3] = 0.f;
        {
          const uint16_t* kn = a.k_new + (int64_t)rq.n0 * a.kv_stride + h * D + q * (D / 4);
          const uint16_t* pa = kn + (ja < rq.m ? ja : 0) * a.kv_stride;
          const uint16_t* pb = kn + (jb < rq.m ? jb : 0) * a.kv_stride;
#pragma unroll
          for (int j = 0; j < D / 32; j++) {
            const uint4 xa = *reinterpret_cast<const uint4*>(pa + 8 * j), xb = *reinterpret_cast<const uint4*>(pb + 8 * j);
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
              const uint4 b = s_qb[(nt * (KK / 2) + j) * 32 + lane];
              mma_bf16(so[nt], prmt(xa.x, xa.z, 0x5410), prmt(xb.x, xb.z, 0x5410), prmt(xa.x, xa.z, 0x7632),
                       prmt(xb.x, xb.z, 0x7632), b.x, b.y);
              mma_bf16(so[nt], prmt(xa.y, xa.w, 0x5410), prmt(xb.y, xb.w, 0x5410), prmt(xa.y, xa.w, 0x7632),
                       prmt(xb.y, xb.w, 0x7632), b.z, b.w);
            }
          }
        }
        float top[NT][2];
        uint32_t seen = 0;  // scores that count
        const int kpa = BIAS && ja < rq.m ? (a.row_pos ? a.row_pos[rq.n0 + ja] : rq.ctx + ja) : 0;
        const int kpb = BIAS && jb < rq.m ? (a.row_pos ? a.row_pos[rq.n0 + jb] : rq.ctx + jb) : 0;
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const int row = nt * 8 + 2 * q + e;
            const uint64_t anc = s_anc[row];
            float ta = so[nt][e] * sc2, tb = so[nt][2 + e] * sc2;
            if (BIAS) {
              float tt[2] = {ta, tb};
              kv4_cap(a.s, tt);
              kv4_bias(a.s, tt, s_slope[row], s_pos[row], start, [&](int i) { return i ? kpb : kpa; });
              ta = tt[0], tb = tt[1];
            }
            so[nt][e] = ja < rq.m && (anc >> ja & 1) ? ta : -INFINITY;
            so[nt][2 + e] = jb < rq.m && (anc >> jb & 1) ? tb : -INFINITY;
            seen |= (uint32_t)(so[nt][e] != -INFINITY) << (4 * nt + e) | (uint32_t)(so[nt][2 + e] != -INFINITY) << (4 * nt + 2 + e);
            top[nt][e] = fmaxf(so[nt][e], so[nt][2 + e]);
          }
        if (over(top, 0.f)) grow(top);  // E counted as 0
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
          for (int i = 0; i < 2; i++) {
            float p[2], w0, w1;
            f2unpack(f2add(f2pack(so[nt][2 * i], so[nt][2 * i + 1]), ref[nt]), p[0], p[1]);
            const uint64_t pp = f2pack(ex2(p[0]), ex2(p[1]));
            l[nt] = f2add(l[nt], pp);
            f2unpack(f2mul(pp, f2pack(1.f / 512.f, 1.f / 512.f)), w0, w1);
            const uint32_t hi = pack_bf16x2(w0, w1);
            const uint32_t lo = pack_bf16x2(w0 - __uint_as_float(hi << 16), w1 - __uint_as_float(hi & 0xFFFF0000u));
            ph[nt][i] = transpose8(hi);
            pl[nt][i] = transpose8(lo);
          }
        // A product with a weight of 0 would carry a NaN or an infinity of a
        // row's values to rows that do not see it: such a row counts as NaN in
        // every dim, 0 here, and makes NaN the sums of the rows that see it
        const uint16_t* vn = a.v_new + (int64_t)rq.n0 * a.kv_stride + h * D + g * (D / 8);
        uint32_t odd[4];
#pragma unroll
        for (int b = 0; b < 4; b++) {
          const int kx = j0 + 8 * (b >> 1) + 2 * q + (b & 1);
          uint32_t any = 0;
#pragma unroll
          for (int c = 0; c < D / 64; c++) {
            const uint4 x = *reinterpret_cast<const uint4*>(vn + (kx < rq.m ? kx : 0) * a.kv_stride + 8 * c);
            any |= ((x.x & 0x7F807F80u) + 0x00800080u) | ((x.y & 0x7F807F80u) + 0x00800080u) |
                   ((x.z & 0x7F807F80u) + 0x00800080u) | ((x.w & 0x7F807F80u) + 0x00800080u);
          }
          odd[b] = __ballot_sync(0xffffffffu, (any & 0x80008000u) != 0);
        }
        if (odd[0] | odd[1] | odd[2] | odd[3]) {
#pragma unroll
          for (int i = 0; i < 2; i++) {
            const int j = j0 + 8 * i + g;
            const bool bad = j < rq.m && ((g & 1 ? odd[2 * i + 1] : odd[2 * i]) >> (g >> 1) & 0x11111111u);
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
              const float x = __int_as_float(0x7FC00000);
              const bool s0 = seen >> (4 * nt + 2 * i) & 1, s1 = seen >> (4 * nt + 2 * i + 1) & 1;
              if (bad) l[nt] = f2add(l[nt], f2pack(s0 ? x : 0.f, s1 ? x : 0.f));
            }
          }
        }
#pragma unroll
        for (int c = 0; c < D / 64; c++) {
          uint32_t x[4][4];
#pragma unroll
          for (int b = 0; b < 4; b++) {
            const int kx = j0 + 8 * (b >> 1) + 2 * q + (b & 1);
            const bool bad = odd[b] >> q & 0x11111111u;
            const uint4 v = *reinterpret_cast<const uint4*>(vn + (kx < rq.m ? kx : 0) * a.kv_stride + 8 * c);
            x[b][0] = bad ? 0u : v.x, x[b][1] = bad ? 0u : v.y, x[b][2] = bad ? 0u : v.z, x[b][3] = bad ? 0u : v.w;
          }
#pragma unroll
          for (int t = 0; t < 4; t++) {
            const uint32_t f0 = prmt(x[0][t], x[1][t], 0x5410), f1 = prmt(x[0][t], x[1][t], 0x7632),
                           f2 = prmt(x[2][t], x[3][t], 0x5410), f3 = prmt(x[2][t], x[3][t], 0x7632);
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
              mma_bf16(o[nt][4 * c + t], f0, f1, f2, f3, ph[nt][0], ph[nt][1]);
              mma_bf16(o[nt][4 * c + t], f0, f1, f2, f3, pl[nt][0], pl[nt][1]);
            }
          }
        }
      }

    // The own rows' E was counted as 0.  Where all of a row's sums are small (two
    // of its tiles mostly say that they are not), its reference goes up again
    if (a.k_new && ua + warp < min(ub, rq.no)) {
      uint32_t fine = 15;
#pragma unroll
      for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const float big = fmaxf(fmaxf(fabsf(o[nt][0][e]), fabsf(o[nt][0][2 + e])), fmaxf(fabsf(o[nt][1][e]), fabsf(o[nt][1][2 + e])));
          const bool none = __uint_as_float((uint32_t)(ref[nt] >> (32 * e))) == kUnset;  // a row that sees no own key
          uint32_t rows = __ballot_sync(0xffffffffu, big > 0.0625f || none);
          rows |= rows >> 16;
          rows |= rows >> 8;
          fine &= rows | rows >> 4;
        }
      if (fine != 15) {
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
          float up[2];
#pragma unroll
          for (int e = 0; e < 2; e++) {
            float big = 0.f;
#pragma unroll
            for (int t = 0; t < KK; t++) big = fmaxf(big, fmaxf(fabsf(o[nt][t][e]), fabsf(o[nt][t][2 + e])));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 4));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 8));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 16));
            up[e] = fmaxf(-exponent(big), 0.f);
          }
          float r0, r1;
          f2unpack(ref[nt], r0, r1);
          ref[nt] = f2pack(r0 + up[0], r1 + up[1]);
          up[0] = ex2(up[0]);
          up[1] = ex2(up[1]);
          l[nt] = f2mul(l[nt], f2pack(up[0], up[1]));
#pragma unroll
          for (int t = 0; t < KK; t++) {
            o[nt][t][0] *= up[0];
            o[nt][t][1] *= up[1];
            o[nt][t][2] *= up[0];
            o[nt][t][3] *= up[1];
          }
        }
      }
    }

    int k = 0;
    for (int u = first_record(); u < ub; u += W) {
      const int stage = used & 1;
      const uint8_t* st = ring + stage * S::kStage;
      if (!kv4_wait(&bar[stage], (used >> 1) & 1, &s_abort)) set_status(a.status, SD_TIMEOUT_AT(30));
      // K: lane (g, q) holds dims q D/4 .. of keys g and g + 8 of a 16-key tile
#pragma unroll
      for (int i = 0; i < 2; i++) {
        uint32_t kw[2][D / 32];
#pragma unroll
        for (int b = 0; b < 2; b++) {
          const uint8_t* p = st + (16 * i + 8 * b + g) * (D / 2) + q * (D / 8);
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            kw[b][0] = v.x, kw[b][1] = v.y, kw[b][2] = v.z, kw[b][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            kw[b][0] = v.x, kw[b][1] = v.y;
          }
        }
        float s2[4] = {0.f, 0.f, 0.f, 0.f};  // a second chain of sums, for one tile of rows alone
#pragma unroll
        for (int nt = 0; nt < NT; nt++) sc[i][nt][0] = sc[i][nt][1] = sc[i][nt][2] = sc[i][nt][3] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 32; j++) {
          const uint32_t wa = kw[0][j], wb = kw[1][j];
#pragma unroll
          for (int nt = 0; nt < NT; nt++) {
            const uint4 b = s_q[(nt * (KK / 2) + j) * 32 + lane];
            mma_f16(sc[i][nt], codes2<0>(wa), codes2<0>(wb), codes2<1>(wa), codes2<1>(wb), b.x, b.y);
            mma_f16(NT == 1 ? s2 : sc[i][nt], codes2<2>(wa), codes2<2>(wb), codes2<3>(wa), codes2<3>(wb), b.z, b.w);
          }
        }
        if (NT == 1)
#pragma unroll
          for (int e = 0; e < 4; e++) sc[i][0][e] += s2[e];
      }
      // slots of this record that the request holds
      const int lim = s_ok[warp * 2 + stage] ? rq.ctx - (rq.g0 + u - rq.no) * kKvGroup : 0;
      float vs[4], vm[4];
      int kp[4];
      float top[NT][2];
      float vb = 0.f;
      uint32_t nan = 0;
#pragma unroll
      for (int nt = 0; nt < NT; nt++) top[nt][0] = top[nt][1] = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; i++) {  // key 8 i + g of the unit
        const int kl = 8 * i + g;
        const uint32_t kw = *reinterpret_cast<const uint32_t*>(st + 16 * D + kl * 4);
        const uint32_t vw = *reinterpret_cast<const uint32_t*>(st + kv4_half(D) + 16 * D + kl * 4);
        const bool in = kl < lim;
        const float ks = __uint_as_float(kw << 16);
        const float km = fmaf(-8.f, ks, __uint_as_float(kw & 0xFFFF0000u));
        vs[i] = in ? __uint_as_float(vw << 16) : 0.f;
        vm[i] = in ? __uint_as_float(vw & 0xFFFF0000u) : 0.f;
        // a value row held as NaN: 0 here, and the sum of whoever sees it NaN below
        if (vs[i] != vs[i]) vs[i] = vm[i] = 0.f, nan |= 1u << i;
        vb = fmaxf(vb, fmaf(8.f, vs[i], fabsf(vm[i])));
        kp[i] = BIAS ? *reinterpret_cast<const int*>(st + kv4_rec(D) + kl * 4) : 0;
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
          float* x = sc[i >> 1][nt] + 2 * (i & 1);
          f2unpack(f2fma(f2pack(ks, ks), f2mul(f2pack(x[0], x[1]), fac[nt]), f2mul(f2pack(km, km), qs[nt])), x[0], x[1]);
        }
      }
      if (BIAS) {
        float t[8 * NT];
#pragma unroll
        for (int i = 0; i < 8 * NT; i++) t[i] = sc[i / (4 * NT)][i / 4 % NT][i % 4];
        kv4_cap(a.s, t);
#pragma unroll
        for (int i = 0; i < 8 * NT; i++) sc[i / (4 * NT)][i / 4 % NT][i % 4] = t[i];
      }
#pragma unroll
      for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          if (BIAS) {
            const int row = nt * 8 + 2 * q + e;
            float t[4] = {sc[0][nt][e], sc[0][nt][2 + e], sc[1][nt][e], sc[1][nt][2 + e]};
            kv4_bias(a.s, t, s_slope[row], s_pos[row], start, [&](int i) { return kp[i]; });
#pragma unroll
            for (int i = 0; i < 4; i++) sc[i >> 1][nt][2 * (i & 1) + e] = t[i];
          }
#pragma unroll
          for (int i = 0; i < 4; i++) {
            float& x = sc[i >> 1][nt][2 * (i & 1) + e];
            x = 8 * i + g < lim ? x : -INFINITY;
            top[nt][e] = fmaxf(top[nt][e], x);
          }
        }
      if (over(top, exponent(vb))) {
        float least = 3e38f;  // of the unit's magnitudes other than 0
#pragma unroll
        for (int i = 0; i < 4; i++)
          if (vs[i] != 0.f || vm[i] != 0.f) least = fminf(least, fmaf(8.f, vs[i], fabsf(vm[i])));
        const float hi = exponent(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vb)))),
                    lo = exponent(__uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(least))));
        if (__builtin_expect(hi - lo <= 6.f, 1)) {  // E of the unit's greatest for all
#pragma unroll
          for (int nt = 0; nt < NT; nt++) top[nt][0] += hi, top[nt][1] += hi;
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
              top[nt][e] = -INFINITY;
#pragma unroll
              for (int i = 0; i < 4; i++)
                top[nt][e] = fmaxf(top[nt][e], sc[i >> 1][nt][2 * (i & 1) + e] + exponent(fmaf(8.f, vs[i], fabsf(vm[i]))));
            }
        }
        grow(top);
      }
      if (__any_sync(0xffffffffu, nan != 0)) {
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
          for (int nt = 0; nt < NT; nt++) {
            const float* x = sc[i >> 1][nt] + 2 * (i & 1);
            const float bad = __int_as_float(0x7FC00000);
            if (nan >> i & 1)
              l[nt] = f2add(l[nt], f2pack(x[0] == -INFINITY ? 0.f : bad, x[1] == -INFINITY ? 0.f : bad));
          }
      }
      // weights, transposed into B fragments [16-key step]
      uint32_t pf[NT][2][2];
#pragma unroll
      for (int nt = 0; nt < NT; nt++) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const float* x = sc[i >> 1][nt] + 2 * (i & 1);
          float p[2], w[2];
          f2unpack(f2add(f2pack(x[0], x[1]), ref[nt]), p[0], p[1]);
          const uint64_t pp = f2pack(ex2(p[0]), ex2(p[1]));
          l[nt] = f2add(l[nt], pp);
          mv[nt] = f2fma(pp, f2pack(vm[i], vm[i]), mv[nt]);
          f2unpack(f2mul(pp, f2pack(vs[i], vs[i])), w[0], w[1]);
          pf[nt][i >> 1][i & 1] = transpose8(pack_f16x2(w[0], w[1]));
        }
      }
      // V: lane (g, q) holds dims g D/8 .. of keys 2q, 2q + 1, 2q + 8, 2q + 9
      // of a 16-key step, merged into words of one key pair's four dims
      const uint8_t* pv = st + kv4_half(D);
#pragma unroll
      for (int i = 0; i < 2; i++) {
        uint32_t w[2][D / 32];
#pragma unroll
        for (int b = 0; b < 2; b++) {
          const int k0 = 16 * i + 8 * b + 2 * q;
          const int ka = k0 + e0, kb = k0 + 1 - e0;
          if constexpr (D == 128) {
            const uint2 x = *reinterpret_cast<const uint2*>(pv + ka * 64 + kv4_vbyte<128>(ka, g * 8));
            const uint2 y = *reinterpret_cast<const uint2*>(pv + kb * 64 + kv4_vbyte<128>(kb, g * 8));
            w[b][0] = prmt(x.x, y.x, sel_lo), w[b][1] = prmt(x.x, y.x, sel_hi);
            w[b][2] = prmt(x.y, y.y, sel_lo), w[b][3] = prmt(x.y, y.y, sel_hi);
          } else {
            const uint32_t x = *reinterpret_cast<const uint32_t*>(pv + ka * 32 + g * 4);
            const uint32_t y = *reinterpret_cast<const uint32_t*>(pv + kb * 32 + g * 4);
            w[b][0] = prmt(x, y, sel_lo), w[b][1] = prmt(x, y, sel_hi);
          }
        }
#pragma unroll
        for (int j = 0; j < D / 32; j++) {
          const uint32_t a0 = centred2<0>(w[0][j]), a1 = centred2<1>(w[0][j]), a2 = centred2<0>(w[1][j]),
                         a3 = centred2<1>(w[1][j]), b0 = centred2<2>(w[0][j]), b1 = centred2<3>(w[0][j]),
                         b2 = centred2<2>(w[1][j]), b3 = centred2<3>(w[1][j]);
#pragma unroll
          for (int nt = 0; nt < NT; nt++) {
            mma_f16(o[nt][2 * j], a0, a1, a2, a3, pf[nt][i][0], pf[nt][i][1]);
            mma_f16(o[nt][2 * j + 1], b0, b1, b2, b3, pf[nt][i][0], pf[nt][i][1]);
          }
        }
      }
      __syncwarp();
      used++;
      k++;
      if (u + 2 * W < ub) {
        if (k == 31) {  // the lanes' addresses run out
          look_up(u + 2 * W);
          k = -1;
        }
        issue(u + 2 * W, k + 1, stage);
      }
    }

    // the next segment: its first records are fetched while this one is joined
    const bool whole = ua == 0 && ub == rq.nu;
    // a part's slot: 2 c for the first segment of CTA c, 2 c + 1 for its last
    const int slot = 2 * blockIdx.x + (seg + ua > u0 ? 1 : 0);
    const int this_seg = seg;
    const Kv4Req tq = rq;
    seg += rq.nu;
    const bool more = seg < u1;
    if (more) {
      if (++s == a.c.hkv * rq.nc) {
        s = 0;
        do rq = kv4_req<RT, 1, BIAS>(a, ++r);
        while (rq.nc == 0);
      }
      ua = 0;
      ub = min(rq.nu, u1 - seg);
      begin();
    }

    // join the warps
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        float le = __uint_as_float((uint32_t)(l[nt] >> (32 * e))), mve = __uint_as_float((uint32_t)(mv[nt] >> (32 * e)));
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          le += __shfl_xor_sync(0xffffffffu, le, x);
          mve += __shfl_xor_sync(0xffffffffu, mve, x);
        }
        const int row = nt * 8 + 2 * q + e;
        if (g == 0) {
          s_m[warp * RT + row] = -__uint_as_float((uint32_t)(ref[nt] >> (32 * e)));
          s_l[warp * RT + row] = le;
        }
        // float pairs [dims 2t, 2t + 1 of lane group g]: 8 t + g, rows 4 banks
        // of pairs apart for the lanes that write together
        float2* dst = reinterpret_cast<float2*>(s_o) + (warp * RT + row) * S::kPairs + g;
#pragma unroll
        for (int t = 0; t < KK; t++)
          dst[8 * t] = make_float2(fmaf(o[nt][t][e], 512.f, mve), fmaf(o[nt][t][2 + e], 512.f, mve));
      }
    __syncthreads();
    float* part = a.part + (int64_t)slot * (RT * (D + 2));  // [RT][D/2] pairs, then [RT] (max, sum)
    auto row_out = [&](int row) {  // (row, query head) of the outputs
      const int rho = rc * RT + row, gq = rho / tq.m;
      return (int64_t)(tq.n0 + rho - gq * tq.m) * a.hq + h * a.G + gq;
    };
    if (tid < rows) {
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w < W; w++) M = fmaxf(M, s_m[w * RT + tid]);
      const float Ms = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int w = 0; w < W; w++) {
        const float f = ex2(s_m[w * RT + tid] - Ms);  // 0 for a warp that saw no key; 0 x NaN for one that saw only NaN
        L += f * s_l[w * RT + tid];
        s_m[w * RT + tid] = f;
      }
      s_L[tid] = L == 0.f ? 0.f : 1.f / L;
      if (whole) {
        if (a.lse) a.lse[row_out(tid)] = L == 0.f ? -INFINITY : (M + log2f(L)) * (1.f / kLog2e);
      } else {
        __stcg(reinterpret_cast<float2*>(part + RT * D) + tid, make_float2(M, L));
      }
    }
    __syncthreads();
    for (int i = tid; i < rows * (D / 2); i += W * 32) {
      const int row = i / (D / 2), x = i % (D / 2);
      float2 acc = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; w++) {
        const float f = s_m[w * RT + row];
        const float2 v = reinterpret_cast<const float2*>(s_o)[(w * RT + row) * S::kPairs + x];
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
      }
      if (whole) {
        const float inv = s_L[row];
        *reinterpret_cast<uint32_t*>(a.out + row_out(row) * D + (x & 7) * (D / 8) + (x >> 3) * 2) =
            pack_bf16x2(acc.x * inv, acc.y * inv);
      } else {
        __stcg(reinterpret_cast<float2*>(part) + i, acc);
      }
    }
    __syncthreads();  // s_o, s_q and the rows' data are free again; a part is written
    if (!whole && tid == W * 32 - 32) {
      // Is this the last of the segment's CTAs to write its part?  Only the
      // warp with the fewest records waits for the answer, which is acted on
      // at this CTA's end: a part is the first of its segments or the last.
      const int c0 = sh.cta_of(this_seg), n = sh.cta_of(this_seg + tq.nu - 1) - c0 + 1;
      const bool last = atomic_add_acq_rel(a.tickets + c0, 1) == n - 1;
      if (last) a.tickets[c0] = 0;
      s_join[more ? 0 : 1] = last ? Kv4Join{this_seg, n, c0, tq.n0, tq.m, h, rc} : Kv4Join{};
    }
    if (!more) break;
  }

  // Join the parts of the segments that this CTA was the last to finish: first
  // each row's factor of every part, a warp a row and a lane a part, then the
  // parts' sums, four dims a thread and P parts of every one of its kItems in
  // flight (a loop with one latency per item and eight parts took a third of
  // a short call).
  constexpr int kItems = (RT * (D / 4) + W * 32 - 1) / (W * 32), P = kItems > 1 ? 4 : 8;
  static_assert(kMaxCtas * RT * 4 <= S::off_q, "factors take the place of the ring and the outputs");
  float* s_f = reinterpret_cast<float*>(sm);  // [RT][n]
  for (int d = 0; d < 2; d++) {
    __syncthreads();
    const Kv4Join jn = s_join[d];
    if (jn.n == 0) continue;
    const int n = jn.n, rows = min(RT, a.G * jn.m - jn.rc * RT);
    // c0's part is its last segment's unless the segment begins its share
    const int slot0 = 2 * jn.c0 + (sh.first(jn.c0) < jn.seg ? 1 : 0);
    auto part_of = [&](int c) { return a.part + (int64_t)(c == 0 ? slot0 : 2 * (jn.c0 + c)) * (RT * (D + 2)); };
    auto row_out = [&](int row) {  // (row, query head) of the outputs
      const int rho = jn.rc * RT + row, gq = rho / jn.m;
      return (int64_t)(jn.n0 + rho - gq * jn.m) * a.hq + jn.h * a.G + gq;
    };
    for (int row = warp; row < rows; row += W) {
      float M = -INFINITY, L = 0.f;
      float2 ml = make_float2(-INFINITY, 0.f);  // the last that this lane read
      for (int c = lane; c < n; c += 32) {
        ml = __ldcg(reinterpret_cast<const float2*>(part_of(c) + RT * D) + row);
        M = fmaxf(M, ml.x);
      }
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
      const float Ms = M == -INFINITY ? 0.f : M;
      for (int c = lane; c < n; c += 32) {
        if (n > 32) ml = __ldcg(reinterpret_cast<const float2*>(part_of(c) + RT * D) + row);
        const float f = ex2(ml.x - Ms);
        L = fmaf(f, ml.y, L);
        s_f[row * n + c] = f;
      }
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
      if (lane == 0) {
        s_L[row] = L == 0.f ? 0.f : 1.f / L;
        if (a.lse) a.lse[row_out(row)] = L == 0.f ? -INFINITY : (M + log2f(L)) * (1.f / kLog2e);
      }
    }
    __syncthreads();
    float4 acc[kItems];
#pragma unroll
    for (int t = 0; t < kItems; t++) acc[t] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = 0; c < n; c += P) {
      float4 v[kItems][P];
#pragma unroll
      for (int k = 0; k < P; k++) {
        const float4* pc = reinterpret_cast<const float4*>(part_of(min(c + k, n - 1)));
#pragma unroll
        for (int t = 0; t < kItems; t++) {
          const int i = tid + t * W * 32;
          if (i < rows * (D / 4)) v[t][k] = __ldcg(pc + i);
        }
      }
#pragma unroll
      for (int k = 0; k < P; k++)
        if (c + k < n) {
#pragma unroll
          for (int t = 0; t < kItems; t++) {
            const int i = tid + t * W * 32;
            if (i < rows * (D / 4)) {
              const float f = s_f[i / (D / 4) * n + c + k];
              acc[t].x = fmaf(f, v[t][k].x, acc[t].x);
              acc[t].y = fmaf(f, v[t][k].y, acc[t].y);
              acc[t].z = fmaf(f, v[t][k].z, acc[t].z);
              acc[t].w = fmaf(f, v[t][k].w, acc[t].w);
            }
          }
        }
    }
#pragma unroll
    for (int t = 0; t < kItems; t++) {
      const int i = tid + t * W * 32;
      if (i >= rows * (D / 4)) continue;
      const int row = i / (D / 4), x = i % (D / 4) * 2;  // pairs x and x + 1, dims D/8 apart
      const float inv = s_L[row];
      uint16_t* o = a.out + row_out(row) * D + (x & 7) * (D / 8) + (x >> 3) * 2;
      *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(acc[t].x * inv, acc[t].y * inv);
      *reinterpret_cast<uint32_t*>(o + D / 8) = pack_bf16x2(acc[t].z * inv, acc[t].w * inv);
    }
  }
}

struct Kv4ObserveArgs {
  Kv4AttnArgs a;
  const float* lse_in;
  const float* row_weight;
  float decay;
  float* out;
};

// ------------------------------------------------------------- observe --
//
// S^T tiles as above, from the K half of the records alone: exp(score - lse)
// of a key is summed over the tile's rows in the lane, over the four lanes
// that share the key at the end.  Rows of weight 0 are left out before the
// products (a verified tree's rejected nodes).  Bound by the bytes of K while
// a kv head has up to about three tiles of eight rows, by the products past
// that.  No sum crosses a warp, so there is nothing to join: a (request, kv
// head)'s groups of 32 slots are dealt over the CTAs like the attention's.
// More than kObsRows rows are taken in passes that add to the output.
// Measured: 32 requests of 2 to 5 rows, 32 query and 8 kv heads, over 1500 to 8192
// keys with positions: 41 us, 2.4 TB/s, 16 warps an SM waiting on their own
// products and exponentials.  (Two tiles of rows at a time, for one making of the
// codes' words: 59 where one takes 53.)

constexpr int kObsWarps = 8, kObsRows = 128, kObsStages = 3;

template <int D>
struct ObserveShape {
  static constexpr int kStage = kv4_half(D) + 128;
  static constexpr int off_q = kObsWarps * kObsStages * kStage;   // [rows/8][D/32][32] uint4
  static constexpr int off_row = off_q + kObsRows * D * 2;        // [rows] (factor, sum q, lse, weight)
  static constexpr int off_bias = off_row + kObsRows * 16;        // [rows] (slope, position)
  static constexpr int off_node = off_bias + kObsRows * 8;        // [64] nodes of weight other than 0
  static constexpr int off_bar = off_node + 64 * 4;
  static constexpr int off_ok = off_bar + kObsWarps * kObsStages * 8;
  static constexpr int smem = off_ok + kObsWarps * kObsStages * 4;
};

template <int D, bool BIAS>
__global__ void __launch_bounds__(kObsWarps * 32, 2) k_kv4_observe(const __grid_constant__ Kv4ObserveArgs b) {
  using S = ObserveShape<D>;
  constexpr int W = kObsWarps, NS = kObsStages;
  const Kv4AttnArgs& a = b.a;
  extern __shared__ __align__(128) uint8_t sm[];
  uint4* s_q = reinterpret_cast<uint4*>(sm + S::off_q);
  float4* s_row = reinterpret_cast<float4*>(sm + S::off_row);
  float2* s_bias = reinterpret_cast<float2*>(sm + S::off_bias);
  int* s_node = reinterpret_cast<int*>(sm + S::off_node);
  uint64_t* s_bar = reinterpret_cast<uint64_t*>(sm + S::off_bar);
  int* s_ok = reinterpret_cast<int*>(sm + S::off_ok);
  __shared__ int s_r0, s_u0, s_u1, s_req0, s_abort, s_n;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;

  auto context = [&](int r) {
    int ctx = a.c.ctx_len[r];
    if (ctx < 0 || ctx > a.c.cap) {
      set_status(a.status, SD_ERR_CAPACITY);
      ctx = ctx < 0 ? 0 : (int)a.c.cap;
    }
    return ctx;
  };
  if (warp == 0) {
    int U = 0, lo = 0, n = 0;
    for (int pass = 0, u0 = 0, u1 = 0; pass < 2; pass++) {
      int before = 0;
      for (int base = 0; base < a.R; base += 32) {
        if (pass == 0 || a.R > 32) {
          n = base + lane < a.R ? a.c.hkv * ((context(base + lane) + 31) / 32) : 0;
          int run = n;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += v;
          }
          lo = before + run - n;
          before += __shfl_sync(0xffffffffu, run, 31);
        }
        if (pass == 1 && u0 >= lo && u0 < lo + n) {
          s_r0 = base + lane;
          s_req0 = lo;
        }
      }
      if (pass == 0) {
        U = before;
        const int C = max(1, min((int)gridDim.x, (U + W - 1) / W)), each = U / C, more = U - each * C;
        u0 = (int)blockIdx.x < C ? (int)blockIdx.x * each + min((int)blockIdx.x, more) : U;
        u1 = (int)blockIdx.x < C ? u0 + each + ((int)blockIdx.x < more) : U;
        if (lane == 0) {
          s_u0 = u0;
          s_u1 = u1;
          s_abort = 0;
        }
      }
    }
  }
  if (lane == 0) {
    for (int i = 0; i < NS; i++) mbar_init(&s_bar[warp * NS + i], 1);
    fence_mbar_init();
  }
  __syncthreads();
  const int u1 = s_u1;
  if (s_u0 >= u1) return;
  uint64_t* const bar = s_bar + warp * NS;
  uint8_t* const ring = sm + warp * NS * S::kStage;
  const float sc2 = BIAS ? 1.f : a.s.scale * kLog2e;
  uint32_t used = 0;

  int r = s_r0, req0 = s_req0, u = s_u0;  // request, its first unit, the segment's first unit of this CTA
  int ctx = context(r);
  while (u < u1) {
    int ng = (ctx + 31) / 32;
    while (u >= req0 + a.c.hkv * ng) {
      req0 += a.c.hkv * ng;
      ctx = context(++r);
      ng = (ctx + 31) / 32;
    }
    const int h = (u - req0) / ng, g0 = u - req0 - h * ng, g1 = min(ng, g0 + u1 - u);
    u += g1 - g0;
    const int n0 = a.cu[r], m = min(max(a.cu[r + 1] - n0, 0), 64);
    const int start = BIAS && a.s.start ? a.s.start[r] : INT32_MIN;
    const int first = BIAS && (a.s.window > 0 || a.s.start)
                          ? kv4_first(a.c, a.s, r, ctx, a.row_pos && m ? a.row_pos[n0] : ctx) / kKvGroup
                          : 0;  // groups before it collect nothing
    if (warp == 0) {  // the rows that count
      int n = 0;
      for (int i = 0; i < m; i += 32) {
        const bool on = i + lane < m && (!b.row_weight || b.row_weight[n0 + i + lane] != 0.f);
        const uint32_t on32 = __ballot_sync(0xffffffffu, on);
        if (on) s_node[n + __popc(on32 & ((1u << lane) - 1))] = i + lane;
        n += __popc(on32);
      }
      if (lane == 0) s_n = n;
    }
    __syncthreads();
    const int n = s_n, rows = n * a.G;
    const float* w_in = a.c.weight + a.c.slot0(r, h);
    float* w_out = b.out + a.c.slot0(r, h);
    for (int pass = 0; pass == 0 || pass * kObsRows < rows; pass++) {
      const int left = min(kObsRows, rows - pass * kObsRows), tiles = (left + 7) / 8;
      // the records of this warp: groups ga, ga + W, ...; a lane holds the
      // address of every 32nd
      const int ga = g0 + warp + (rows > 0 && first > g0 + warp ? (first - g0 - warp + W - 1) / W * W : 0);
      const int ge = rows > 0 ? g1 : g0;
      const uint8_t* addr = nullptr;
      auto look_up = [&](int x) {
        x += lane * W;
        addr = x < ge ? a.c.record(D, r, h, x) : nullptr;
      };
      auto issue = [&](int x, int k, int stage) {
        const uint8_t* rec = reinterpret_cast<const uint8_t*>(
            __shfl_sync(0xffffffffu, (unsigned long long)reinterpret_cast<uintptr_t>(addr), k));
        if (lane == 0) {
          s_ok[warp * NS + stage] = rec != nullptr;
          if (rec) {
            uint8_t* dst = ring + stage * S::kStage;
            mbar_arrive_expect_tx(&bar[stage], kv4_half(D) + (BIAS ? 128 : 0));
            bulk_g2s(dst, rec, kv4_half(D), &bar[stage]);
            if (BIAS) bulk_g2s(dst + kv4_half(D), a.c.pos + a.c.slot0(r, h) + x * kKvGroup, 128, &bar[stage]);
          } else {
            set_status(a.status, SD_ERR_CAPACITY);
            mbar_arrive(&bar[stage]);
          }
        }
        __syncwarp();
      };
      if (ga < ge) look_up(ga);
#pragma unroll
      for (int i = 0; i < NS; i++)
        if (ga + i * W < ge) issue(ga + i * W, i, (used + i) % NS);
      // groups before the first that any row sees only fade
      if (pass == 0)
        for (int x = g0 + warp; x < (rows > 0 ? min(g1, first) : g1); x += W) {
          const int t = x * kKvGroup + lane;
          if (t < ctx) w_out[t] = b.decay * w_in[t];
        }
      for (int i = tid; i < tiles * 8 * (D / 8); i += W * 32) {
        const int row = i / (D / 8), oct = i % (D / 8);
        const int rho = pass * kObsRows + row;
        const bool ok = rho < rows;
        const int gq = ok ? rho / n : 0, node = ok ? s_node[rho - gq * n] : 0, hq = h * a.G + gq;
        // a row that sees nothing, or whose lse is not finite, gives no weight:
        // its queries (NaN, perhaps) are taken as 0 and its lse as infinite
        uint4 x = make_uint4(0, 0, 0, 0);
        float lse = INFINITY, rw = 1.f, slope = 0.f;
        int pos = ctx + node;
        if (ok) {
          x = *reinterpret_cast<const uint4*>(a.q + (int64_t)(n0 + node) * a.q_stride + hq * D + oct * 8);
          lse = b.lse_in[(int64_t)(n0 + node) * a.hq + hq];
          if (b.row_weight) rw = b.row_weight[n0 + node];
          if (BIAS && a.s.slopes) slope = a.s.slopes[hq];
        }
        if (BIAS && a.row_pos) pos = a.row_pos[n0 + node];
        const bool gives = fabsf(lse) < INFINITY;
        if (!gives) x = make_uint4(0, 0, 0, 0);
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
        float f[8], qs = 0.f, big = 0.f;
#pragma unroll
        for (int k = 0; k < 8; k++) {
          f[k] = bf2f((uint16_t)(xs[k >> 1] >> (16 * (k & 1))));
          qs += f[k];
          big = fmaxf(big, fabsf(f[k]));
        }
#pragma unroll
        for (int o = D / 16; o > 0; o >>= 1) {
          qs += __shfl_xor_sync(0xffffffffu, qs, o);
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
        }
        const int e = min(max(14 + 127 - (int)(__float_as_uint(big) >> 23), -100), 100);
        const float up = pow2i(e), up4 = pow2i(e - 4);
        s_q[((row >> 3) * (D / 32) + oct % (D / 32)) * 32 + 4 * (row & 7) + oct / (D / 32)] =
            make_uint4(pack_f16x2(f[0] * up, f[4] * up), pack_f16x2(f[1] * up4, f[5] * up4),
                       pack_f16x2(f[2] * up, f[6] * up), pack_f16x2(f[3] * up4, f[7] * up4));
        if (oct == 0) {
          s_row[row] = make_float4(pow2i(24 - e) * sc2, qs * sc2, gives ? lse * kLog2e : INFINITY, gives ? rw : 0.f);
          s_bias[row] = make_float2(gives ? slope : 0.f, __int_as_float(pos));
        }
      }
      __syncthreads();
      int k = 0;
      for (int x = ga; x < ge; x += W) {
        const int stage = used % NS;
        const uint8_t* st = ring + stage * S::kStage;
        const int t = x * kKvGroup + 8 * q + g;  // the slot whose sum this lane writes
        float old = 0.f;  // not looked at before the end
        if (t < ctx) old = pass ? w_out[t] : w_in[t];
        if (!kv4_wait(&bar[stage], (used / NS) & 1, &s_abort)) set_status(a.status, SD_TIMEOUT_AT(31));
        const bool ok = s_ok[warp * NS + stage] != 0;
        uint32_t kw[4][D / 32];
        float ks[4], km[4];
        int kp[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const uint8_t* p = st + (8 * i + g) * (D / 2) + q * (D / 8);
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            kw[i][0] = v.x, kw[i][1] = v.y, kw[i][2] = v.z, kw[i][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            kw[i][0] = v.x, kw[i][1] = v.y;
          }
          const uint32_t w = *reinterpret_cast<const uint32_t*>(st + 16 * D + (8 * i + g) * 4);
          ks[i] = __uint_as_float(w << 16);
          km[i] = fmaf(-8.f, ks[i], __uint_as_float(w & 0xFFFF0000u));
          kp[i] = BIAS ? *reinterpret_cast<const int*>(st + kv4_half(D) + (8 * i + g) * 4) : 0;
        }
        __syncwarp();
        used++;
        k++;
        if (x + NS * W < ge) {
          if (k + NS - 1 == 32) {  // the lanes' addresses run out
            look_up(x + NS * W);
            k = 1 - NS;
          }
          issue(x + NS * W, k + NS - 1, stage);
        }
        uint64_t sum2[4] = {0, 0, 0, 0};  // of either row of a pair
        for (int nt = 0; nt < tiles; nt++) {
          float sc[2][2][4];  // [16-key tile][chain]
#pragma unroll
          for (int i = 0; i < 2; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) sc[i][0][e] = sc[i][1][e] = 0.f;
#pragma unroll
          for (int j = 0; j < D / 32; j++) {
            const uint4 bq = s_q[(nt * (D / 32) + j) * 32 + lane];
#pragma unroll
            for (int i = 0; i < 2; i++) {
              const uint32_t wa = kw[2 * i][j], wb = kw[2 * i + 1][j];
              mma_f16(sc[i][0], codes2<0>(wa), codes2<0>(wb), codes2<1>(wa), codes2<1>(wb), bq.x, bq.y);
              mma_f16(sc[i][1], codes2<2>(wa), codes2<2>(wb), codes2<3>(wa), codes2<3>(wb), bq.z, bq.w);
            }
          }
          const int row = nt * 8 + 2 * q;
          const float4 r0 = s_row[row], r1 = s_row[row + 1];
          const uint64_t fac = f2pack(r0.x, r1.x), qs = f2pack(r0.y, r1.y), lse = f2pack(-r0.z, -r1.z), rw = f2pack(r0.w, r1.w);
          float v[2][4];
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const float *x = sc[i >> 1][0] + 2 * (i & 1), *y = sc[i >> 1][1] + 2 * (i & 1);
            f2unpack(f2fma(f2pack(ks[i], ks[i]), f2mul(f2add(f2pack(x[0], x[1]), f2pack(y[0], y[1])), fac),
                           f2mul(f2pack(km[i], km[i]), qs)), v[0][i], v[1][i]);
          }
          if (BIAS) {
            float t[8];
#pragma unroll
            for (int i = 0; i < 8; i++) t[i] = v[i & 1][i >> 1];
            kv4_cap(a.s, t);
#pragma unroll
            for (int i = 0; i < 8; i++) v[i & 1][i >> 1] = t[i];
#pragma unroll
            for (int e = 0; e < 2; e++) {
              const float2 bi = s_bias[row + e];
              kv4_bias(a.s, v[e], bi.x, __float_as_int(bi.y), start, [&](int i) { return kp[i]; });
            }
          }
#pragma unroll
          for (int i = 0; i < 4; i++) {
            float p[2];
            f2unpack(f2add(f2pack(v[0][i], v[1][i]), lse), p[0], p[1]);
            sum2[i] = f2fma(rw, f2pack(ex2(p[0]), ex2(p[1])), sum2[i]);
          }
        }
        float sum[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          float lo, hi;
          f2unpack(sum2[i], lo, hi);
          sum[i] = lo + hi;
        }
        float mine = 0.f, s = 0.f;  // of the slot that this lane writes
#pragma unroll
        for (int i = 0; i < 4; i++) {
          sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
          sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
          if (q == i) mine = sum[i], s = ks[i];
        }
        // a key held as NaN collects nothing: who sees it has no finite lse
        if (t < ctx) w_out[t] = (pass ? old : b.decay * old) + (ok && s == s ? mine : 0.f);
      }
      __syncthreads();  // s_q, s_row and s_node are free again
    }
  }
}

// ---------------------------------------------------------------- launch --

constexpr size_t kTicketBytes = 4096;  // one ticket a CTA

template <int D, int NT, int W>
static int launch_attn_tile(const Kv4AttnArgs& a, int64_t units, bool bias, cudaStream_t st) {
  auto kern = bias ? k_kv4_attn<D, NT, W, true> : k_kv4_attn<D, NT, W, false>;
  constexpr int smem = AttnShape<D, NT, W>::smem;
  static const cudaError_t set[2] = {
      cudaFuncSetAttribute(k_kv4_attn<D, NT, W, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
      cudaFuncSetAttribute(k_kv4_attn<D, NT, W, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)};
  SD_CK(set[bias]);
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>({2ll * num_sms(), kMaxCtas, units}));
  kern<<<(unsigned)grid, W * 32, smem, st>>>(a);
  SD_CK(cudaGetLastError());
  return SD_OK;
}

template <int D>
static int launch_observe(const Kv4ObserveArgs& b, int64_t units, bool bias, cudaStream_t st) {
  constexpr int smem = ObserveShape<D>::smem;
  static const cudaError_t set[2] = {
      cudaFuncSetAttribute(k_kv4_observe<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
      cudaFuncSetAttribute(k_kv4_observe<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)};
  SD_CK(set[bias]);
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(2ll * num_sms(), (units + kObsWarps - 1) / kObsWarps));
  (bias ? k_kv4_observe<D, true> : k_kv4_observe<D, false>)<<<(unsigned)grid, kObsWarps * 32, smem, st>>>(b);
  SD_CK(cudaGetLastError());
  return SD_OK;
}

// Rows (query heads x nodes) that one kv head may have on the warp kernel;
// more take the tensor cores.  Measured at 8 kv heads, D = 128, calls one after
// another from a graph, warp kernel against tensor cores, us:
//   rows   one request of 2000, 16000, 65536 keys    eight of 2000, 16000
//   96     19, 45, 128 / 20, 46, 100                 52, 242 / 46, 173
//   64     16, 37, 92 / 19, 43, 91                   36, 165 / 41, 151
//   32     16, 28, 58 / 18, 42, 90                   28, 94 / 40, 153
// The rule goes by the rows of the largest request alone: at 64 rows and the
// longest contexts the tensor cores would save a tenth, and a batch of one large
// tree and single tokens would do better on both kernels.  With one tile of eight
// rows a warp (NT = 1) eight warps fit, with two six.
constexpr int kWarpRows = 64;

template <int D>
static int launch_attn(const Kv4AttnArgs& a, int total, int rows, int64_t units, bool bias, cudaStream_t st) {
  if (rows <= 8) return launch_attn_tile<D, 1, 8>(a, units, bias, st);
  if (rows <= kWarpRows) return launch_attn_tile<D, 2, 6>(a, units, bias, st);
  return kv4_launch_attn_tc(a, D, total, rows, (units + 1) / 2, bias, st);
}

// ---------------------------------------------------------------- checks --

static int check_call(const char* who, const sd_kv4* c, const uint16_t* q, int64_t q_stride, int32_t hq,
                      const int32_t* cu, const int32_t* cu_host, int32_t R, const sd_kv4_score* score, int32_t max_ctx,
                      Kv4AttnArgs* a) {
  if (int rc = kv4_check(c, R, who, &a->c)) return rc;
  if (int rc = kv4_check_rows(cu, cu_host, R, who)) return rc;
  if (int rc = kv4_check_score(score, who, &a->s, c->head_dim)) return rc;
  if (cu_host[R] && (!q || (reinterpret_cast<uintptr_t>(q) & 15)))
    return kv4_bad(SD_ERR_INVALID_ARG, who, "q must be set and 16-byte aligned");
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
  const size_t warp = (size_t)4 * num_sms() * 16 * (head_dim + 2) * sizeof(float);  // two parts a CTA, two CTAs an SM
  const int most = std::min(rows, 64) * (n_q_heads / n_kv_heads);
  return kTicketBytes + (most > kWarpRows ? std::max(warp, kv4_tc_workspace(R, n_kv_heads, head_dim)) : warp);
}

extern "C" int sd_kv4_attn(const sd_kv4* c, const uint16_t* q, int64_t q_stride, int32_t n_q_heads, const int32_t* cu,
                           const int32_t* cu_host, int32_t R, const uint16_t* k_new, const uint16_t* v_new,
                           int64_t kv_stride, const uint64_t* anc, const int32_t* row_pos, const sd_kv4_score* score,
                           int32_t max_ctx, uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                           int32_t* status, void* stream) {
  const char* who = "sd_kv4_attn";
  Kv4AttnArgs a = {};
  if (int rc = check_call(who, c, q, q_stride, n_q_heads, cu, cu_host, R, score, max_ctx, &a)) return rc;
  const int rows = cu_host[R];
  if (rows == 0) return SD_OK;  // the arrays of no rows may be null
  if (!out || (reinterpret_cast<uintptr_t>(out) & 15)) return kv4_bad(SD_ERR_INVALID_ARG, who, "out must be set and 16-byte aligned");
  if (!k_new != !v_new) return kv4_bad(SD_ERR_INVALID_ARG, who, "k_new and v_new go together");
  if (k_new) {
    if (((reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) & 15) ||
        kv_stride < (int64_t)c->n_kv_heads * c->head_dim || kv_stride % 8)
      return kv4_bad(SD_ERR_INVALID_ARG, who,
                     "k_new and v_new must be 16-byte aligned, kv_stride must cover a row and be a multiple of 8");
  }
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return kv4_bad(SD_ERR_INVALID_ARG, who, "workspace must be set and 256-byte aligned");
  if (workspace_bytes < sd_kv4_attn_workspace(R, rows, n_q_heads, c->n_kv_heads, c->head_dim))
    return kv4_bad(SD_ERR_WORKSPACE, who, "workspace too small");
  a.k_new = k_new;
  a.v_new = v_new;
  a.kv_stride = kv_stride;
  a.anc = anc;
  a.row_pos = row_pos;
  a.out = out;
  a.lse = lse;
  a.status = status;
  a.tickets = (int32_t*)workspace;
  a.part = (float*)((uint8_t*)workspace + kTicketBytes);
  int most = 0;
  for (int r = 0; r < R; r++) most = std::max(most, (cu_host[r + 1] - cu_host[r]) * a.G);
  const int64_t ctx = max_ctx > 0 ? std::min<int64_t>(max_ctx, a.c.cap) : a.c.cap;
  const int64_t units = (int64_t)R * c->n_kv_heads * ((most + 31) / 32) * ((ctx + 31) / 32 + 2);
  if ((int64_t)R * c->n_kv_heads * ((most + 7) / 8) * ((a.c.cap + 31) / 32 + 2) > 0x7FFFFFFF)
    return kv4_bad(SD_ERR_UNSUPPORTED, who, "more than 2^31 runs of 32 keys");
  const bool bias = a.s.cap > 0.f || a.s.slopes || a.s.window > 0 || a.s.start;
  return c->head_dim == 128 ? launch_attn<128>(a, rows, most, units, bias, (cudaStream_t)stream)
                            : launch_attn<64>(a, rows, most, units, bias, (cudaStream_t)stream);
}

extern "C" int sd_kv4_observe(const sd_kv4* c, const uint16_t* q, int64_t q_stride, int32_t n_q_heads,
                              const float* lse, const int32_t* cu, const int32_t* cu_host, int32_t R,
                              const int32_t* row_pos, const float* row_weight, const sd_kv4_score* score,
                              int32_t max_ctx, float decay, float* weight_out, int32_t* status, void* stream) {
  const char* who = "sd_kv4_observe";
  Kv4ObserveArgs b = {};
  if (int rc = check_call(who, c, q, q_stride, n_q_heads, cu, cu_host, R, score, max_ctx, &b.a)) return rc;
  if (!lse && cu_host[R]) return kv4_bad(SD_ERR_INVALID_ARG, who, "null lse");
  if (!weight_out || (reinterpret_cast<uintptr_t>(weight_out) & 15))
    return kv4_bad(SD_ERR_INVALID_ARG, who, "weight_out must be set and 16-byte aligned");
  if (!(decay >= 0.f) || !(decay <= 1e30f)) return kv4_bad(SD_ERR_INVALID_ARG, who, "decay must be finite and not negative");
  b.a.row_pos = row_pos;
  b.a.status = status;
  b.lse_in = lse;
  b.row_weight = row_weight;
  b.decay = decay;
  b.out = weight_out;
  // a request longer than max_ctx is still read whole: the CTAs share the units there are
  const int64_t ctx = max_ctx > 0 ? std::min<int64_t>(max_ctx, b.a.c.cap) : b.a.c.cap;
  const int64_t units = (int64_t)R * c->n_kv_heads * ((ctx + 31) / 32);
  if ((int64_t)R * c->n_kv_heads * ((b.a.c.cap + 31) / 32) > 0x7FFFFFFF)
    return kv4_bad(SD_ERR_UNSUPPORTED, who, "more than 2^31 runs of 32 keys");
  const bool bias = b.a.s.cap > 0.f || b.a.s.slopes || b.a.s.window > 0 || b.a.s.start;
  return c->head_dim == 128 ? launch_observe<128>(b, units, bias, (cudaStream_t)stream)
                            : launch_observe<64>(b, units, bias, (cudaStream_t)stream);
}
