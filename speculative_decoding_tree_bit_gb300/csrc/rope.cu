// Rotary positions of queries and keys.
#include <algorithm>
#include <cmath>

#include "common.cuh"

namespace sdv {

// ------------------------------------------------------------------ angles --
//
// A pair's frequency is kept as turns a position, a fraction of 2^64, so the
// angle of any int32 position is one wrapping product: its upper half is the turn as a
// signed fraction, cut at 2^-32, which sincospi takes after one conversion (2^-26 of a
// turn).  The frequency itself comes from 64-bit floating point, off by at most 2^-53 of
// a turn a position.  (In fp32 pos f would be off by 0.06 rad at position 10^6.)

__device__ __forceinline__ void rope_angle(uint64_t turns, int pos, float amplitude, float& c, float& s) {
  const int32_t frac = (int32_t)(((uint64_t)(int64_t)pos * turns) >> 32);
  sincospif((float)frac * 0x1p-31f, &s, &c);
  c *= amplitude;
  s *= amplitude;
}

struct RopeArgs {
  const uint64_t* turns;
  const int32_t* pos;
  const uint16_t* in[2];   // q, k
  uint16_t* out[2];
  int64_t in_stride[2], out_stride[2];
  int heads[2];
  int rows, rot, D;        // rot: rot_dim
  int groups;              // threads of a row and a run of heads
  int each;                // heads of a run, at most
  int q_runs, runs;        // runs of a row: of queries, and in all
  float amplitude;
};

struct HeadRun {
  const uint16_t* in;
  uint16_t* out;
  int n;
};

__device__ __forceinline__ HeadRun head_run(const RopeArgs& a, int64_t row, int run) {
  const bool k = run >= a.q_runs;
  const int h = (k ? run - a.q_runs : run) * a.each;
  return {(k ? a.in[1] : a.in[0]) + row * (k ? a.in_stride[1] : a.in_stride[0]) + (int64_t)h * a.D,
          (k ? a.out[1] : a.out[0]) + row * (k ? a.out_stride[1] : a.out_stride[0]) + (int64_t)h * a.D,
          min(a.each, (k ? a.heads[1] : a.heads[0]) - h)};
}

// Eight pairs of two pieces: (p, q) becomes (p c - q s, p s + q c), each rounded once.
template <bool INTERLEAVED>
__device__ __forceinline__ void turn_pairs(uint32_t* u, uint32_t* v, const float* c, const float* s) {
  if (INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      uint32_t& wd = i < 4 ? u[i] : v[i - 4];
      const float p = __uint_as_float(wd << 16), q = __uint_as_float(wd & 0xFFFF0000u);
      wd = pack_bf16x2(fmaf(p, c[i], -q * s[i]), fmaf(p, s[i], q * c[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float p0 = __uint_as_float(u[i] << 16), p1 = __uint_as_float(u[i] & 0xFFFF0000u);
      const float q0 = __uint_as_float(v[i] << 16), q1 = __uint_as_float(v[i] & 0xFFFF0000u);
      u[i] = pack_bf16x2(fmaf(p0, c[2 * i], -q0 * s[2 * i]), fmaf(p1, c[2 * i + 1], -q1 * s[2 * i + 1]));
      v[i] = pack_bf16x2(fmaf(p0, s[2 * i], q0 * c[2 * i]), fmaf(p1, s[2 * i + 1], q1 * c[2 * i + 1]));
    }
  }
}

// A thread has eight pairs of a row (two 16-byte pieces a head) and turns them in
// `each` heads, so their sines are computed once for all of those; the pieces of
// the dims that do not turn are copied by further threads.  Bound by memory: each
// value crosses once.  What counts is how much a thread has under way, because a
// store may not pass a load of the same tensor and so ends a run of loads: 403 MB
// (16384 rows, 40 + 8 heads of 128) take 69 us with one head's loads at a time, 63
// with two, 61 (6.6 TB/s) with four, 64 with eight and the fewer warps of their
// registers.  4099 rows of 16 + 16 heads of 64, interleaved, 32 dims turned: 7.4 us.
constexpr int kBatch = 4;

template <bool INTERLEAVED>
__global__ void __launch_bounds__(256, 3) k_rope(RopeArgs a) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t part = id / a.groups;
  const int g = (int)(id - part * a.groups);
  const int64_t row = part / a.runs;
  if (row >= a.rows) return;
  const int run = (int)(part - row * a.runs);
  const int np = a.rot / 16;  // threads that turn pairs
  const bool turn = g < np;
  // the two pieces' first dims
  int d0, d1;
  if (turn) {
    d0 = INTERLEAVED ? g * 16 : g * 8;
    d1 = INTERLEAVED ? d0 + 8 : d0 + a.rot / 2;
  } else {
    d0 = a.rot + (g - np) * 16;
    d1 = d0 + 8;
  }
  const bool two = d1 < a.D;
  float c[8], s[8];
  if (turn) {
    const int p = a.pos[row];
#pragma unroll
    for (int i = 0; i < 8; i++) rope_angle(a.turns[g * 8 + i], p, a.amplitude, c[i], s[i]);
  }
  const HeadRun r = head_run(a, row, run);
  const uint16_t* x = r.in;
  uint16_t* y = r.out;
  for (int left = r.n; left > 0; left -= kBatch, x += kBatch * a.D, y += kBatch * a.D) {
    // a store may not pass a load of the same tensor, so kBatch heads' loads come first
    uint4 u[kBatch], v[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; j++) {
      if (j >= left) break;
      u[j] = *reinterpret_cast<const uint4*>(x + j * a.D + d0);
      if (two) v[j] = *reinterpret_cast<const uint4*>(x + j * a.D + d1);
    }
#pragma unroll
    for (int j = 0; j < kBatch; j++) {
      if (j >= left) break;
      if (turn) turn_pairs<INTERLEAVED>(&u[j].x, &v[j].x, c, s);
      *reinterpret_cast<uint4*>(y + j * a.D + d0) = u[j];
      if (two) *reinterpret_cast<uint4*>(y + j * a.D + d1) = v[j];
    }
  }
}

// The same for sizes and addresses that 16-byte pieces do not fit: a thread has
// one pair, or one dim that does not turn.
template <bool INTERLEAVED>
__global__ void __launch_bounds__(256) k_rope_any(RopeArgs a) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t part = id / a.groups;
  const int g = (int)(id - part * a.groups);
  const int64_t row = part / a.runs;
  if (row >= a.rows) return;
  const int run = (int)(part - row * a.runs);
  const int np = a.rot / 2;
  const bool turn = g < np;
  const int d0 = turn ? (INTERLEAVED ? 2 * g : g) : a.rot + g - np;
  const int d1 = INTERLEAVED ? d0 + 1 : d0 + np;
  float c = 1.f, s = 0.f;
  if (turn) rope_angle(a.turns[g], a.pos[row], a.amplitude, c, s);
  const HeadRun r = head_run(a, row, run);
  const uint16_t* x = r.in;
  uint16_t* y = r.out;
  for (int j = 0; j < r.n; j++, x += a.D, y += a.D) {
    if (turn) {
      const float p = bf2f(x[d0]), q = bf2f(x[d1]);
      y[d0] = f2bf(fmaf(p, c, -q * s));
      y[d1] = f2bf(fmaf(p, s, q * c));
    } else {
      y[d0] = x[d0];
    }
  }
}

static int bad(const char* what) {
  set_error(std::string("sd_rope: ") + what);
  return SD_ERR_INVALID_ARG;
}

}  // namespace sdv

using namespace sdv;

extern "C" int sd_rope_turns_host(int32_t rot_dim, double base, const sd_rope_scaling* scaling, uint64_t* turns,
                                  float* amplitude) {
  auto positive = [](double x) { return x > 0.0 && x <= 1e300; };
  if (!turns || !amplitude) return bad("turns and amplitude must be set");
  if (rot_dim < 2 || rot_dim % 2) return bad("rot_dim must be even and at least 2");
  if (!positive(base)) return bad("base must be positive and finite");
  const sd_rope_scaling none = {SD_ROPE_PLAIN, 1, 1, 1, 2, 0};
  const sd_rope_scaling& s = scaling ? *scaling : none;
  if (s.kind < SD_ROPE_PLAIN || s.kind > SD_ROPE_RAMP) return bad("unknown scaling");
  if (s.kind != SD_ROPE_PLAIN && !positive(s.factor)) return bad("factor must be positive and finite");
  if (s.kind == SD_ROPE_BANDS || s.kind == SD_ROPE_RAMP) {
    if (!positive(s.original) || !positive(s.low) || !positive(s.high)) return bad("original, low and high must be positive and finite");
    if (s.low >= s.high) return bad("low must be below high");
  }
  if (!(s.amplitude <= 1e30)) return bad("amplitude must be finite");
  const double two_pi = 6.283185307179586476925;
  double lo = 0, hi = 0;
  if (s.kind == SD_ROPE_RAMP) {
    if (base == 1.0) return bad("base 1 has one frequency");
    auto pair_of = [&](double t) { return rot_dim * std::log(s.original / (two_pi * t)) / (2 * std::log(base)); };
    lo = std::fmax(std::floor(pair_of(s.high)), 0.0);
    hi = std::fmin(std::ceil(pair_of(s.low)), rot_dim - 1.0);
  }
  for (int i = 0; i < rot_dim / 2; i++) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    if (s.kind == SD_ROPE_LINEAR) {
      f /= s.factor;
    } else if (s.kind == SD_ROPE_BANDS) {
      const double t = s.original * f / two_pi, part = std::fmin(std::fmax((t - s.low) / (s.high - s.low), 0.0), 1.0);
      f = part * f + (1 - part) * f / s.factor;
    } else if (s.kind == SD_ROPE_RAMP) {
      const double part = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
      f = (1 - part) * f + part * f / s.factor;
    }
    if (!positive(f)) return bad("a frequency is not finite");
    const double t = f / two_pi;
    turns[i] = (uint64_t)std::ldexp(t - std::floor(t), 64);  // whole turns drop out: positions are whole
  }
  *amplitude = s.amplitude > 0 ? (float)s.amplitude : s.kind == SD_ROPE_RAMP ? (float)(0.1 * std::log(s.factor) + 1.0) : 1.f;
  return SD_OK;
}

extern "C" int sd_rope(const uint64_t* turns, float amplitude, int32_t head_dim, int32_t rot_dim, int32_t interleaved,
                       const int32_t* pos, int32_t rows, const uint16_t* q, int64_t q_stride, int32_t n_q_heads,
                       uint16_t* q_out, int64_t q_out_stride, const uint16_t* k, int64_t k_stride, int32_t n_kv_heads,
                       uint16_t* k_out, int64_t k_out_stride, void* stream) {
  if (rows < 0 || n_q_heads < 1 || n_q_heads > 65536 || n_kv_heads < 0 || n_kv_heads > 65536)
    return bad("rows >= 0 and 1 .. 65536 query heads (0 .. 65536 key heads) are needed");
  if (head_dim < 1 || head_dim > 1024 || rot_dim < 2 || rot_dim % 2 || rot_dim > head_dim)
    return bad("1 <= head_dim <= 1024 and an even 2 <= rot_dim <= head_dim are needed");
  if (rows == 0) return SD_OK;
  if (!turns || !pos || !q || !q_out || (n_kv_heads && (!k || !k_out)) || (!n_kv_heads && (k || k_out)))
    return bad("null argument, or k without heads");
  const int64_t qn = (int64_t)n_q_heads * head_dim, kn = (int64_t)n_kv_heads * head_dim;
  if (q_stride < qn || q_out_stride < qn || (n_kv_heads && (k_stride < kn || k_out_stride < kn)))
    return bad("a row stride is shorter than the row");
  // an output shares no byte with another tensor, and with its own input all or none
  auto clash = [&](const uint16_t* x, int64_t xs, int64_t xn, const uint16_t* y, int64_t ys, int64_t yn, bool own) {
    if (!x || !y) return false;
    if (own && x == y && (xs == ys || rows == 1)) return false;
    const uintptr_t x0 = (uintptr_t)x, x1 = x0 + 2 * ((uintptr_t)(rows - 1) * xs + xn);
    const uintptr_t y0 = (uintptr_t)y, y1 = y0 + 2 * ((uintptr_t)(rows - 1) * ys + yn);
    if (x1 <= y0 || y1 <= x0) return false;
    if (xs != ys || rows == 1) return true;
    // slices of one tensor's rows: apart where neither reaches the other within a row
    const uintptr_t period = 2 * (uintptr_t)xs, d = y0 >= x0 ? (y0 - x0) % period : (period - (x0 - y0) % period) % period;
    return d < 2 * (uintptr_t)xn || d + 2 * (uintptr_t)yn > period;
  };
  if (clash(q, q_stride, qn, q_out, q_out_stride, qn, true) || clash(k, k_stride, kn, k_out, k_out_stride, kn, true) ||
      clash(q, q_stride, qn, k_out, k_out_stride, kn, false) || clash(k, k_stride, kn, q_out, q_out_stride, qn, false) ||
      clash(q_out, q_out_stride, qn, k_out, k_out_stride, kn, false))
    return bad("an output overlaps a tensor that is not its own input");
  RopeArgs a = {turns, pos, {q, k}, {q_out, k_out}, {q_stride, k_stride}, {q_out_stride, k_out_stride},
                {n_q_heads, n_kv_heads}, rows, rot_dim, head_dim, 0, 0, 0, 0, amplitude};
  const uintptr_t al = (uintptr_t)q | (uintptr_t)q_out | (uintptr_t)k | (uintptr_t)k_out;
  const int64_t st = q_stride | q_out_stride | (n_kv_heads ? k_stride | k_out_stride : 0);
  const bool wide = al % 16 == 0 && st % 8 == 0 && head_dim % 8 == 0 && rot_dim % 16 == 0;
  a.groups = wide ? rot_dim / 16 + (head_dim - rot_dim + 15) / 16 : rot_dim / 2 + head_dim - rot_dim;
  // heads of a thread: eight spread the sines' cost enough (four and 16 take 66 us
  // for the 61 of the kernel's comment, 48 take 74), fewer where eight would leave
  // SMs without a CTA
  const int heads = n_q_heads + n_kv_heads;
  const int64_t threads = (int64_t)rows * a.groups * heads;
  a.each = (int)std::min<int64_t>(8, std::max<int64_t>(1, threads / ((int64_t)num_sms() * 256)));
  a.q_runs = (n_q_heads + a.each - 1) / a.each;
  a.runs = a.q_runs + (n_kv_heads + a.each - 1) / a.each;
  const int64_t blocks = ((int64_t)rows * a.runs * a.groups + 255) / 256;
  if (blocks > 0x7FFFFFFF) return bad("too many rows");
  auto kern = wide ? (interleaved ? k_rope<true> : k_rope<false>) : (interleaved ? k_rope_any<true> : k_rope_any<false>);
  kern<<<(unsigned)blocks, 256, 0, (cudaStream_t)stream>>>(a);
  SD_CK(cudaGetLastError());
  return SD_OK;
}
