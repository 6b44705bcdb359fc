// The 4-bit key/value cache: layout and the helpers its kernels share.
//
// Slots come in groups of 32.  The record of a group, for one kv head of D
// dims, is one run of 32 D + 256 bytes:
//   K codes [32][D/2] | K (s, m) [32] | V codes [32][D/2] | V (s, m) [32]
// A slot's codes lie in dim order, two a byte, the lower nibble first; with D
// = 128 the two 32-byte halves of a V row are exchanged in the slots whose
// bit 1 is set, so that the attention kernel's reads of four keys at once
// fall into different shared-memory banks.  (s, m): scale and middle as a
// bf16 pair, s in the lower half.  A record is one contiguous bulk copy, its
// K part (the first half) another.
#pragma once

#include "common.cuh"

namespace sdv {

constexpr int kKvGroup = 32;  // slots of a record

__host__ __device__ constexpr int kv4_rec(int D) { return 32 * D + 256; }
__host__ __device__ constexpr int kv4_half(int D) { return 16 * D + 128; }  // the K part; V codes follow

struct Kv4View {
  uint8_t* blocks;   // [n_pages][hkv][groups per page][record]
  int32_t* pos;      // [R][hkv][cap]
  float* weight;     // [R][hkv][cap]
  const int32_t* page_table;  // [R][max_pages]
  int32_t* ctx_len;  // [R]
  int32_t n_pages, gpp, hkv, max_pages;  // gpp: groups per page
  int64_t cap;       // slots a request can hold

  // record of group g of request r and kv head h; null where the page table
  // has no page of the pool
  __device__ __forceinline__ uint8_t* record(int D, int r, int h, int g) const {
    const int pi = g / gpp;
    const int page = page_table[(int64_t)r * max_pages + pi];
    if (page < 0 || page >= n_pages) return nullptr;
    return blocks + (((int64_t)page * hkv + h) * gpp + (g - pi * gpp)) * kv4_rec(D);
  }
  __device__ __forceinline__ int64_t slot0(int r, int h) const { return ((int64_t)r * hkv + h) * cap; }
};

// Byte of code pair `b` (dims 2b, 2b + 1) within the V row of slot t.
template <int D>
__device__ __forceinline__ int kv4_vbyte(int t, int b) {
  return D == 128 ? b ^ ((t & 2) << 4) : b;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

// The request of row e, by the whole warp: a search 32 offsets at a time.
__device__ __forceinline__ int request_of(const int32_t* __restrict__ cu, int R, int e) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = R;  // cu[lo] <= e < cu[hi]
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, x = lo + lane * step;
    const int n = __popc(__ballot_sync(0xffffffffu, x < hi && cu[x] <= e));
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// Pairs of fp32 values: one instruction for two.
__device__ __forceinline__ uint64_t f2pack(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void f2unpack(uint64_t r, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r));
}
__device__ __forceinline__ uint64_t f2fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// What the scores of a call go by.
struct Kv4Score {
  float scale, cap;        // cap 0: none
  const float* slopes;     // [hq] or null
  int32_t window;          // 0: none
  const int32_t* start;    // [R] or null
};

// The least position that a row at position p0 or later sees.
__device__ __forceinline__ int64_t kv4_since(const Kv4Score& s, int r, int p0) {
  int64_t since = s.window > 0 ? (int64_t)p0 - s.window + 1 : INT64_MIN;
  if (s.start) since = max(since, (int64_t)s.start[r]);
  return since;
}

// First slot that rows at position p0 or later can see in any kv head, or one
// before it: positions do not fall from slot to slot, so the slots before one
// whose predecessor is hidden are hidden too.  The guess is right where
// positions count up one by one to p0 or the row before it: one load a head
// confirms it, and where it fails (rows cached already, positions past the
// rows') the slot goes back in growing steps until a load does.
__device__ __forceinline__ int kv4_guess(const Kv4Score& s, int r, int ctx, int p0) {
  int64_t n = ctx;
  if (s.window > 0) n = min(n, (int64_t)s.window);
  if (s.start) n = min(n, max((int64_t)0, (int64_t)p0 - s.start[r] + 1));
  return ctx - (int)n;
}
__device__ __forceinline__ int kv4_back(const int32_t* __restrict__ pos, int f, int64_t since) {
  for (int step = kKvGroup; f > 0 && pos[f - 1] >= since; step *= 2) f = max(0, f - step);
  return f;
}
// By a lane for a request of its own ...
__device__ __forceinline__ int kv4_first_lane(const Kv4View& c, const Kv4Score& s, int r, int ctx, int p0) {
  const int f = kv4_guess(s, r, ctx, p0);
  const int64_t since = kv4_since(s, r, p0);
  bool bad = false;
  if (f > 0) {
#pragma unroll 8
    for (int h = 0; h < c.hkv; h++) bad |= c.pos[c.slot0(r, h) + f - 1] >= since;
  }
  int first = f;
  if (bad)
    for (int h = 0; h < c.hkv; h++) first = min(first, kv4_back(c.pos + c.slot0(r, h), f, since));
  return first;
}
// ... and, the same, by a whole warp for one request.
__device__ __forceinline__ int kv4_first(const Kv4View& c, const Kv4Score& s, int r, int ctx, int p0) {
  const int f = kv4_guess(s, r, ctx, p0);
  const int64_t since = kv4_since(s, r, p0);
  int first = f;
  for (int h = threadIdx.x & 31; h < c.hkv; h += 32) first = min(first, kv4_back(c.pos + c.slot0(r, h), f, since));
  return __reduce_min_sync(0xffffffffu, first);
}

int kv4_check(const sd_kv4* c, int32_t R, const char* who, Kv4View* view);
int kv4_check_rows(const int32_t* cu, const int32_t* cu_host, int32_t R, const char* who);
int kv4_bad(int code, const char* who, const char* what);
int kv4_check_score(const sd_kv4_score* sc, const char* who, Kv4Score* out, int head_dim);

}  // namespace sdv
