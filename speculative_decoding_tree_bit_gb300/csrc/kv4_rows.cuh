// Which rows of a request each tile of the tensor-core attention over the
// 4-bit cache works on.  Plain integer arithmetic, for the host as well.
#pragma once

#ifdef __CUDACC__
#define SDV_HD __host__ __device__ __forceinline__
#else
#define SDV_HD inline
#endif

namespace sdv {

SDV_HD int least(int a, int b) { return a < b ? a : b; }

// Rows of a segment: a request's G m rows in nc even runs.  Tile t holds `of(t)`
// of them from row first(t) on, `copies` times, 128 / copies lanes apart.
template <bool WIDE>
struct TcRowsOf {
  int base, rows, split, copies, run;
  SDV_HD TcRowsOf(int gm, int nc, int rc) {
    run = ((gm + nc - 1) / nc + 31) / 32 * 32;
    base = rc * run;
    rows = least(run, gm - base);
    split = WIDE ? least(rows, (rows / 2 + 31) / 32 * 32) : rows;
    copies = WIDE || rows > 64 ? 1 : rows > 32 ? 2 : 4;
  }
  SDV_HD int of(int t) const { return !WIDE || t == 0 ? split : rows - split; }
  SDV_HD int first(int t) const { return base + (!WIDE || t == 0 ? 0 : split); }
  // The request's row whose data index ridx of tile t loads: its own, or the
  // segment's first where it has none (a tile may have no rows at all, and the
  // row after a request's last belongs to a query head past the array).
  SDV_HD int row(int t, int ridx) const { return ridx < of(t) ? first(t) + ridx : base; }
};

}  // namespace sdv
