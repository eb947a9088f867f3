// The tiles of rows grouped by expert, shared by the kernels of moe_grouped_mm.
#pragma once
#include "ffn_common.h"
#include "train.h"

namespace train {

// The tiles of a product: expert e has ceil(c_e / BM) tiles of rows, its c_e rows split evenly over them (rounded up to 64), times
// NT tiles of columns, numbered expert by expert, then by columns, then by rows.  A lane holds how many tiles the experts
// up to its group of G have, so that a tile is found with one ballot and at most G scalar loads.
struct MmTile {
  int nt, r0, rows, trows;
  bool once;  // the expert's only tile of rows: its matrix is read once
  const void *w;
};
template <typename C, int ESZ = 2>
struct MmTiles {
  const __attribute__((address_space(4))) int *off;
  int El, R_cap, NT, G, upto, total;
  // Rows of an expert that lie in the buffers, whatever the offsets say.
  static __device__ __forceinline__ int rows_in(int a, int b, int R_cap) { return max(min(b, R_cap) - max(a, 0), 0); }
  __device__ __forceinline__ int of(int e) const {
    return (rows_in(off[e], off[e + 1], R_cap) + C::BM - 1) / C::BM * NT;
  }
  __device__ __forceinline__ MmTiles(const MmArgs &p, int lane) {
    off = (const __attribute__((address_space(4))) int *)(uintptr_t)p.offsets;
    El = p.El;
    R_cap = p.R_cap;
    NT = (p.N + C::BN - 1) / C::BN;
    G = (El + 63) / 64;
    int n = 0;
    for (int i = 0; i < G; i++) {
      const int e = lane * G + i;
      if (e < El) n += (rows_in(p.offsets[e], p.offsets[e + 1], R_cap) + C::BM - 1) / C::BM * NT;
    }
    upto = ffn::wave_incl_scan_i(n, lane);
    total = __builtin_amdgcn_readlane(upto, 63);
  }
  // Tile L < total.
  __device__ __forceinline__ MmTile at(int L, const MmArgs &p) const {
    const int g = __ffsll((long long)__ballot(upto > L)) - 1;
    int before = g == 0 ? 0 : __builtin_amdgcn_readlane(upto, g - 1), e = g * G;
    for (int n = of(e); L >= before + n; n = of(e)) before += n, e++;
    const int beg = max(off[e], 0), cnt = rows_in(beg, off[e + 1], R_cap), mtiles = (cnt + C::BM - 1) / C::BM, rr = L - before;
    MmTile t;
    t.nt = rr / mtiles;
    t.trows = min(C::BM, ((cnt + mtiles - 1) / mtiles + 63) & ~63);
    t.r0 = beg + (rr - t.nt * mtiles) * t.trows;
    t.once = mtiles == 1;
    t.rows = min(t.trows, beg + cnt - t.r0);
    t.w = (const char *)p.w + (size_t)e * p.N * p.K * ESZ;
    return t;
  }
};

}  // namespace train
