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
  __device__ __forceinline__ int tiles_of(int begin, int end) const {
    int r0, rows;
    clip_rows(begin, end, R_cap, r0, rows);
    return (rows + C::BM - 1) / C::BM * NT;
  }
  __device__ __forceinline__ int of(int e) const { return tiles_of(off[e], off[e + 1]); }
  __device__ __forceinline__ MmTiles(const MmArgs &p, int lane) {
    off = (const __attribute__((address_space(4))) int *)(uintptr_t)p.offsets;
    El = p.El;
    R_cap = p.R_cap;
    NT = (p.N + C::BN - 1) / C::BN;
    G = (El + 63) / 64;
    // Offsets that do not ascend name rows more than once: sums stop at kMost instead of wrapping, and no more tiles are taken
    // than ascending ones can have.
    constexpr uint32_t kMost = 0x7fffffffu;
    uint32_t n = 0;
    for (int i = 0; i < G; i++) {
      const int e = lane * G + i;
      if (e < El) n = min(n + (uint32_t)tiles_of(p.offsets[e], p.offsets[e + 1]), kMost);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t before = __shfl_up(n, o, 64);
      if (lane >= o) n = min(n + before, kMost);
    }
    upto = (int)n;
    total = min(__builtin_amdgcn_readlane(upto, 63), min((R_cap + El * (C::BM - 1)) / C::BM, R_cap) * NT);
  }
  // Tile L < total.
  __device__ __forceinline__ MmTile at(int L, const MmArgs &p) const {
    const int g = __ffsll((long long)__ballot(upto > L)) - 1;
    int before = g == 0 ? 0 : __builtin_amdgcn_readlane(upto, g - 1), e = g * G;
    for (int n = of(e); L - before >= n; n = of(e)) before += n, e++;
    int beg, cnt;
    clip_rows(off[e], off[e + 1], R_cap, beg, cnt);
    const int mtiles = (cnt + C::BM - 1) / C::BM, rr = L - before;
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
