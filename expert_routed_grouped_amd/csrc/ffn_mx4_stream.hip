// MXFP4 grouped expert FFN of a small batch: the weight-streaming halves of mx4_stream.h, two launches.
#include "mx4_stream.h"

namespace {

using ffn::TileParams;

// Workgroup b: NW / S neighbouring column blocks of one tile, S waves each.
template <int FA>
__global__ __launch_bounds__(mx4s::NTHR, 2) void gate_up_stream_kernel(TileParams p, mx4s::Half w, uint8_t *h,
                                                                       uint8_t *hs, int S) {
  extern __shared__ __attribute__((aligned(16))) float red[];  // RED_FLOATS if S > 1
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), per = mx4s::NW / S;
  int e, nt, r0, rows;
  if (!ffn::find_tile<mx4s::TM>(p, (p.I / 32 + per - 1) / per, e, nt, r0, rows)) return;
  e = __builtin_amdgcn_readfirstlane(e);  // the same in every lane: keep them scalar
  r0 = __builtin_amdgcn_readfirstlane(r0);
  const int cb = __builtin_amdgcn_readfirstlane(nt) * per + wave / S;
  rows = cb * 32 < p.I ? __builtin_amdgcn_readfirstlane(rows) : 0;
  mx4s::gate_up_tile<FA>(
      w, p.H, p.I, e, cb * 32, r0, rows, S, wave & (S - 1),
      [&](int r) { return (size_t)min((unsigned)p.row_token[r], (unsigned)p.T - 1u); }, h, hs, red);
}

template <int FA>
hipError_t launch(const FfnMx4Args &a, uint8_t *h, uint8_t *hs, hipStream_t s) {
  TileParams p{};
  p.offsets = a.offsets;
  p.row_token = a.row_token;
  p.El = a.El;
  p.H = a.H;
  p.I = a.I;
  p.R_cap = a.R_cap;
  p.T = a.T;
  // tiles: at most one per row, and one per expert plus the full ones
  const long long t1 = ((long long)a.R_cap + (long long)a.El * (mx4s::TM - 1)) / mx4s::TM;
  const int tiles = (int)(t1 < a.R_cap ? t1 : a.R_cap);
  const int S = mx4s::split_for((a.R_cap < a.El ? a.R_cap : a.El) * (a.I / 32), a.H);
  hipLaunchKernelGGL(gate_up_stream_kernel<FA>, dim3(tiles * ceil_div_i(a.I / 32, mx4s::NW / S)), dim3(mx4s::NTHR),
                     S > 1 ? mx4s::RED_FLOATS * sizeof(float) : 0, s, p, (mx4s::Half{a.a, a.a_s, a.wgu, a.wgu_s}), h, hs,
                     S);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  return launch_down_sum_mx4(a, h, hs, s);
}

template <int FA, bool BF16>
hipError_t launch_down(const FfnMx4Args &a, const uint8_t *h, const uint8_t *hs, hipStream_t s) {
  mx4s::DownArgs d{a.offsets, a.row_token, a.row_w, a.El, a.T, a.R_cap, a.H, a.I, {h, hs, a.wd, a.wd_s}, a.y, a.tiles, a.ntiles,
                   a.zero, a.n_zero};
  hipLaunchKernelGGL((mx4s::down_sum_kernel<FA, BF16>), dim3(a.H / 16), dim3(mx4s::NTHR),
                     mx4s::down_lds_bytes<FA>(a.T, a.El, a.R_cap), s, d);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_down_sum_mx4(const FfnMx4Args &a, const uint8_t *h, const uint8_t *hs, hipStream_t s) {
  if (a.a_fp4) return a.y_bf16 ? launch_down<mx4::FP4, true>(a, h, hs, s) : launch_down<mx4::FP4, false>(a, h, hs, s);
  return a.y_bf16 ? launch_down<mx4::FP8, true>(a, h, hs, s) : launch_down<mx4::FP8, false>(a, h, hs, s);
}

hipError_t launch_ffn_mx4_stream(const FfnMx4Args &a, uint8_t *h, uint8_t *hs, hipStream_t s) {
  if (a.a_fp4) return launch<mx4::FP4>(a, h, hs, s);
  return launch<mx4::FP8>(a, h, hs, s);
}
