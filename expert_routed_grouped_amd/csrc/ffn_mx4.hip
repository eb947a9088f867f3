// Grouped expert FFN with MXFP4 weights (moe_grouped_ffn_mx4) for gfx950.
//
// h = Q(silu(G) U), G, U = Wgu a; o = Wd h; y[t] = sum over t's rows of row_w o, in three launches: gate/up,
// down (rows scaled by their gate into the workspace) and the sum to token order, which adds a token's rows
// in slot order, so the result does not depend on scheduling.
#include "mx4_common.h"

namespace {

using ffn::TileParams;
using mx4::v8i_t;

struct Mx4Params {
  TileParams tp;               // offsets, row_token, row_w, El, H, I, R_cap, T; a / w / out: codes (out: rows for down)
  const uint8_t *a_scales;     // [rows, K/32]
  const uint8_t *w_scales;     // packed
  uint8_t *out_scales;         // gate/up: h scales
};

constexpr int SM = 16;  // rows per tile

// One wave: 16 rows of an expert x 32 intermediate columns (gate/up) or 64 output columns (down).
template <int FA, bool DOWN, bool BF16>
__global__ __launch_bounds__(256) void ffn_mx4_simple_kernel(Mx4Params p) {
  const int K = DOWN ? p.tp.I : p.tp.H, Nw = DOWN ? p.tp.H : 2 * p.tp.I;
  constexpr int COLS = DOWN ? 64 : 32;
  const int ncols = DOWN ? p.tp.H : p.tp.I;
  int e, nt, r0, rows;
  if (!ffn::find_tile<SM>(p.tp, (ncols + 4 * COLS - 1) / (4 * COLS), e, nt, r0, rows)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, q = lane >> 4;
  const int c0 = (nt * 4 + wave) * COLS;
  if (c0 >= ncols) return;
  const int r = r0 + min(n, rows - 1);
  const size_t src = DOWN ? (size_t)r : (size_t)p.tp.row_token[r];
  const uint8_t *arow = (const uint8_t *)p.tp.a + src * mx4::code_bytes<FA>(K);
  const uint8_t *srow = p.a_scales + src * (DOWN ? mx4::h_scale_stride(K) : (size_t)(K / 32));
  size_t group[4];
#pragma unroll
  for (int g = 0; g < 4; g++)
    group[g] = ((size_t)e * Nw + c0 + (DOWN ? 16 * g : 16 * (g & 1) + (g >> 1) * p.tp.I)) / 16;
  f32x4_t acc[4];
#pragma unroll
  for (int g = 0; g < 4; g++) acc[g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < K / 128; s++) {
    const v8i_t a = mx4::act_frag<FA>(arow, s, q);
    const uint32_t sa = DOWN ? *(const uint32_t *)(srow + (size_t)(s >> 2) * 16 + 4 * q) >> (8 * (s & 3))
                             : mx4::act_scale(srow, s, q);
#pragma unroll
    for (int g = 0; g < 4; g++) {
      const u32x4_t w = *(const u32x4_t *)((const uint8_t *)p.tp.w + group[g] * mx4::group_codes(K) +
                                           (size_t)s * mx4::kBlk + lane * 16);
      const uint32_t sw = *(const uint32_t *)(p.w_scales + group[g] * mx4::group_scales(K) +
                                              (size_t)(s >> 2) * mx4::kSblk + lane * 4) >> (8 * (s & 3));
      acc[g] = mx4::mfma<FA, 0>(mx4::piece4(w), a, acc[g], sw, sa);
    }
  }
  const bool on = n < rows;
  if constexpr (!DOWN) {
    float v[2][4];
#pragma unroll
    for (int g = 0; g < 2; g++)
#pragma unroll
      for (int i = 0; i < 4; i++) v[g][i] = silu_fast(acc[g][i]) * acc[2 + g][i];
    mx4::store_h_block<FA>(v, on, (uint8_t *)p.tp.out + (size_t)r * mx4::code_bytes<FA>(p.tp.I),
                           p.out_scales + (size_t)r * mx4::h_scale_stride(p.tp.I), c0, q);
  } else if (on) {
    const float w = p.tp.row_w[r];
#pragma unroll
    for (int g = 0; g < 4; g++)
      mx4::store4<BF16>(p.tp.out, (size_t)r * p.tp.H + c0 + 16 * g + 4 * q, acc[g] * w);
  }
}

// y[t] = sum of t's rows in slot order; a slot without a row (or with one out of range) adds nothing.
template <bool BF16>
__global__ __launch_bounds__(256) void sum_rows_kernel(const void *__restrict__ rows, const int32_t *__restrict__ token_row,
                                                       int T, int k, int R_cap, int H, void *__restrict__ y) {
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    for (int c = threadIdx.x * 4; c < H; c += blockDim.x * 4) {
      f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
      for (int j = 0; j < k; j++) {
        const int r = token_row[(size_t)t * k + j];
        if ((unsigned)r >= (unsigned)R_cap) continue;
        const size_t i = (size_t)r * H + c;
        if constexpr (BF16) {
          const uint2 v = *(const uint2 *)((const uint16_t *)rows + i);
          acc += f32x4_t{bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
        } else {
          acc += *(const f32x4_t *)((const float *)rows + i);
        }
      }
      mx4::store4<BF16>(y, (size_t)t * H + c, acc);
    }
  }
}

// Workspace: h codes [R_cap, I] (a byte each, half of it used by E2M1), h scales, rows [R_cap, H].
size_t h_bytes(int R_cap, int I) { return align_up((size_t)R_cap * I, 256); }
size_t hs_bytes(int R_cap, int I) { return align_up((size_t)R_cap * mx4::h_scale_stride(I), 256); }

template <int FA, bool BF16>
hipError_t launch(const FfnMx4Args &a, hipStream_t s) {
  uint8_t *h = (uint8_t *)a.ws, *hs = h + h_bytes(a.R_cap, a.I), *rows = hs + hs_bytes(a.R_cap, a.I);
  if (a.R_cap > 0) {
    Mx4Params p{};
    p.tp.offsets = a.offsets;
    p.tp.row_token = a.row_token;
    p.tp.row_w = a.row_w;
    p.tp.El = a.El;
    p.tp.H = a.H;
    p.tp.I = a.I;
    p.tp.R_cap = a.R_cap;
    p.tp.T = a.T;
    const long long mt1 = ((long long)a.R_cap + (long long)a.El * (SM - 1)) / SM;
    const long long mt2 = (long long)a.El * ceil_div_i(a.T, SM);
    const int mt = (int)(mt1 < mt2 ? mt1 : mt2);
    Mx4Params g = p;
    g.tp.a = a.a;
    g.a_scales = a.a_s;
    g.tp.w = a.wgu;
    g.w_scales = a.wgu_s;
    g.tp.out = h;
    g.out_scales = hs;
    hipLaunchKernelGGL((ffn_mx4_simple_kernel<FA, false, BF16>), dim3(mt * ceil_div_i(a.I, 128)), dim3(256), 0, s, g);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    Mx4Params d = p;
    d.tp.a = h;
    d.a_scales = hs;
    d.tp.w = a.wd;
    d.w_scales = a.wd_s;
    d.tp.out = rows;
    hipLaunchKernelGGL((ffn_mx4_simple_kernel<FA, true, BF16>), dim3(mt * ceil_div_i(a.H, 256)), dim3(256), 0, s, d);
    err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  hipLaunchKernelGGL(sum_rows_kernel<BF16>, dim3(a.T < 16384 ? a.T : 16384), dim3(256), 0, s, rows, a.token_row, a.T,
                     a.k, a.R_cap, a.H, a.y);
  return hipGetLastError();
}

}  // namespace

size_t ffn_mx4_ws_bytes(int R_cap, int H, int I, int y_bf16) {
  return h_bytes(R_cap, I) + hs_bytes(R_cap, I) + align_up((size_t)R_cap * H * (y_bf16 ? 2 : 4), 256);
}

hipError_t launch_ffn_mx4(const FfnMx4Args &a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  if (a.T <= kMx4StreamMaxT) {
    uint8_t *h = (uint8_t *)a.ws;
    return launch_ffn_mx4_stream(a, h, h + h_bytes(a.R_cap, a.I), s);
  }
  if (a.a_fp4) return a.y_bf16 ? launch<mx4::FP4, true>(a, s) : launch<mx4::FP4, false>(a, s);
  return a.y_bf16 ? launch<mx4::FP8, true>(a, s) : launch<mx4::FP8, false>(a, s);
}
