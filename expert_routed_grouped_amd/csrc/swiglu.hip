// SwiGLU between two grouped projections, and its gradient (moe_swiglu, moe_swiglu_backward).
//
//   h = w_r silu(g) u,  silu(g) = g s, s = 1 / (1 + exp(-g))
//   dg = w_r dh u s (1 + g (1 - s)),  du = w_r dh silu(g),  dw_r = sum over the row of dh silu(g) u
//
// The gate w_r multiplies h rather than the expert's output, which is the same sum (the down projection is linear) and
// leaves the weight's gradient to this kernel: no row of expert outputs has to be kept or scaled.
//
// One wave per row, 16 bytes a lane and step; the sum of a row stays in its wave.  Bound by memory: three values per
// element forward, six backward (g, u, dh read; dg, du, h written).  48000 rows of 1536 in bf16: 88 us forward (5.0 TB/s), 153
// backward (5.8).
#include "train.h"

namespace {

using train::load_n;
using train::store_n;
using train::SwigluArgs;

template <bool EXACT>
__device__ __forceinline__ float sigmoid(float g) {
  // fp32 results keep expf (its argument is not rounded); results that are rounded to bf16 take the hardware exp2
  if constexpr (EXACT) return 1.0f / (1.0f + expf(-g));
  else return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * g));
}

constexpr int kWaves = 4;

template <typename T, int N>
__global__ __launch_bounds__(kWaves * 64) void swiglu_kernel(SwigluArgs a) {
  constexpr bool EXACT = sizeof(T) == 4;
  const int R = a.offsets ? min(a.offsets[a.El], a.R_cap) : a.R_cap, lane = threadIdx.x & 63;
  const int r = train::block_of() * kWaves + (threadIdx.x >> 6);
  if (r >= R) return;
  const T *g = (const T *)a.gu + (size_t)r * 2 * a.I, *u = g + a.I;
  T *h = (T *)a.h + (size_t)r * a.I;
  const float w = a.row_w ? a.row_w[r] : 1.0f;
#pragma unroll 2
  for (int i = lane * N; i < a.I; i += 64 * N) {
    float gv[N], uv[N];
    load_n<N>(g + i, gv);
    load_n<N>(u + i, uv);
#pragma unroll
    for (int j = 0; j < N; j++) gv[j] = gv[j] * sigmoid<EXACT>(gv[j]) * uv[j] * w;
    store_n<N>(h + i, gv);
  }
}

template <typename T, int N>
__global__ __launch_bounds__(kWaves * 64) void swiglu_backward_kernel(SwigluArgs a) {
  constexpr bool EXACT = sizeof(T) == 4;
  const int R = a.offsets ? min(a.offsets[a.El], a.R_cap) : a.R_cap, lane = threadIdx.x & 63;
  const int r = train::block_of() * kWaves + (threadIdx.x >> 6);
  if (r >= R) return;
  const T *g = (const T *)a.gu + (size_t)r * 2 * a.I, *u = g + a.I, *dh = (const T *)a.dh + (size_t)r * a.I;
  T *dg = (T *)a.dgu + (size_t)r * 2 * a.I, *du = dg + a.I, *h = a.h ? (T *)a.h + (size_t)r * a.I : nullptr;
  const float w = a.row_w ? a.row_w[r] : 1.0f;
  float sum = 0.0f;
#pragma unroll 2
  for (int i = lane * N; i < a.I; i += 64 * N) {
    float gv[N], uv[N], dv[N], hv[N];
    load_n<N>(g + i, gv);
    load_n<N>(u + i, uv);
    load_n<N>(dh + i, dv);
#pragma unroll
    for (int j = 0; j < N; j++) {
      const float s = sigmoid<EXACT>(gv[j]), si = gv[j] * s, act = si * uv[j], d = dv[j] * w;
      sum = fmaf(dv[j], act, sum);
      hv[j] = act * w;
      const float dgate = d * uv[j] * (s * (1.0f + gv[j] * (1.0f - s)));
      uv[j] = d * si;
      gv[j] = dgate;
    }
    store_n<N>(dg + i, gv);
    store_n<N>(du + i, uv);
    if (h) store_n<N>(h + i, hv);
  }
  if (a.d_row_w) {
    sum = train::wave_sum(sum);
    if (lane == 0) a.d_row_w[r] = sum;
  }
}

template <typename T, int N>
hipError_t launch(const SwigluArgs &a, bool backward, hipStream_t s) {
  const dim3 grid = train::grid_of(ceil_div_i(a.R_cap, kWaves), kWaves * 64), block(kWaves * 64);
  if (backward) hipLaunchKernelGGL((swiglu_backward_kernel<T, N>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((swiglu_kernel<T, N>), grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t pick(const SwigluArgs &a, bool backward, hipStream_t s) {
  if (a.bf16) return a.I % 8 == 0 ? launch<uint16_t, 8>(a, backward, s) : launch<uint16_t, 1>(a, backward, s);
  return a.I % 4 == 0 ? launch<float, 4>(a, backward, s) : launch<float, 1>(a, backward, s);
}

}  // namespace

hipError_t train::launch_swiglu(const SwigluArgs &a, hipStream_t s) { return pick(a, false, s); }
hipError_t train::launch_swiglu_backward(const SwigluArgs &a, hipStream_t s) { return pick(a, true, s); }
