// The gradient that reaches the router and the layer's input (moe_route_backward).
//
// The gates of a token are the softmax over its k selected logits, so with d_j the gradient of gate j
//   dl_j = g_j (d_j - sum_i g_i d_i)
// and, with W_r the router weight, b its bias and x the layer's input,
//   dW_r[e] = sum over (t, j) with id e of dl_j x_t,  db[e] = sum of dl_j,
//   dx_t = sum_j dl_j W_r[id_j] + sum_j rows[at_j]     (the gradients of the token's copies, one per local expert).
//
// Launch 1, a workgroup per token: dl to the workspace in the order of the rows grouped by expert, and dx.  Launch 2, a
// workgroup per expert and piece of H: the weighted sum of the expert's token rows in their order, so that the result
// does not depend on scheduling.
#include "train.h"

namespace {

using train::load_n;
using train::RouteGradArgs;
using train::store_n;

constexpr int kThr = 256;

template <typename T, typename TR, typename TO, int N>
__global__ __launch_bounds__(kThr) void token_kernel(RouteGradArgs a) {
  __shared__ float dl[32];
  __shared__ int id[32], at[32];
  const int t = blockIdx.x, tid = threadIdx.x, k = a.k;
  if (tid < 64) {
    float g = 0.0f, d = 0.0f;
    if (tid < k) g = a.gates[(size_t)t * k + tid], d = a.d_gates[(size_t)t * k + tid];
    const float s = train::wave_sum(g * d), l = g * (d - s);
    if (tid < k) {
      dl[tid] = l;
      id[tid] = min(max(a.ids[(size_t)t * k + tid], 0), a.E - 1);
      at[tid] = a.rows ? a.rows_at[(size_t)t * k + tid] : -1;
      if (at[tid] >= a.R_cap) at[tid] = -1;
      if (a.dwr || a.dbias) {
        const int r = a.token_row[(size_t)t * k + tid];
        if (r >= 0 && r < a.T * k) ((float *)a.ws)[r] = l;
      }
    }
  }
  __syncthreads();
  if (!a.dx) return;
  const T *wr = (const T *)a.wr;
  const TR *rows = (const TR *)a.rows;
  for (int h = tid * N; h < a.H; h += kThr * N) {
    float sum[N];
#pragma unroll
    for (int i = 0; i < N; i++) sum[i] = 0.0f;
#pragma unroll 4
    for (int j = 0; j < k; j++) {
      float w[N];
      load_n<N>(wr + (size_t)id[j] * a.H + h, w);
#pragma unroll
      for (int i = 0; i < N; i++) sum[i] = fmaf(dl[j], w[i], sum[i]);
      if (at[j] >= 0) {
        load_n<N>(rows + (size_t)at[j] * a.H + h, w);
#pragma unroll
        for (int i = 0; i < N; i++) sum[i] += w[i];
      }
    }
    store_n<N>((TO *)a.dx + (size_t)t * a.H + h, sum);
  }
}

template <typename T, int N>
__global__ __launch_bounds__(64) void weight_kernel(RouteGradArgs a) {
  const int e = blockIdx.x, h = (blockIdx.y * 64 + threadIdx.x) * N;
  const int r0 = max(a.offsets[e], 0), r1 = min(a.offsets[e + 1], a.T * a.k);
  const float *dl = (const float *)a.ws;
  const T *x = (const T *)a.x;
  if (h < a.H && a.dwr) {
    float sum[N];
#pragma unroll
    for (int i = 0; i < N; i++) sum[i] = 0.0f;
#pragma unroll 8
    for (int r = r0; r < r1; r++) {
      float v[N];
      const int t = min(max(a.row_token[r], 0), a.T - 1);
      const float d = dl[r];
      load_n<N>(x + (size_t)t * a.H + h, v);
#pragma unroll
      for (int i = 0; i < N; i++) sum[i] = fmaf(d, v[i], sum[i]);
    }
    store_n<N>(a.dwr + (size_t)e * a.H + h, sum);
  }
  if (a.dbias && blockIdx.y == 0) {
    float b = 0.0f;
    for (int r = r0 + threadIdx.x; r < r1; r += 64) b += dl[r];
    b = train::wave_sum(b);
    if (threadIdx.x == 0) a.dbias[e] = b;
  }
}

template <typename T, typename TR, typename TO>
hipError_t launch(const RouteGradArgs &a, hipStream_t s) {
  const bool wide = a.H % 8 == 0;
  if (a.T == 0) {
  } else if (wide) hipLaunchKernelGGL((token_kernel<T, TR, TO, 8>), dim3(a.T), dim3(kThr), 0, s, a);
  else hipLaunchKernelGGL((token_kernel<T, TR, TO, 1>), dim3(a.T), dim3(kThr), 0, s, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || (!a.dwr && !a.dbias)) return err;
  if (wide) hipLaunchKernelGGL((weight_kernel<T, 8>), dim3(a.E, ceil_div_i(a.H, 512)), dim3(64), 0, s, a);
  else hipLaunchKernelGGL((weight_kernel<T, 1>), dim3(a.E, ceil_div_i(a.H, 64)), dim3(64), 0, s, a);
  return hipGetLastError();
}

template <typename T, typename TR>
hipError_t by_out(const RouteGradArgs &a, hipStream_t s) {
  return a.dx_bf16 ? launch<T, TR, uint16_t>(a, s) : launch<T, TR, float>(a, s);
}
template <typename T>
hipError_t by_rows(const RouteGradArgs &a, hipStream_t s) {
  return a.rows_bf16 ? by_out<T, uint16_t>(a, s) : by_out<T, float>(a, s);
}

}  // namespace

size_t train::route_grad_ws_bytes(int T, int k, int E, int H) { return align_up((size_t)T * k * sizeof(float), 256); }

hipError_t train::launch_route_grad(const RouteGradArgs &a, hipStream_t s) {
  return a.bf16 ? by_rows<uint16_t>(a, s) : by_rows<float>(a, s);
}
