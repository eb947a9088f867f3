// The gradient that reaches the router and the layer's input (moe_route_backward), in one launch.
//
// The gates of a token are the softmax over its k selected logits, so with d_j the gradient of gate j
//   dl_j = g_j (d_j - sum_i g_i d_i)
// and, with W_r the router weight, b its bias and x the layer's input,
//   dW_r[e] = sum over (t, j) with id e of dl_j x_t,  db[e] = sum of dl_j,
//   dx_t = sum_j dl_j W_r[id_j] + sum_j rows[at_j]     (the gradients of the token's copies, one per local expert).
//
// Some workgroups take an expert and a piece of H: their waves share the expert's rows, a lane works out the dl of a row,
// and the waves' sums are joined in their order, so that the result does not depend on scheduling.  The others take a token
// for every four waves.  dl is a few operations on 2k numbers: working it out twice costs less than a launch between
// the two (64 tokens: 23 us in two launches).  Bound by memory: rows and dx by HBM, x and W_r mostly by L2:
// 6000 tokens x 8 of 128 experts x 4096, bf16, 126 us (3.9 TB/s), 91 without dW_r and 44 with it alone.
#include "train.h"

namespace {

using train::load_n;
using train::RouteGradArgs;
using train::store_n;

// Columns [64 N piece, 64 N (piece + 1)) of expert e's dW_r, and its db.
template <typename T, int N, int THR>
__device__ __forceinline__ void weight_part(const RouteGradArgs &a, int e, int piece, float *buf) {
  constexpr int kWaves = THR / 64;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = min((piece * 64 + lane) * N, a.H - N);
  int r0, cnt;
  train::clip_rows(a.offsets[e], a.offsets[e + 1], a.T * a.k, r0, cnt);
  const int per = (cnt + kWaves - 1) / kWaves, b = r0 + min(wave * per, cnt), end = min(b + per, r0 + cnt);
  float sum[N], bias = 0.0f;
#pragma unroll
  for (int i = 0; i < N; i++) sum[i] = 0.0f;
  for (int r = b; r < end; r += 64) {
    const int n = min(end - r, 64);
    // lanes behind the last row repeat it with weight zero: what they read belongs to this expert too
    const int t = min(max(a.row_token[r + min(lane, n - 1)], 0), a.T - 1);
    float dot = 0.0f, g = 0.0f, d = 0.0f;
    const float *const gt = a.gates + (size_t)t * a.k, *const dt = a.d_gates + (size_t)t * a.k;
    const int32_t *const it = a.ids + (size_t)t * a.k;
    auto one = [&](float gj, float dj, int id) __attribute__((always_inline)) {
      dot = fmaf(gj, dj, dot);
      if (id == e) g = gj, d = dj;
    };
    if ((a.k & 3) == 0 && (((uintptr_t)a.gates | (uintptr_t)a.d_gates | (uintptr_t)a.ids) & 15) == 0) {
      for (int j = 0; j < a.k; j += 4) {
        const float4 gv = *(const float4 *)(gt + j), dv = *(const float4 *)(dt + j);
        const int4 iv = *(const int4 *)(it + j);
        one(gv.x, dv.x, iv.x);
        one(gv.y, dv.y, iv.y);
        one(gv.z, dv.z, iv.z);
        one(gv.w, dv.w, iv.w);
      }
    } else {
      for (int j = 0; j < a.k; j++) one(gt[j], dt[j], it[j]);
    }
    const float dl = lane < n ? g * (d - dot) : 0.0f;
    bias += dl;
    if (a.dwr) {
      const T *x = (const T *)a.x + h;
#pragma unroll 8
      for (int i = 0; i < n; i++) {
        float v[N];
        const float s = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(dl), i));
        const int at = __builtin_amdgcn_readlane(t, i);
        load_n<N>(x + (size_t)at * a.H, v);
#pragma unroll
        for (int c = 0; c < N; c++) sum[c] = fmaf(s, v[c], sum[c]);
      }
    }
  }
  if (a.dbias && piece == 0) {
    bias = train::wave_sum(bias);
    if (lane == 0) buf[wave] = bias;
    __syncthreads();
    if (threadIdx.x == 0) {
      float s = 0.0f;
      for (int w = 0; w < kWaves; w++) s += buf[w];
      a.dbias[e] = s;
    }
    __syncthreads();
  }
  if (!a.dwr) return;
#pragma unroll
  for (int c = 0; c < N; c++) buf[wave * 64 * N + c * 64 + lane] = sum[c];
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * N; i += THR) {
    const int col = (piece * 64 + (i & 63)) * N + (i >> 6);
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; w++) s += buf[w * 64 * N + i];
    if (col < a.H) a.dwr[(size_t)e * a.H + col] = s;
  }
}

// THR / 256 tokens.
template <typename T, typename TR, typename TO, int N, int THR>
__device__ __forceinline__ void token_part(const RouteGradArgs &a, int block, float *buf) {
  const int sub = threadIdx.x >> 8, tid = threadIdx.x & 255, t = block * (THR / 256) + sub, k = a.k;
  float *const dl = buf + sub * 96;
  int *const id = (int *)dl + 32, *const at = (int *)dl + 64;
  if (tid < 64 && t < a.T) {
    float g = 0.0f, d = 0.0f;
    if (tid < k) g = a.gates[(size_t)t * k + tid], d = a.d_gates[(size_t)t * k + tid];
    const float s = train::wave_sum(g * d);
    if (tid < k) {
      dl[tid] = g * (d - s);
      id[tid] = min(max(a.ids[(size_t)t * k + tid], 0), a.E - 1);
      const int r = a.rows ? a.rows_at[(size_t)t * k + tid] : -1;
      at[tid] = r < a.R_cap ? r : -1;
    }
  }
  __syncthreads();
  if (t >= a.T) return;
  const T *wr = (const T *)a.wr;
  const TR *rows = (const TR *)a.rows;
  const bool have = a.rows && a.R_cap > 0;
  for (int h = tid * N; h < a.H; h += 256 * N) {
    float sum[N];
#pragma unroll
    for (int i = 0; i < N; i++) sum[i] = 0.0f;
    if (have) {  // a row that is not there is read as the first one, and dropped
#pragma unroll 8
      for (int j = 0; j < k; j++) {
        float v[N];
        load_n<N>(rows + (size_t)max(at[j], 0) * a.H + h, v);
#pragma unroll
        for (int i = 0; i < N; i++) sum[i] += at[j] >= 0 ? v[i] : 0.0f;
      }
    }
#pragma unroll 8
    for (int j = 0; j < k; j++) {
      float w[N];
      load_n<N>(wr + (size_t)id[j] * a.H + h, w);
#pragma unroll
      for (int i = 0; i < N; i++) sum[i] = fmaf(dl[j], w[i], sum[i]);
    }
    store_n<N>((TO *)a.dx + (size_t)t * a.H + h, sum);
  }
}

template <typename T, typename TR, typename TO, int N, int THR>
__global__ __launch_bounds__(THR) void route_grad_kernel(RouteGradArgs a, int pieces) {
  __shared__ float buf[THR * N > THR / 256 * 96 ? THR * N : THR / 256 * 96];
  const int b = train::block_of(), weights = a.E * pieces;
  if (b < weights) weight_part<T, N, THR>(a, b / pieces, b % pieces, buf);
  else if (a.dx) token_part<T, TR, TO, N, THR>(a, b - weights, buf);  // without dx: workgroups too many of a last row
}

template <typename T, typename TR, typename TO, int N, int THR>
hipError_t launch(const RouteGradArgs &a, hipStream_t s) {
  const int pieces = a.dwr ? ceil_div_i(a.H, 64 * N) : (a.dbias ? 1 : 0);
  const dim3 grid = train::grid_of(a.E * pieces + (a.dx ? ceil_div_i(a.T, THR / 256) : 0), THR);
  hipLaunchKernelGGL((route_grad_kernel<T, TR, TO, N, THR>), grid, dim3(THR), 0, s, a, pieces);
  return hipGetLastError();
}

// Four waves share an expert's rows, sixteen where there are many a wave: 6000 tokens x 8 of 128 experts 126 us with four, 150
// with sixteen, 2000 tokens 42 and 50; 6000 x 1 of 4 (half of them on one expert) 129 and 41.
template <typename T, typename TR, typename TO>
hipError_t by_size(const RouteGradArgs &a, hipStream_t s) {
  const bool wide = a.H % 8 == 0, many = (long long)a.T * a.k > 1024LL * a.E;
  if (wide) return many ? launch<T, TR, TO, 8, 1024>(a, s) : launch<T, TR, TO, 8, 256>(a, s);
  return many ? launch<T, TR, TO, 1, 1024>(a, s) : launch<T, TR, TO, 1, 256>(a, s);
}

template <typename T, typename TR>
hipError_t by_out(const RouteGradArgs &a, hipStream_t s) {
  return a.dx_bf16 ? by_size<T, TR, uint16_t>(a, s) : by_size<T, TR, float>(a, s);
}
template <typename T>
hipError_t by_rows(const RouteGradArgs &a, hipStream_t s) {
  return a.rows_bf16 ? by_out<T, uint16_t>(a, s) : by_out<T, float>(a, s);
}

}  // namespace

hipError_t train::launch_route_grad(const RouteGradArgs &a, hipStream_t s) {
  return a.bf16 ? by_rows<uint16_t>(a, s) : by_rows<float>(a, s);
}
