// Residual, gate and the RMS norms around a block (moe_block_norm, moe_block_norm_backward).
//
//   u = rms(y) w_post (or y),  x' = scale x + gate u,  n = rms(x') w_next,  rms(v) = v / sqrt(mean v^2 + eps)
//
// Backward, with r and rp the reciprocal roots, xh = x' r, yh = y rp, H the row's length:
//   D  = dx' + r (dn w_next - xh c / H),  c = sum dn w_next xh          dx = scale D
//   dv = gate D w_post,  dy = rp (dv - yh q / H),  q = sum dv yh
//   dw_next = sum_t dn xh,  dw_post = sum_t gate D yh,  dgate = sum D u (over the tokens or over the row)
// q follows from sums over dx' + r dn w_next and over xh apart, so that one reduction gives c and q:
//   q = sum gate w_post yh (dx' + r dn w_next) - (r c / H) sum gate w_post yh xh.
//
// A workgroup holds a row in registers: every array is read once.  The column sums of the backward pass are kept per
// workgroup over its rows and joined by a second launch, in a fixed order.  Bound by memory: 6000 x 4096, bf16 and an fp32 y, 39 to 46 us
// forward (6.3 to 5.3 TB/s), 79 backward (5.0).  Rows of more than 8192 values (odd ones: 4096) do not fit in the backward pass's registers
// and spill, odd ones of more than 8192 in the forward pass too: 3000 x 16384 100 and 543 us, 3000 x 16383 3310 and 1730.
#include "train.h"

#include <type_traits>

namespace {

using train::load_n;
using train::NormArgs;
using train::store_n;

// Sums of M values over a workgroup of W waves, the same in every thread.  ``buf`` holds 2 * M * W floats, its
// halves used in turn, so that one barrier per sum is enough.
template <int M, int W>
__device__ __forceinline__ void block_sum(float (&v)[M], float *buf, int half) {
#pragma unroll
  for (int m = 0; m < M; m++) v[m] = train::wave_sum(v[m]);
  if constexpr (W > 1) {
    float *b = buf + half * M * W;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int m = 0; m < M; m++) b[m * W + (threadIdx.x >> 6)] = v[m];
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < M; m++) {
      v[m] = 0.0f;
#pragma unroll
      for (int w = 0; w < W; w++) v[m] += b[m * W + w];
    }
  }
}

// Values of a type that the launch tells (weights and gates: fp32 or bf16).
template <int N>
__device__ __forceinline__ void load_w(const void *p, int bf16, size_t i, float (&v)[N]) {
  if (bf16) load_n<N>((const uint16_t *)p + i, v);
  else load_n<N>((const float *)p + i, v);
}
__device__ __forceinline__ float one_w(const void *p, int bf16, size_t i) {
  return bf16 ? bf16_to_f32(((const uint16_t *)p)[i]) : ((const float *)p)[i];
}

// W waves a row, NV pieces of N values a thread.
template <typename TX, typename TY, int W, int NV, int N>
__global__ __launch_bounds__(W * 64) void block_norm_kernel(NormArgs a) {
  __shared__ float buf[2 * W];
  const int t = train::block_of(), H = a.H;
  if (t >= a.T) return;
  const size_t row = (size_t)t * H;
  float x[NV][N], y[NV][N];
#pragma unroll
  for (int v = 0; v < NV; v++) {
    const int h = (v * W * 64 + threadIdx.x) * N;
#pragma unroll
    for (int i = 0; i < N; i++) x[v][i] = 0.0f, y[v][i] = 0.0f;
    if (h < H) {
      load_n<N>((const TX *)a.x + row + h, x[v]);
      if (a.y) load_n<N>((const TY *)a.y + row + h, y[v]);
    }
  }
  if (a.y) {
    float rp = 1.0f;
    if (a.w_post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int v = 0; v < NV; v++)
#pragma unroll
        for (int i = 0; i < N; i++) s[0] = fmaf(y[v][i], y[v][i], s[0]);
      block_sum<1, W>(s, buf, 0);
      rp = 1.0f / sqrtf(s[0] / (float)H + a.eps);
      if (a.rstd_post && threadIdx.x == 0) a.rstd_post[t] = rp;
    }
    const float gt = a.gate_kind == train::kGateToken ? one_w(a.gate, a.w_bf16, t) : 1.0f;
#pragma unroll
    for (int v = 0; v < NV; v++) {
      const int h = (v * W * 64 + threadIdx.x) * N;
      if (h < H) {
        float f[N];
        if (a.w_post) {
          load_w<N>(a.w_post, a.w_bf16, h, f);
#pragma unroll
          for (int i = 0; i < N; i++) y[v][i] = y[v][i] * rp * f[i];
        }
        if (a.gate_kind == train::kGateChannel) {
          load_w<N>(a.gate, a.w_bf16, h, f);
#pragma unroll
          for (int i = 0; i < N; i++) y[v][i] *= f[i];
        }
#pragma unroll
        for (int i = 0; i < N; i++) x[v][i] = fmaf(a.scale, x[v][i], gt * y[v][i]);
        if (a.x_out) store_n<N>((TX *)a.x_out + row + h, x[v]);
      }
    }
  }
  if (!a.n && !a.rstd_next) return;
  float s[1] = {0.0f};
#pragma unroll
  for (int v = 0; v < NV; v++)
#pragma unroll
    for (int i = 0; i < N; i++) s[0] = fmaf(x[v][i], x[v][i], s[0]);
  block_sum<1, W>(s, buf, 1);
  const float r = 1.0f / sqrtf(s[0] / (float)H + a.eps);
  if (a.rstd_next && threadIdx.x == 0) a.rstd_next[t] = r;
  if (!a.n) return;
#pragma unroll
  for (int v = 0; v < NV; v++) {
    const int h = (v * W * 64 + threadIdx.x) * N;
    if (h < H) {
      float f[N];
      load_w<N>(a.w_next, a.w_bf16, h, f);
#pragma unroll
      for (int i = 0; i < N; i++) f[i] *= x[v][i] * r;
      store_n<N>((TX *)a.n + row + h, f);
    }
  }
}

// N values as they lie in memory, loaded now and looked at later.
template <typename T, int N>
struct Raw {
  static constexpr int Q = N == 1 ? 1 : N * (int)sizeof(T) / 16;
  std::conditional_t<N == 1, T, u32x4_t> v[Q];
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (N == 1) v[0] = *p;
    else {
#pragma unroll
      for (int i = 0; i < Q; i++) v[i] = ((const u32x4_t *)p)[i];
    }
  }
  __device__ __forceinline__ void get(float (&f)[N]) const {
    if constexpr (N == 1) f[0] = train::to_f32(v[0]);
    else {
#pragma unroll
      for (int i = 0; i < Q; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
          if constexpr (sizeof(T) == 4) f[4 * i + j] = __uint_as_float(v[i][j]);
          else f[8 * i + 2 * j] = bf16_lo(v[i][j]), f[8 * i + 2 * j + 1] = bf16_hi(v[i][j]);
        }
    }
  }
};

// Partial column sums of one workgroup: dw_next, dw_post and a channel gate's, [3][H] each.  The next row's values are on
// their way while a row is summed, and the weights stay in registers (6000 x 4096, bf16 and an fp32 y: 99 us without, 85), where a
// thread has one piece of a row; with more there are not enough registers for it.
template <typename TX, typename TY, typename TD, int W, int NV, int N>
__global__ __launch_bounds__(W * 64) void block_norm_backward_kernel(NormArgs a) {
  __shared__ float buf[2 * 3 * W];
  const int H = a.H, tid = threadIdx.x;
  const bool channel = a.gate_kind == train::kGateChannel;
  constexpr bool HOLD = NV * N <= 8;
  float dwn[NV][N], dwp[NV][N], dgc[NV][N], wn[HOLD ? NV : 1][N], wp[HOLD ? NV : 1][N], gc[HOLD ? NV : 1][N];
  auto weights = [&](int v, int h) __attribute__((always_inline)) {  // of piece v, into its place (or the one there is)
    const int at = HOLD ? v : 0;
#pragma unroll
    for (int i = 0; i < N; i++) wn[at][i] = wp[at][i] = gc[at][i] = 1.0f;
    if (h < H) {
      if (a.dn) load_w<N>(a.w_next, a.w_bf16, h, wn[at]);
      if (a.w_post) load_w<N>(a.w_post, a.w_bf16, h, wp[at]);
      if (channel) load_w<N>(a.gate, a.w_bf16, h, gc[at]);
    }
  };
#pragma unroll
  for (int v = 0; v < NV; v++) {
    if constexpr (HOLD) weights(v, (v * W * 64 + tid) * N);
#pragma unroll
    for (int i = 0; i < N; i++) dwn[v][i] = 0.0f, dwp[v][i] = 0.0f, dgc[v][i] = 0.0f;
  }
  Raw<TX, N> rx[NV], rdn[NV], rds[NV];
  Raw<TY, N> ry[NV];
  float rn = 0.0f, rp = 1.0f, gt = 1.0f;
  auto fetch = [&](int t) __attribute__((always_inline)) {
    const size_t row = (size_t)t * H;
#pragma unroll
    for (int v = 0; v < NV; v++) {
      const int h = (v * W * 64 + tid) * N;
      if (h < H) {
        if (a.dx_out) rds[v].load((const TX *)a.dx_out + row + h);
        if (a.dn) rx[v].load((const TX *)a.x + row + h), rdn[v].load((const TX *)a.dn + row + h);
        if (a.y) ry[v].load((const TY *)a.y + row + h);
      }
    }
    if (a.dn) rn = a.rn[t];
    if (a.w_post) rp = a.rp[t];
    if (a.gate_kind == train::kGateToken) gt = one_w(a.gate, a.w_bf16, t);
  };
  int half = 0;
  if (HOLD && (int)blockIdx.x < a.T) fetch(blockIdx.x);
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, half ^= 1) {
    if constexpr (!HOLD) fetch(t);
    const size_t row = (size_t)t * H;
    const float rnt = rn, rpt = rp, gtt = gt;
    float xh[NV][N], yh[NV][N], b[NV][N];  // b = dx' + r dn w_next
    float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < NV; v++) {
      const int h = (v * W * 64 + tid) * N;
#pragma unroll
      for (int i = 0; i < N; i++) xh[v][i] = 0.0f, yh[v][i] = 0.0f, b[v][i] = 0.0f;
      if (h < H) {
        const int at = HOLD ? v : 0;
        if constexpr (!HOLD) weights(v, h);
        if (a.dx_out) rds[v].get(b[v]);
        if (a.dn) {
          float dn[N];
          rx[v].get(xh[v]);
          rdn[v].get(dn);
#pragma unroll
          for (int i = 0; i < N; i++) {
            xh[v][i] *= rnt;
            dwn[v][i] = fmaf(dn[i], xh[v][i], dwn[v][i]);
            dn[i] *= wn[at][i];
            s[0] = fmaf(dn[i], xh[v][i], s[0]);
            b[v][i] = fmaf(rnt, dn[i], b[v][i]);
          }
        }
        if (a.y) {
          ry[v].get(yh[v]);
#pragma unroll
          for (int i = 0; i < N; i++) {
            yh[v][i] *= rpt;
            const float q = gc[at][i] * wp[at][i] * yh[v][i];
            s[1] = fmaf(q, b[v][i], s[1]);
            s[2] = fmaf(q, xh[v][i], s[2]);
          }
        }
      }
    }
    if (HOLD && t + (int)gridDim.x < a.T) fetch(t + gridDim.x);  // this workgroup's own row: nothing that it writes here is read there
    block_sum<3, W>(s, buf, half);
    const float c = rnt * s[0] / (float)H;           // D = b - xh c
    const float dot = s[1] - c * s[2], q = gtt * dot / (float)H;  // sum of D u; mean of dv yh
    if (a.d_gate && !channel && tid == 0) a.d_gate[t] = dot;
#pragma unroll
    for (int v = 0; v < NV; v++) {
      const int h = (v * W * 64 + tid) * N;
      if (h < H) {
        const int at = HOLD ? v : 0;
        if constexpr (!HOLD) weights(v, h);
        float D[N], o[N];
#pragma unroll
        for (int i = 0; i < N; i++) {
          D[i] = fmaf(-xh[v][i], c, b[v][i]);
          o[i] = a.scale * D[i];
        }
        if (a.dx) store_n<N>((TX *)a.dx + row + h, o);
        if (a.y) {
#pragma unroll
          for (int i = 0; i < N; i++) {
            const float du = gtt * gc[at][i] * D[i], u = yh[v][i] * wp[at][i];
            if (channel) dgc[v][i] = fmaf(D[i], u, dgc[v][i]);
            dwp[v][i] = fmaf(du, yh[v][i], dwp[v][i]);
            o[i] = a.w_post ? rpt * (du * wp[at][i] - yh[v][i] * q) : du;
          }
          if (a.dy) store_n<N>((TD *)a.dy + row + h, o);
        }
      }
    }
  }
  float *const ws = (float *)a.ws + (size_t)blockIdx.x * 3 * H;
  const bool alone = gridDim.x == 1;  // the sums are the results
#pragma unroll
  for (int v = 0; v < NV; v++) {
    const int h = (v * W * 64 + tid) * N;
    if (h < H) {
      if (a.dw_next) store_n<N>((alone ? a.dw_next : ws) + h, dwn[v]);
      if (a.dw_post) store_n<N>((alone ? a.dw_post : ws + H) + h, dwp[v]);
      if (a.d_gate && channel) store_n<N>((alone ? a.d_gate : ws + 2 * (size_t)H) + h, dgc[v]);
    }
  }
}

// The column sums of G workgroups, 64 columns a workgroup: sixteen waves take every sixteenth partial sum each.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(kSumWaves * 64) void column_sum_kernel(const float *ws, int G, int H, float *o0, float *o1,
                                                                    float *o2) {
  __shared__ float buf[kSumWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = blockIdx.x * 64 + lane;
  float *o = blockIdx.y == 0 ? o0 : (blockIdx.y == 1 ? o1 : o2);
  if (!o) return;
  float s = 0.0f;
  if (h < H) {
    const float *p = ws + (size_t)blockIdx.y * H + h;
#pragma unroll 8
    for (int g = wave; g < G; g += kSumWaves) s += p[(size_t)g * 3 * H];
  }
  buf[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && h < H) {
#pragma unroll
    for (int w = 1; w < kSumWaves; w++) s += buf[w][lane];
    o[h] = s;
  }
}

// Workgroups of a backward pass: one to a compute unit (6000 x 4096: 80 us, 85 with two, 90 with three), two of short rows.  Up to
// four rows one workgroup takes them all: a row takes about 1.5 us, a second launch 4.5.
int blocks(int T, int H) {
  const int most = H > 512 ? 256 : 512;
  return T <= 4 ? (T > 0 ? 1 : 0) : (T < most ? T : most);
}

// TD: type of dy, void for the forward pass.
template <typename TX, typename TY, typename TD, int W, int NV, int N>
hipError_t launch(const NormArgs &a, hipStream_t s) {
  if constexpr (std::is_void_v<TD>) {  // T >= 1
    hipLaunchKernelGGL((block_norm_kernel<TX, TY, W, NV, N>), train::grid_of(a.T, W * 64), dim3(W * 64), 0, s, a);
    return hipGetLastError();
  } else {
    const int G = blocks(a.T, a.H);
    if (G > 0) hipLaunchKernelGGL((block_norm_backward_kernel<TX, TY, TD, W, NV, N>), dim3(G), dim3(W * 64), 0, s, a);
    hipError_t err = hipGetLastError();
    float *gate = a.gate_kind == train::kGateChannel ? a.d_gate : nullptr;
    if (err != hipSuccess || G == 1 || (!a.dw_next && !a.dw_post && !gate)) return err;
    hipLaunchKernelGGL(column_sum_kernel, dim3(ceil_div_i(a.H, 64), 3), dim3(kSumWaves * 64), 0, s, (const float *)a.ws, G, a.H,
                       a.dw_next, a.dw_post, gate);
    return hipGetLastError();
  }
}

template <typename TX, typename TY, typename TD>
hipError_t pick(const NormArgs &a, hipStream_t s) {
  const int H = a.H;
  if (H % 8 == 0) {
    if (H <= 512) return launch<TX, TY, TD, 1, 1, 8>(a, s);
    if (H <= 2048) return launch<TX, TY, TD, 4, 1, 8>(a, s);
    if (H <= 4096) return launch<TX, TY, TD, 8, 1, 8>(a, s);
    if (H <= 8192) return launch<TX, TY, TD, 16, 1, 8>(a, s);
    return launch<TX, TY, TD, 16, 2, 8>(a, s);
  }
  if (H <= 256) return launch<TX, TY, TD, 1, 4, 1>(a, s);
  if (H <= 2048) return launch<TX, TY, TD, 4, 8, 1>(a, s);
  if (H <= 4096) return launch<TX, TY, TD, 16, 4, 1>(a, s);
  if (H <= 8192) return launch<TX, TY, TD, 16, 8, 1>(a, s);
  return launch<TX, TY, TD, 16, 16, 1>(a, s);
}

template <typename TX>
hipError_t forward(const NormArgs &a, hipStream_t s) {
  return a.y_bf16 ? pick<TX, uint16_t, void>(a, s) : pick<TX, float, void>(a, s);
}
template <typename TX, typename TY>
hipError_t backward(const NormArgs &a, hipStream_t s) {
  return a.dy_bf16 ? pick<TX, TY, uint16_t>(a, s) : pick<TX, TY, float>(a, s);
}

}  // namespace

size_t train::norm_grad_ws_bytes(int T, int H) {
  const int G = blocks(T, H);
  return G <= 1 ? 0 : align_up((size_t)G * 3 * H * sizeof(float), 256);
}
hipError_t train::launch_block_norm(const NormArgs &a, hipStream_t s) {
  return a.x_bf16 ? forward<uint16_t>(a, s) : forward<float>(a, s);
}
hipError_t train::launch_block_norm_backward(const NormArgs &a, hipStream_t s) {
  if (a.x_bf16) return a.y_bf16 ? backward<uint16_t, uint16_t>(a, s) : backward<uint16_t, float>(a, s);
  return a.y_bf16 ? backward<float, uint16_t>(a, s) : backward<float, float>(a, s);
}
