// Launchers of the operators that train a MoE block (grouped products, SwiGLU, router gradient, block norms).
// Arguments are validated by the ABI layer (abi_train.hip).
#pragma once
#include "common.h"

namespace train {

// A launch has fewer than 2^32 threads along an axis: more workgroups than that go into rows of 2^21, the last of which may
// have workgroups too many.  block_of is a workgroup's number, and the same XCD takes it as in one row.
constexpr int kGridRow = 1 << 21;
inline dim3 grid_of(long long blocks, int threads) {
  if (blocks * threads < (1LL << 32)) return dim3((unsigned)blocks);
  return dim3(kGridRow, (unsigned)((blocks + kGridRow - 1) / kGridRow));
}
__device__ __forceinline__ int block_of() { return (int)(blockIdx.y * kGridRow + blockIdx.x); }

// The rows [r0, r0 + rows) between an expert's offsets that lie in the buffers.  Both ends are clipped before they are
// subtracted: whatever the offsets say, the difference fits.
__device__ __forceinline__ void clip_rows(int begin, int end, int R_cap, int &r0, int &rows) {
  r0 = min(max(begin, 0), R_cap);
  rows = max(min(end, R_cap), r0) - r0;
}

// One product grouped by expert.  Rows r of expert e are offsets[e] .. offsets[e+1] - 1, never past R_cap.
struct MmArgs {
  const void *a;              // [a_rows, K]; row r of the product reads a[a_index ? a_index[r] : r]
  const int32_t *a_index;
  int a_rows;
  const void *w;              // [El, N, K], or [El, K, N] with kn
  const int32_t *offsets;     // [El + 1]
  int El, R_cap, N, K;
  void *out;                  // [R_cap, N]
  int bf16, out_bf16, kn;
};
hipError_t launch_grouped_mm(const MmArgs &a, hipStream_t s);
bool mm_dma_fits(const MmArgs &a);  // grouped_mm_dma.hip
hipError_t launch_mm_dma(const MmArgs &a, bool few, hipStream_t s);  // fp32: few only

// dw[e] = sum over e's rows of a_r b_r^T (+ dw[e] with add).
struct WgradArgs {
  const void *a, *b;          // [a_rows, M], [b_rows, N]
  const int32_t *a_index, *b_index;
  int a_rows, b_rows;
  const int32_t *offsets;
  int El, R_cap, M, N;
  void *dw;                   // [El, M, N]
  int bf16, out_bf16, add;
  void *ws;                   // wgrad_ws_bytes
  int splits;                 // set by the launchers: an expert's rows in so many parts, part s's sums at dw + s El M N
};
// Rows of part s of an expert's rows [r0, r0 + rows), whole 64s but for the last.
__device__ __forceinline__ void part_of(int s, int splits, int &r0, int &rows) {
  const int per = ((rows + splits - 1) / splits + 63) & ~63, at = min(s * per, rows);
  r0 += at;
  rows = min(per, rows - at);
}
size_t wgrad_ws_bytes(int El, int R_cap, int M, int N, int bf16);
hipError_t launch_grouped_wgrad(const WgradArgs &a, hipStream_t s);
bool wgrad_dma_fits(const WgradArgs &a);  // grouped_mm_dma.hip
hipError_t launch_wgrad_dma(const WgradArgs &a, hipStream_t s);

// h = row_w silu(gate) up; offsets NULL: every one of the R_cap rows.
struct SwigluArgs {
  const void *gu, *dh;        // [R_cap, 2I], [R_cap, I]
  const int32_t *offsets;
  const float *row_w;
  int El, R_cap, I, bf16;
  void *h, *dgu;
  float *d_row_w;
};
hipError_t launch_swiglu(const SwigluArgs &a, hipStream_t s);
hipError_t launch_swiglu_backward(const SwigluArgs &a, hipStream_t s);

struct RouteGradArgs {
  const int32_t *ids;         // [T, k]
  const float *gates, *d_gates;
  int T, k, E, H;
  const void *x, *wr;         // [T, H], [E, H]
  int bf16;
  const int32_t *offsets, *row_token;  // grouping over all E experts: [E + 1], [T * k]
  const void *rows;           // [R_cap, H] or NULL
  int rows_bf16;
  const int32_t *rows_at;     // [T, k]: row of an assignment in ``rows``, -1 none
  int R_cap;
  void *dx;
  int dx_bf16;
  float *dwr, *dbias;
};
hipError_t launch_route_grad(const RouteGradArgs &a, hipStream_t s);

enum { kGateNone = 0, kGateChannel = 1, kGateToken = 2 };
struct NormArgs {
  const void *x, *y;          // x: the residual (forward) or the sum that it gave (backward)
  int x_bf16, y_bf16, dy_bf16;
  const void *w_next, *w_post, *gate;
  int w_bf16, gate_kind;
  float scale, eps;
  int T, H;
  void *x_out, *n;
  float *rstd_next, *rstd_post;
  const float *rn, *rp;       // backward: the reciprocal roots of the forward call
  const void *dx_out, *dn;
  void *dx, *dy;
  float *dw_next, *dw_post, *d_gate;
  void *ws;                   // norm_grad_ws_bytes
};
constexpr int kNormMaxH = 16384;
size_t norm_grad_ws_bytes(int T, int H);
hipError_t launch_block_norm(const NormArgs &a, hipStream_t s);
hipError_t launch_block_norm_backward(const NormArgs &a, hipStream_t s);

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t *p, float v) { *p = f32_to_bf16(v); }

// N consecutive values, N a multiple of 4 or 1; 8-byte loads of four bf16.
template <int N>
__device__ __forceinline__ void load_n(const float *p, float (&v)[N]) {
  if constexpr (N == 1) v[0] = *p;
  else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 t = *(const float4 *)(p + i);
      v[i] = t.x, v[i + 1] = t.y, v[i + 2] = t.z, v[i + 3] = t.w;
    }
  }
}
template <int N>
__device__ __forceinline__ void load_n(const uint16_t *p, float (&v)[N]) {
  if constexpr (N == 1) v[0] = bf16_to_f32(*p);
  else if constexpr (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 8) {
      const u32x4_t t = *(const u32x4_t *)(p + i);
#pragma unroll
      for (int j = 0; j < 4; j++) v[i + 2 * j] = bf16_lo(t[j]), v[i + 2 * j + 1] = bf16_hi(t[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint2 t = *(const uint2 *)(p + i);
      v[i] = bf16_lo(t.x), v[i + 1] = bf16_hi(t.x), v[i + 2] = bf16_lo(t.y), v[i + 3] = bf16_hi(t.y);
    }
  }
}
template <int N>
__device__ __forceinline__ void store_n(float *p, const float (&v)[N]) {
  if constexpr (N == 1) *p = v[0];
  else {
#pragma unroll
    for (int i = 0; i < N; i += 4) *(float4 *)(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  }
}
template <int N>
__device__ __forceinline__ void store_n(uint16_t *p, const float (&v)[N]) {
  if constexpr (N == 1) *p = f32_to_bf16(v[0]);
  else if constexpr (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 8)
      *(u32x4_t *)(p + i) = u32x4_t{pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]),
                                    pack_bf16x2(v[i + 4], v[i + 5]), pack_bf16x2(v[i + 6], v[i + 7])};
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *(uint2 *)(p + i) = make_uint2(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]));
  }
}

// Sum over a wave, the same in every lane.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

}  // namespace train
