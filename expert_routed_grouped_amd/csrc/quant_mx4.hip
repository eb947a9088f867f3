// moe_quantize_mx4, moe_dequantize_mx and moe_pack_mx4 for gfx950.
//
// Quantisation and its inverse move each element once and compute next to nothing: both are bound by
// HBM.  A lane takes 16 bytes of values, 8 of bf16 or 4 of fp32, so that a wave's access is contiguous whatever the
// type; four or eight neighbouring lanes hold a block of 32, whose maximum takes two or three steps inside a row
// of lanes (DPP), and each lane stores its own codes.  Grid-stride loops; all offsets are 64-bit.
//
// Below 256 MiB of values (what the last-level cache holds) a lane has one vector at a time and ordinary accesses:
// what was written is often read soon (6000 x 4096 bf16: 10.9 us there, 11.1 us back; with the other scheme 12.9 and
// 14.6).  Above, four vectors per lane in flight and non-temporal accesses (128 x 4096 x 1536 fp32: 769 us there, 871
// back, against 819 and 1017).
#include "mx4_common.h"

namespace {

// Largest value over the lanes of a block (N = 4: the quad; N = 8: half a row of 16), in all of them.
template <int N>
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true));  // quad_perm [1, 0, 3, 2]
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true));  // quad_perm [2, 3, 0, 1]
  if constexpr (N == 8)
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true));  // row_half_mirror
  return v;
}

template <bool NT, typename T>
__device__ __forceinline__ T get(const T *p) {
  if constexpr (NT) return __builtin_nontemporal_load(p);
  else return *p;
}
template <bool NT, typename T>
__device__ __forceinline__ void put(T v, T *p) {
  if constexpr (NT) __builtin_nontemporal_store(v, p);
  else *p = v;
}

// U vectors per lane and turn, a stride apart, all loaded before any is converted.  nvec (16-byte vectors) and the
// stride are multiples of the lanes of a block, which are therefore always on together.
template <bool BF16, bool NT, int U>
__global__ __launch_bounds__(256) void quantize_mx4_kernel(const u32x4_t *__restrict__ x, long long nvec,
                                                           void *__restrict__ codes, uint8_t *__restrict__ scales) {
  constexpr int V = BF16 ? 8 : 4, N = 32 / V;  // values per lane, lanes per block
  const long long stride = (long long)gridDim.x * blockDim.x;
  for (long long v0 = (long long)blockIdx.x * blockDim.x + threadIdx.x; v0 < nvec; v0 += U * stride) {
    u32x4_t r[U];
#pragma unroll
    for (int u = 0; u < U; u++) r[u] = get<NT>(x + min(v0 + u * stride, nvec - 1));  // past the end: again, not stored
#pragma unroll
    for (int u = 0; u < U; u++) {
      const long long v = v0 + u * stride;
      float f[V];
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < V; j++) {
        if constexpr (BF16) f[j] = (j & 1) ? bf16_hi(r[u][j >> 1]) : bf16_lo(r[u][j >> 1]);
        else f[j] = __uint_as_float(r[u][j]);
        m = max(m, mx_abs_bits(f[j]));
      }
      const uint32_t s = mx_scale_of_bits<2>(block_max<N>(m));
#pragma unroll
      for (int j = 0; j < V; j++) f[j] = ldexpf(f[j], 127 - (int)s);
      if (v >= nvec) continue;
      uint32_t w = mx4::e2m1_quad(f[0], f[1], f[2], f[3]);
      if constexpr (BF16) {
        w |= mx4::e2m1_quad(f[V - 4], f[V - 3], f[V - 2], f[V - 1]) << 16;
        put<NT>(s == 255 ? 0u : w, (uint32_t *)codes + v);
      } else {
        put<NT>((uint16_t)(s == 255 ? 0u : w), (uint16_t *)codes + v);
      }
      if ((v & (N - 1)) == 0) scales[v / N] = (uint8_t)s;
    }
  }
}

template <bool FP4, bool BF16, bool NT, int U>
__global__ __launch_bounds__(256) void dequantize_mx_kernel(const void *__restrict__ codes,
                                                            const uint8_t *__restrict__ scales, long long nvec,
                                                            u32x4_t *__restrict__ out) {
  constexpr int V = BF16 ? 8 : 4, N = 32 / V, CB = FP4 ? V / 2 : V;  // bytes of codes per lane: 2, 4 or 8
  typedef uint16_t u16;
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const long long stride = (long long)gridDim.x * blockDim.x;
  for (long long v0 = (long long)blockIdx.x * blockDim.x + threadIdx.x; v0 < nvec; v0 += U * stride) {
    uint32_t c[U][2], sc[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const long long v = min(v0 + u * stride, nvec - 1);
      sc[u] = scales[v / N];
      c[u][1] = 0;
      if constexpr (CB == 2) {
        c[u][0] = get<NT>((const u16 *)codes + v);
      } else if constexpr (CB == 4) {
        c[u][0] = get<NT>((const uint32_t *)codes + v);
      } else {
        const u32x2 p = get<NT>((const u32x2 *)codes + v);
        c[u][0] = p.x;
        c[u][1] = p.y;
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      const long long v = v0 + u * stride;
      if (v >= nvec) break;
      float f[8];
      auto two = [&](int j, auto p) __attribute__((always_inline)) { f[j] = p[0]; f[j + 1] = p[1]; };
      if constexpr (FP4) {
        two(0, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u][0], 1.0f, 0));
        two(2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u][0], 1.0f, 1));
        two(4, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u][0], 1.0f, 2));
        two(6, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u][0], 1.0f, 3));
      } else {
        two(0, __builtin_amdgcn_cvt_pk_f32_fp8((int)c[u][0], false));
        two(2, __builtin_amdgcn_cvt_pk_f32_fp8((int)c[u][0], true));
        two(4, __builtin_amdgcn_cvt_pk_f32_fp8((int)c[u][1], false));
        two(6, __builtin_amdgcn_cvt_pk_f32_fp8((int)c[u][1], true));
      }
      // exact in fp32; exact in bf16 too, but for results below its least subnormal 2^-133 (E4M3 only), which round
#pragma unroll
      for (int j = 0; j < V; j++) f[j] = sc[u] == 255 ? __uint_as_float(0x7fc00000u) : ldexpf(f[j], (int)sc[u] - 127);
      u32x4_t w;
#pragma unroll
      for (int j = 0; j < 4; j++) w[j] = BF16 ? pack_bf16x2(f[2 * j], f[2 * j + 1]) : __float_as_uint(f[j]);
      put<NT>(w, out + v);
    }
  }
}

// One thread per 16-byte piece of codes: piece (q, n) of block c of group g is bytes 64c + 16q of row 16g + n.
__global__ __launch_bounds__(256) void pack_codes_kernel(const u32x4_t *__restrict__ codes, long long pieces, int K,
                                                         u32x4_t *__restrict__ packed) {
  const long long stride = (long long)gridDim.x * blockDim.x;
  const int kb = K / 128;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < pieces; i += stride) {
    const int l = (int)(i & 63), n = l & 15, q = l >> 4;
    const long long b = i >> 6, g = b / kb;
    const int c = (int)(b - g * kb);
    packed[i] = codes[(g * 16 + n) * (K / 32) + c * 4 + q];
  }
}

// One thread per dword of scales: byte j of lane (n, q) of block c of group g is scale 16c + 4j + q of row
// 16g + n (0 past the end of the row).
__global__ __launch_bounds__(256) void pack_scales_kernel(const uint8_t *__restrict__ scales, long long dwords, int K,
                                                          uint32_t *__restrict__ packed) {
  const long long stride = (long long)gridDim.x * blockDim.x;
  const int sb = (K + 511) / 512, kb = K / 32;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < dwords; i += stride) {
    const int l = (int)(i & 63), n = l & 15, q = l >> 4;
    const long long b = i >> 6, g = b / sb;
    const int c = (int)(b - g * sb);
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int k = 16 * c + 4 * j + q;
      if (k < kb) w |= (uint32_t)scales[(g * 16 + n) * kb + k] << (8 * j);
    }
    packed[i] = w;
  }
}

constexpr long long kCached = 256LL << 20;  // bytes of values (see the top)

unsigned grid_for(long long n) {
  const long long blocks = (n + 255) / 256;
  return (unsigned)(blocks < 8192 ? blocks : 8192);
}

}  // namespace

hipError_t launch_quantize_mx4(const void *x, int x_bf16, long long rows, int K, uint8_t *codes, uint8_t *scales,
                               hipStream_t s) {
  const long long n = rows * K / (x_bf16 ? 8 : 4);
  if (n == 0) return hipSuccess;
  const bool big = n * 16 > kCached;
  const dim3 g(big ? 4096 : grid_for(n)), b(256);
  const u32x4_t *v = (const u32x4_t *)x;
  if (x_bf16 && big) hipLaunchKernelGGL((quantize_mx4_kernel<true, true, 4>), g, b, 0, s, v, n, codes, scales);
  else if (x_bf16) hipLaunchKernelGGL((quantize_mx4_kernel<true, false, 1>), g, b, 0, s, v, n, codes, scales);
  else if (big) hipLaunchKernelGGL((quantize_mx4_kernel<false, true, 4>), g, b, 0, s, v, n, codes, scales);
  else hipLaunchKernelGGL((quantize_mx4_kernel<false, false, 1>), g, b, 0, s, v, n, codes, scales);
  return hipGetLastError();
}

template <bool FP4, bool BF16>
static hipError_t launch_dequantize(const uint8_t *codes, const uint8_t *scales, long long n, void *out, hipStream_t s) {
  const bool big = n * 16 > kCached;
  const dim3 g(big ? 4096 : grid_for(n)), b(256);
  u32x4_t *o = (u32x4_t *)out;
  if (big) hipLaunchKernelGGL((dequantize_mx_kernel<FP4, BF16, true, 4>), g, b, 0, s, codes, scales, n, o);
  else hipLaunchKernelGGL((dequantize_mx_kernel<FP4, BF16, false, 1>), g, b, 0, s, codes, scales, n, o);
  return hipGetLastError();
}

hipError_t launch_dequantize_mx(const uint8_t *codes, const uint8_t *scales, int fp4, long long rows, int K, void *out,
                                int out_bf16, hipStream_t s) {
  const long long n = rows * K / (out_bf16 ? 8 : 4);
  if (n == 0) return hipSuccess;
  if (fp4) return out_bf16 ? launch_dequantize<true, true>(codes, scales, n, out, s) : launch_dequantize<true, false>(codes, scales, n, out, s);
  return out_bf16 ? launch_dequantize<false, true>(codes, scales, n, out, s) : launch_dequantize<false, false>(codes, scales, n, out, s);
}

hipError_t launch_pack_mx4(const uint8_t *codes, const uint8_t *scales, long long rows, int K, uint8_t *pcodes,
                           uint8_t *pscales, hipStream_t s) {
  const long long pieces = rows * (K / 32), dwords = rows / 16 * ((K + 511) / 512) * 64;
  if (rows == 0) return hipSuccess;
  hipLaunchKernelGGL(pack_codes_kernel, dim3(grid_for(pieces)), dim3(256), 0, s, (const u32x4_t *)codes, pieces, K,
                     (u32x4_t *)pcodes);
  hipLaunchKernelGGL(pack_scales_kernel, dim3(grid_for(dwords)), dim3(256), 0, s, scales, dwords, K,
                     (uint32_t *)pscales);
  return hipGetLastError();
}
