// moe_quantize_mx4, moe_dequantize_mx and moe_pack_mx4 for gfx950.
//
// Quantisation and its inverse move each element once and compute next to nothing: both are bound by
// HBM.  A lane takes 8 neighbouring values (16 bytes of bf16, 32 of fp32), four neighbouring lanes one
// block of 32, so the block maximum needs two steps inside a quad (DPP) and every lane stores its 8
// codes at once.  Grid-stride loops; all offsets are 64-bit.
#include "mx4_common.h"

namespace {

// Largest value over the quad of lanes 4i .. 4i+3, in all four.  Every lane of the quad takes part.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true));  // quad_perm [1, 0, 3, 2]
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true));  // quad_perm [2, 3, 0, 1]
}

template <bool BF16>
__global__ __launch_bounds__(256) void quantize_mx4_kernel(const void *__restrict__ x, long long nvec,
                                                           uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
  // nvec = elements / 8 and the stride are multiples of 4: the four lanes of a block loop together
  const long long stride = (long long)gridDim.x * blockDim.x;
  for (long long v = (long long)blockIdx.x * blockDim.x + threadIdx.x; v < nvec; v += stride) {
    float f[8];
    if constexpr (BF16) {
      const u32x4_t p = *((const u32x4_t *)x + v);
      f[0] = bf16_lo(p.x); f[1] = bf16_hi(p.x); f[2] = bf16_lo(p.y); f[3] = bf16_hi(p.y);
      f[4] = bf16_lo(p.z); f[5] = bf16_hi(p.z); f[6] = bf16_lo(p.w); f[7] = bf16_hi(p.w);
    } else {
      const f32x4_t a = *((const f32x4_t *)x + 2 * v), b = *((const f32x4_t *)x + 2 * v + 1);
#pragma unroll
      for (int j = 0; j < 4; j++) { f[j] = a[j]; f[4 + j] = b[j]; }
    }
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) m = max(m, mx4::abs_bits(f[j]));
    const uint32_t s = mx4::scale_of_bits<2>(quad_max(m));
    const int ex = 127 - (int)s;
#pragma unroll
    for (int j = 0; j < 8; j++) f[j] = ldexpf(f[j], ex);
    const uint32_t w = mx4::e2m1_quad(f[0], f[1], f[2], f[3]) | (mx4::e2m1_quad(f[4], f[5], f[6], f[7]) << 16);
    *((uint32_t *)codes + v) = s == 255 ? 0u : w;
    if ((v & 3) == 0) scales[v >> 2] = (uint8_t)s;
  }
}

template <bool FP4, bool BF16>
__global__ __launch_bounds__(256) void dequantize_mx_kernel(const uint8_t *__restrict__ codes,
                                                            const uint8_t *__restrict__ scales, long long nvec,
                                                            void *__restrict__ out) {
  const long long stride = (long long)gridDim.x * blockDim.x;
  for (long long v = (long long)blockIdx.x * blockDim.x + threadIdx.x; v < nvec; v += stride) {
    const uint32_t s = scales[v >> 2];
    float f[8];
    auto put = [&](int j, auto p) { f[j] = p[0]; f[j + 1] = p[1]; };
    if constexpr (FP4) {
      const uint32_t w = *((const uint32_t *)codes + v);
      put(0, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0));
      put(2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1));
      put(4, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2));
      put(6, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3));
    } else {
      const uint2 w = *((const uint2 *)codes + v);
      put(0, __builtin_amdgcn_cvt_pk_f32_fp8((int)w.x, false));
      put(2, __builtin_amdgcn_cvt_pk_f32_fp8((int)w.x, true));
      put(4, __builtin_amdgcn_cvt_pk_f32_fp8((int)w.y, false));
      put(6, __builtin_amdgcn_cvt_pk_f32_fp8((int)w.y, true));
    }
    // exact in fp32; exact in bf16 too, but for results below its least subnormal 2^-133 (E4M3 only), which round
#pragma unroll
    for (int j = 0; j < 8; j++) f[j] = s == 255 ? __uint_as_float(0x7fc00000u) : ldexpf(f[j], (int)s - 127);
    if constexpr (BF16) {
      *((u32x4_t *)out + v) = u32x4_t{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                      pack_bf16x2(f[6], f[7])};
    } else {
      *((f32x4_t *)out + 2 * v) = f32x4_t{f[0], f[1], f[2], f[3]};
      *((f32x4_t *)out + 2 * v + 1) = f32x4_t{f[4], f[5], f[6], f[7]};
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

unsigned grid_for(long long n) {
  const long long blocks = (n + 255) / 256;
  return (unsigned)(blocks < 8192 ? blocks : 8192);
}

}  // namespace

hipError_t launch_quantize_mx4(const void *x, int x_bf16, long long rows, int K, uint8_t *codes, uint8_t *scales,
                               hipStream_t s) {
  const long long n = rows * K / 8;
  if (n == 0) return hipSuccess;
  if (x_bf16) hipLaunchKernelGGL(quantize_mx4_kernel<true>, dim3(grid_for(n)), dim3(256), 0, s, x, n, codes, scales);
  else hipLaunchKernelGGL(quantize_mx4_kernel<false>, dim3(grid_for(n)), dim3(256), 0, s, x, n, codes, scales);
  return hipGetLastError();
}

hipError_t launch_dequantize_mx(const uint8_t *codes, const uint8_t *scales, int fp4, long long rows, int K, void *out,
                                int out_bf16, hipStream_t s) {
  const long long n = rows * K / 8;
  if (n == 0) return hipSuccess;
  const dim3 g(grid_for(n)), b(256);
  if (fp4 && out_bf16) hipLaunchKernelGGL((dequantize_mx_kernel<true, true>), g, b, 0, s, codes, scales, n, out);
  else if (fp4) hipLaunchKernelGGL((dequantize_mx_kernel<true, false>), g, b, 0, s, codes, scales, n, out);
  else if (out_bf16) hipLaunchKernelGGL((dequantize_mx_kernel<false, true>), g, b, 0, s, codes, scales, n, out);
  else hipLaunchKernelGGL((dequantize_mx_kernel<false, false>), g, b, 0, s, codes, scales, n, out);
  return hipGetLastError();
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
