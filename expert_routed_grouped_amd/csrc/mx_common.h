// MXFP8 helpers shared by the quantisation kernel and the W8A8 grouped FFN.
//
// MXFP8 (OCP microscaling, the format of the "Quantization" section of "Hosting
// Qwen on Blackwell"): 32 consecutive values along the contraction axis share
// one E8M0 scale byte s (value 2^(s-127)); each value is an OCP E4M3 code.
// Block rule used here: s = clamp(floor(log2 amax) - 8 + 127, 0, 254) (s = 0 for
// an all-zero block), code = E4M3 nearest to v / 2^(s-127), ties to even,
// magnitudes >= 448 saturate to 448, sign bit kept; a block that holds a NaN or an infinity gets
// s = 255, so that all of it reads as NaN.
#pragma once
#include "common.h"

#include <type_traits>

// E8M0 scale byte of a block from the bit pattern of its largest magnitude (the maximum over bit patterns
// orders NaN above infinity above every finite value; the floating-point maximum would drop NaN).  EMAX:
// exponent of the format's largest power of two (2 for E2M1, 8 for E4M3).  The exponent field ef gives
// floor(log2 amax) = ef - 127 for normal amax, and ef - EMAX <= 0 covers zero, subnormal and tiny blocks.
template <int EMAX>
__device__ __forceinline__ uint32_t mx_scale_of_bits(uint32_t amax_bits) {
  const int ef = (int)(amax_bits >> 23);
  return ef == 255 ? 255u : (uint32_t)max(ef - EMAX, 0);
}
__device__ __forceinline__ uint32_t mx_abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// E4M3 code of a finite fp32 value: round to nearest, ties to the even code,
// saturating at 448, sign bit kept.  The gfx950 packed conversion to OCP E4M3
// rounds to nearest even; clamping to +-448 first gives the saturation (checked
// on the GPU against a bit-by-bit encoder of the same rule over every E4M3 value,
// every midpoint between neighbours and one fp32 ulp either side of it, the
// saturation range and 4 M log-uniform random values: no difference).
__device__ __forceinline__ uint32_t e4m3_encode(float v) {
  const float c = fminf(fmaxf(v, -448.0f), 448.0f);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, 0.0f, 0, false) & 0xFFu;
}

// Bit pattern of the largest magnitude over the 32 lanes of this half-wave (lanes 0-31 or 32-63), in
// every lane of it: DPP butterflies inside each row of 16 lanes (quad swaps, then the mirrored half
// row, then the mirrored row), then one exchange between the two rows.  Every lane must take part.
__device__ __forceinline__ uint32_t halfwave_amax(float v) {
  auto dpp = [](uint32_t x, auto CTRL) __attribute__((always_inline)) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(CTRL)::value, 0xf, 0xf, true);
  };
  uint32_t a = mx_abs_bits(v);
  a = max(a, dpp(a, std::integral_constant<int, 0xB1>{}));   // quad_perm [1, 0, 3, 2]
  a = max(a, dpp(a, std::integral_constant<int, 0x4E>{}));   // quad_perm [2, 3, 0, 1]
  a = max(a, dpp(a, std::integral_constant<int, 0x141>{}));  // row_half_mirror
  a = max(a, dpp(a, std::integral_constant<int, 0x140>{}));  // row_mirror
  return max(a, (uint32_t)__shfl_xor((int)a, 16, 64));
}
