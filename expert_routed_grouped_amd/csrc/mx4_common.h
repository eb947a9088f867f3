// MXFP4 helpers shared by the quantisation kernels, the grouped FFN and the few-token layer.
//
// MXFP4 (OCP microscaling): 32 consecutive values along the contraction axis share one E8M0 scale
// byte s (value 2^(s-127), 255 = NaN); each value is an E2M1 code (sign, magnitudes 0, 0.5, 1, 1.5,
// 2, 3, 4, 6), two codes per byte, the even index in the low half.  Block rule:
// s = max(floor(log2 amax) - 2 + 127, 0), code = E2M1 nearest to v / 2^(s-127), ties to the even
// code, magnitudes above 6 saturate, sign kept; a block that holds a NaN or an infinity gets s = 255,
// so that all of it reads as NaN.
//
// The products run on v_mfma_scale_f32_16x16x128_f8f6f4: 128 k per instruction, the block scales
// applied inside the matrix core.  Operand layout, measured on MI355X, for lane l = 16 q + n: row (or
// column) n; an E2M1 operand is one 16-byte piece, k = 32q .. 32q+31; an E4M3 operand is two, k = 16q
// .. 16q+15 and k = 64+16q .. 64+16q+15; either way lane (n, q) supplies the scale of the 32-wide block
// q.  The weights are the first operand, so D holds weight rows 4q .. 4q+3 of token n in lane (n, q):
// four neighbouring output columns of one token, and a 32-column block of the intermediate in the four
// lanes of one token, which is what the quantising epilogue and the stores want.
#pragma once
#include "ffn_common.h"
#include "mx_common.h"

namespace mx4 {

typedef int v8i_t __attribute__((ext_vector_type(8)));

// element formats of an operand, as the matrix instruction numbers them
constexpr int FP8 = 0, FP4 = 4;

// Bytes of K values of format F.
template <int F>
__host__ __device__ constexpr size_t code_bytes(size_t K) { return F == FP8 ? K : K / 2; }

// Packed weights (moe_pack_mx4): rows in groups of 16 over all experts.  Codes: per group K/128 blocks
// of 1 KB, piece (q, n) of a block at (16 q + n) * 16: lane (n, q) reads its piece of every block, a wave
// 1 KB contiguously.  Scales: per group ceil(K/512) blocks of 256 bytes, the dword of lane (n, q) at
// (16 q + n) * 4, its byte j the scale of k = 128 j + 32 q .. of the block's 512 values.
constexpr int kBlk = 1024, kSblk = 256;
__host__ __device__ __forceinline__ size_t group_codes(int K) { return (size_t)(K / 128) * kBlk; }
__host__ __device__ __forceinline__ size_t group_scales(int K) { return (size_t)((K + 511) / 512) * kSblk; }

// By value: a component read through a reference would become a load without type information, and the compiler
// then waits for every load into LDS in flight before it.
__device__ __forceinline__ v8i_t piece4(const u32x4_t p) {
  return v8i_t{(int)p.x, (int)p.y, (int)p.z, (int)p.w, 0, 0, 0, 0};
}
__device__ __forceinline__ v8i_t piece8(const u32x4_t lo, const u32x4_t hi) {
  return v8i_t{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// acc += weights (16 rows) x activations (16 tokens) over 128 k; byte J of sw and byte JA of sa scale.
template <int FA, int J, int JA = 0>
__device__ __forceinline__ f32x4_t mfma(const v8i_t &w, const v8i_t &a, const f32x4_t &acc, uint32_t sw, uint32_t sa) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, acc, FP4, FA, J, (int)sw, JA, (int)sa);
}

// One 128-k step of an activation row-major operand: row points at this lane's row.
template <int FA>
__device__ __forceinline__ v8i_t act_frag(const uint8_t *row, int step, int q) {
  if constexpr (FA == FP8) {
    const uint8_t *p = row + (size_t)step * 128 + 16 * q;
    return piece8(*(const u32x4_t *)p, *(const u32x4_t *)(p + 64));
  } else {
    return piece4(*(const u32x4_t *)(row + (size_t)step * 64 + 16 * q));
  }
}
// Its scale (in the low byte): srow points at this lane's row of scales.
__device__ __forceinline__ uint32_t act_scale(const uint8_t *srow, int step, int q) {
  return *(const uint32_t *)(srow + 4 * (size_t)step) >> (8 * q);
}

// Scales of the intermediate h (workspace): per row ceil(I/512) pieces of 16 bytes; lane quarter q takes the dword
// at 4 q of a piece, whose byte j is the scale of step j, as for the packed weights.
__host__ __device__ __forceinline__ size_t h_scale_stride(int I) { return (size_t)((I + 511) / 512) * 16; }
// Place of block b (columns 32b ..) in its row.
__device__ __forceinline__ int h_scale_pos(int b) { return (b & ~15) + (b & 3) * 4 + ((b >> 2) & 3); }

// E2M1 codes of a and b (already divided by the scale), a in the low half.  The packed conversion of
// gfx950 rounds to nearest, ties to even, and saturates at 6 (checked over -8 .. 8 in steps of 1/512
// and at every midpoint).
__device__ __forceinline__ uint32_t e2m1_pair(float a, float b) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, a, b, 1.0f, 0) & 0xffu;
}
__device__ __forceinline__ uint32_t e2m1_quad(float a, float b, float c, float d) {
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, a, b, 1.0f, 0);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, c, d, 1.0f, 1) & 0xffffu;
}
__device__ __forceinline__ uint32_t e4m3_quad(float a, float b, float c, float d) {
  auto clip = [](float v) { return fminf(fmaxf(v, -448.0f), 448.0f); };
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(clip(a), clip(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clip(c), clip(d), lo, true);
}

// Quantise and store this lane's part of one 32-column block of the intermediate of one token:
// v[g][r] is column 16 g + 4 q + r.  The four lanes (n, 0..3) of a token hold the block.  Every lane of the
// wave takes part; ``on`` says whether the token exists.  hrow / srow: the token's code row and its scales.
template <int FA>
__device__ __forceinline__ void store_h_block(const float (&v)[2][4], bool on, uint8_t *hrow, uint8_t *srow, int col0,
                                              int q) {
  uint32_t m = 0;
#pragma unroll
  for (int g = 0; g < 2; g++)
#pragma unroll
    for (int r = 0; r < 4; r++) m = max(m, mx_abs_bits(v[g][r]));
  m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
  const uint32_t s = mx_scale_of_bits<FA == FP8 ? 8 : 2>(m);
  const int ex = 127 - (int)s;
  if (!on) return;
#pragma unroll
  for (int g = 0; g < 2; g++) {
    float u[4];
#pragma unroll
    for (int r = 0; r < 4; r++) u[r] = ldexpf(v[g][r], ex);
    const int col = col0 + 16 * g + 4 * q;
    if constexpr (FA == FP8) *(uint32_t *)(hrow + col) = s == 255 ? 0u : e4m3_quad(u[0], u[1], u[2], u[3]);
    else *(uint16_t *)(hrow + col / 2) = s == 255 ? (uint16_t)0 : (uint16_t)e2m1_quad(u[0], u[1], u[2], u[3]);
  }
  if (q == 0) srow[h_scale_pos(col0 / 32)] = (uint8_t)s;
}

// Four neighbouring output values of one row, fp32 or rounded to bf16 (nearest even).
template <bool BF16>
__device__ __forceinline__ void store4(void *base, size_t index, const f32x4_t &v) {
  if constexpr (BF16) *(uint2 *)((uint16_t *)base + index) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  else *(f32x4_t *)((float *)base + index) = v;
}

// Two neighbouring 16-column groups of one row, a and b (this lane: columns 4q .. 4q+3 of each): bf16 values are
// exchanged between lane quarters first (row-pair swap), so that a lane stores 16 contiguous bytes and the four
// lanes of a row 64, twice what they would without (32-byte pieces took 130 us for 6000 tokens' rows).
// ``base``: the row at the first column of a.  The whole wave takes part; ``on``: this lane's row exists.
template <bool BF16>
__device__ __forceinline__ void store_pair(void *base, size_t index, int q, const f32x4_t &a, const f32x4_t &b, bool on) {
  if constexpr (BF16) {
    u32x4_t v;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const auto s = __builtin_amdgcn_permlane16_swap(pack_bf16x2(a[2 * i], a[2 * i + 1]),
                                                      pack_bf16x2(b[2 * i], b[2 * i + 1]), false, false);
      v[i] = s[0];
      v[2 + i] = s[1];
    }
    // quarter 0: a 0-7, 1: b 0-7, 2: a 8-15, 3: b 8-15
    if (on) *(u32x4_t *)((uint16_t *)base + index + (q & 1) * 16 + (q >> 1) * 8) = v;
  } else if (on) {
    *(f32x4_t *)((float *)base + index + 4 * q) = a;
    *(f32x4_t *)((float *)base + index + 16 + 4 * q) = b;
  }
}

}  // namespace mx4

// ---------------------------------------------------------------------------
// Internal launchers (host side).  Arguments are validated by the ABI layer.
// ---------------------------------------------------------------------------
hipError_t launch_quantize_mx4(const void *x, int x_bf16, long long rows, int K, uint8_t *codes, uint8_t *scales,
                               hipStream_t s);
hipError_t launch_dequantize_mx(const uint8_t *codes, const uint8_t *scales, int fp4, long long rows, int K, void *out,
                                int out_bf16, hipStream_t s);
hipError_t launch_pack_mx4(const uint8_t *codes, const uint8_t *scales, long long rows, int K, uint8_t *pcodes,
                           uint8_t *pscales, hipStream_t s);

struct FfnMx4Args {
  const uint8_t *a, *a_s;      // activations [T, H] (E4M3 or E2M1 codes) and scales [T, H/32]
  int a_fp4;                   // 1: E2M1 activations and intermediate, 0: E4M3
  const int32_t *offsets;      // [El+1]
  const int32_t *row_token;    // [R_cap]
  const float *row_w;          // [R_cap]
  const int32_t *token_row;    // [T, k]
  int El, T, k, R_cap, H, I;
  const uint8_t *wgu, *wgu_s;  // packed codes and scales of [El, 2I, H]
  const uint8_t *wd, *wd_s;    // packed codes and scales of [El, H, I]
  void *y;                     // [T, H], overwritten
  int y_bf16;
  void *ws;
  // launch_down_sum_mx4 only
  const int2 *tiles;           // its tiles {first row, expert | rows << 16}, or NULL: found from the offsets
  const int *ntiles;
  uint32_t *zero;              // n_zero words that it zeroes, or NULL
  int n_zero;
};
size_t ffn_mx4_ws_bytes(int T, int R_cap, int El, int H, int I, int y_bf16);
hipError_t launch_ffn_mx4(const FfnMx4Args &a, hipStream_t s);
// Weight-streaming path for few rows per expert (ffn_mx4_stream.hip), T <= kMx4StreamMaxT: h and its scales into
// ``h`` / ``hs``, then the down half, which also sums to token order; launch_down_sum_mx4 is that half alone.
// (Beyond, a tile kernel: 128 experts of 4096 x 1536, top 8, 64 tokens 201 us this way, 65 by tiles 206.)
constexpr int kMx4StreamMaxT = 64;
hipError_t launch_ffn_mx4_stream(const FfnMx4Args &a, uint8_t *h, uint8_t *hs, hipStream_t s);
hipError_t launch_down_sum_mx4(const FfnMx4Args &a, const uint8_t *h, const uint8_t *hs, hipStream_t s);

// The whole layer of a few tokens (decode_mx4.hip): T <= kMx4StreamMaxT.  Its workspace starts with control words that
// are zero before the call and after it (the error word, uint32 number 4, excepted).
constexpr int kDecodeMx4MaxH = 8192, kDecodeMx4MaxE = 256;
struct DecodeMx4Args {
  const void *x;               // [T, H] bf16
  const float *wr;             // router weight, fp32 packed [H/4, E, 4]
  const float *bias;           // [E] or NULL
  int T, H, E, k, lo, El, I;
  const uint8_t *wgu, *wgu_s;  // packed codes and scales of [El, 2I, H]
  const uint8_t *wd, *wd_s;    // packed codes and scales of [El, H, I]
  int32_t *ids;                // [T, k]
  float *gates;                // [T, k]
  void *y;                     // [T, H], overwritten
  int y_bf16;
  void *ws;
};
size_t decode_layer_mx4_ws_bytes(int T, int k, int El, int H, int I);
hipError_t launch_decode_layer_mx4(const DecodeMx4Args &a, hipStream_t s);
