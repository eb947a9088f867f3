// C ABI of the MXFP4 operators: argument checks on the host, then launches.  Every check runs before
// anything is enqueued; no call allocates, frees or synchronises.
#include "../../include/moe.h"
#include "mx4_common.h"

namespace {

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }
inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
  return (uintptr_t)a < (uintptr_t)b + nb && (uintptr_t)b < (uintptr_t)a + na;
}

// Sizes the expert FFN takes.  The operand offsets inside a launch are 32-bit: activations, intermediate and
// one expert's weights stay below 2^31 bytes (per-row outputs are addressed with 64 bits).
bool ffn_sizes_ok(int T, int k, int El, int H, int I) {
  if (T < 0 || El < 1 || El > 1024 || k < 1 || k > 32 || H < 128 || I < 128 || H % 128 != 0 || I % 128 != 0) return false;
  const long long R = (long long)T * (k < El ? k : El);
  return (long long)T * H < (1LL << 31) && R * I < (1LL << 31) && (long long)H * I < (1LL << 30) && R < (1LL << 28);
}

}  // namespace

extern "C" {

int moe_quantize_mx4(const void *x, int x_dtype, int64_t rows, int K, uint8_t *codes, uint8_t *scales, void *stream) {
  if (rows < 0 || K < 32 || K % 32 != 0 || rows >= (1LL << 40) / K) return MOE_ERR_SHAPE;
  if (x_dtype != MOE_F32 && x_dtype != MOE_BF16) return MOE_ERR_DTYPE;
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales) return MOE_ERR_NULL;
  if (!aligned(x, 16) || !aligned(codes, 4)) return MOE_ERR_ALIGN;
  const size_t n = (size_t)rows * K, nx = n * (x_dtype == MOE_BF16 ? 2 : 4), nc = n / 2, ns = n / 32;
  if (overlap(x, nx, codes, nc) || overlap(x, nx, scales, ns) || overlap(codes, nc, scales, ns)) return MOE_ERR_SHAPE;
  return hip_status(launch_quantize_mx4(x, x_dtype == MOE_BF16, rows, K, codes, scales, (hipStream_t)stream));
}

int moe_dequantize_mx(const uint8_t *codes, const uint8_t *scales, int mx_dtype, int64_t rows, int K, void *out,
                      int out_dtype, void *stream) {
  if (rows < 0 || K < 32 || K % 32 != 0 || rows >= (1LL << 40) / K) return MOE_ERR_SHAPE;
  if ((mx_dtype != MOE_MXFP4 && mx_dtype != MOE_MXFP8) || (out_dtype != MOE_F32 && out_dtype != MOE_BF16))
    return MOE_ERR_DTYPE;
  if (rows == 0) return MOE_OK;
  if (!codes || !scales || !out) return MOE_ERR_NULL;
  if (!aligned(codes, mx_dtype == MOE_MXFP4 ? 4 : 8) || !aligned(out, 16)) return MOE_ERR_ALIGN;
  const size_t n = (size_t)rows * K, nc = mx_dtype == MOE_MXFP4 ? n / 2 : n, no = n * (out_dtype == MOE_BF16 ? 2 : 4);
  if (overlap(out, no, codes, nc) || overlap(out, no, scales, n / 32)) return MOE_ERR_SHAPE;
  return hip_status(launch_dequantize_mx(codes, scales, mx_dtype == MOE_MXFP4, rows, K, out, out_dtype == MOE_BF16,
                                         (hipStream_t)stream));
}

size_t moe_mx4_packed_scale_bytes(int64_t rows, int K) {
  if (rows < 0 || rows % 16 != 0 || K < 128 || K % 128 != 0 || rows >= (1LL << 40) / K) return 0;
  return (size_t)(rows / 16) * mx4::group_scales(K);
}

int moe_pack_mx4(const uint8_t *codes, const uint8_t *scales, int64_t rows, int K, uint8_t *packed_codes,
                 uint8_t *packed_scales, void *stream) {
  if (rows < 16 || rows % 16 != 0 || K < 128 || K % 128 != 0 || rows >= (1LL << 40) / K) return MOE_ERR_SHAPE;
  if (!codes || !scales || !packed_codes || !packed_scales) return MOE_ERR_NULL;
  if (!aligned(codes, 16) || !aligned(packed_codes, 16) || !aligned(packed_scales, 16)) return MOE_ERR_ALIGN;
  const size_t nc = (size_t)rows * (K / 2), ns = (size_t)rows * (K / 32), ps = moe_mx4_packed_scale_bytes(rows, K);
  if (overlap(codes, nc, packed_codes, nc) || overlap(codes, nc, packed_scales, ps) ||
      overlap(scales, ns, packed_codes, nc) || overlap(scales, ns, packed_scales, ps) ||
      overlap(packed_codes, nc, packed_scales, ps))
    return MOE_ERR_SHAPE;
  return hip_status(launch_pack_mx4(codes, scales, rows, K, packed_codes, packed_scales, (hipStream_t)stream));
}

size_t moe_ffn_mx4_workspace_size(int T, int k, int E_loc, int H, int I, int y_dtype) {
  if (!ffn_sizes_ok(T, k, E_loc, H, I) || (y_dtype != MOE_F32 && y_dtype != MOE_BF16)) return 0;
  return ffn_mx4_ws_bytes(T, T * (k < E_loc ? k : E_loc), E_loc, H, I, y_dtype == MOE_BF16);
}

int moe_grouped_ffn_mx4(const uint8_t *a_codes, const uint8_t *a_scales, int a_dtype, const int32_t *offsets,
                        const int32_t *row_token, const float *row_w, const int32_t *token_row, int E_loc, int T, int k,
                        int H, int I, const uint8_t *wgu_codes, const uint8_t *wgu_scales, const uint8_t *wd_codes,
                        const uint8_t *wd_scales, void *y, int y_dtype, void *workspace, size_t workspace_bytes,
                        void *stream) {
  if (!ffn_sizes_ok(T, k, E_loc, H, I)) return MOE_ERR_SHAPE;
  if ((a_dtype != MOE_MXFP8 && a_dtype != MOE_MXFP4) || (y_dtype != MOE_F32 && y_dtype != MOE_BF16)) return MOE_ERR_DTYPE;
  if (T == 0) return MOE_OK;
  if (!a_codes || !a_scales || !offsets || !row_token || !row_w || !token_row || !wgu_codes || !wgu_scales ||
      !wd_codes || !wd_scales || !y)
    return MOE_ERR_NULL;
  if (!workspace || workspace_bytes < moe_ffn_mx4_workspace_size(T, k, E_loc, H, I, y_dtype)) return MOE_ERR_WORKSPACE;
  if (!aligned(a_codes, 16) || !aligned(a_scales, 4) || !aligned(wgu_codes, 16) || !aligned(wgu_scales, 16) ||
      !aligned(wd_codes, 16) || !aligned(wd_scales, 16) || !aligned(y, 16) || !aligned(workspace, 256))
    return MOE_ERR_ALIGN;
  FfnMx4Args fa{};
  fa.a = a_codes;
  fa.a_s = a_scales;
  fa.a_fp4 = a_dtype == MOE_MXFP4;
  fa.offsets = offsets;
  fa.row_token = row_token;
  fa.row_w = row_w;
  fa.token_row = token_row;
  fa.El = E_loc;
  fa.T = T;
  fa.k = k;
  fa.R_cap = T * (k < E_loc ? k : E_loc);
  fa.H = H;
  fa.I = I;
  fa.wgu = wgu_codes;
  fa.wgu_s = wgu_scales;
  fa.wd = wd_codes;
  fa.wd_s = wd_scales;
  fa.y = y;
  fa.y_bf16 = y_dtype == MOE_BF16;
  fa.ws = workspace;
  return hip_status(launch_ffn_mx4(fa, (hipStream_t)stream));
}

size_t moe_decode_layer_mx4_workspace_size(int T, int k, int E_loc, int H, int I) {
  if (T < 0 || T > kMx4StreamMaxT || E_loc > kDecodeMx4MaxE || H > kDecodeMx4MaxH || !ffn_sizes_ok(T, k, E_loc, H, I)) return 0;
  return decode_layer_mx4_ws_bytes(T, k, E_loc, H, I);
}

int moe_decode_layer_mx4(const void *x, const float *w_router_packed, const float *bias, int T, int H, int E, int k,
                         int e_begin, int e_end, int I, const uint8_t *wgu_codes, const uint8_t *wgu_scales,
                         const uint8_t *wd_codes, const uint8_t *wd_scales, int32_t *topk_ids, float *topk_w, void *y,
                         int y_dtype, void *workspace, size_t workspace_bytes, void *stream) {
  if (T < 0 || T > kMx4StreamMaxT || E < 1 || E > kDecodeMx4MaxE || k < 1 || k > E || e_begin < 0 || e_end <= e_begin ||
      e_end > E || H > kDecodeMx4MaxH || !ffn_sizes_ok(T, k, e_end - e_begin, H, I))
    return MOE_ERR_SHAPE;
  if (y_dtype != MOE_F32 && y_dtype != MOE_BF16) return MOE_ERR_DTYPE;
  if (T == 0) return MOE_OK;
  if (!x || !w_router_packed || !wgu_codes || !wgu_scales || !wd_codes || !wd_scales || !topk_ids || !topk_w || !y)
    return MOE_ERR_NULL;
  const int El = e_end - e_begin;
  if (!workspace || workspace_bytes < moe_decode_layer_mx4_workspace_size(T, k, El, H, I)) return MOE_ERR_WORKSPACE;
  if (!aligned(x, 16) || !aligned(w_router_packed, 16) || !aligned(wgu_codes, 16) || !aligned(wgu_scales, 16) ||
      !aligned(wd_codes, 16) || !aligned(wd_scales, 16) || !aligned(y, 16) || !aligned(workspace, 256))
    return MOE_ERR_ALIGN;
  DecodeMx4Args a{};
  a.x = x;
  a.wr = w_router_packed;
  a.bias = bias;
  a.T = T;
  a.H = H;
  a.E = E;
  a.k = k;
  a.lo = e_begin;
  a.El = El;
  a.I = I;
  a.wgu = wgu_codes;
  a.wgu_s = wgu_scales;
  a.wd = wd_codes;
  a.wd_s = wd_scales;
  a.ids = topk_ids;
  a.gates = topk_w;
  a.y = y;
  a.y_bf16 = y_dtype == MOE_BF16;
  a.ws = workspace;
  return hip_status(launch_decode_layer_mx4(a, (hipStream_t)stream));
}

}  // extern "C"
