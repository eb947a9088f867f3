// C ABI of the operators that train a MoE block: argument checks on the host, then launches.  Every check runs
// before anything is enqueued; no call allocates, frees or synchronises.
#include "../../include/moe.h"
#include "train.h"

namespace {

constexpr long long kMaxRows = 1LL << 28, kMaxGrid = (1LL << 31) - 1;

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }
inline bool is_float(int dt) { return dt == MOE_F32 || dt == MOE_BF16; }
inline size_t esize(int dt) { return dt == MOE_BF16 ? 2 : 4; }
inline long long tiles(long long n, int b) { return (n + b - 1) / b; }
// Whether two buffers share a byte; a NULL one shares none.
inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
  return a && b && na && nb && (uintptr_t)a < (uintptr_t)b + nb && (uintptr_t)b < (uintptr_t)a + na;
}

// Rows of a grouped call and one matrix of an expert: below 2^31 bytes each matrix, 2^47 bytes of rows.
bool grouped_ok(int El, int R_cap, int a, int b) {
  return El >= 1 && El <= 1024 && R_cap >= 0 && R_cap < kMaxRows && a >= 1 && b >= 1 && a < (1 << 24) && b < (1 << 24) &&
         (long long)a * b < (1LL << 29);
}

bool norm_sizes_ok(int T, int H) { return T >= 0 && T < (1 << 30) && H >= 1 && H <= train::kNormMaxH; }

}  // namespace

extern "C" {

int moe_grouped_mm(const void *a, const int32_t *row_index, int a_rows, const void *w, int dtype, const int32_t *offsets,
                   int E_loc, int R_cap, int N, int K, void *out, int out_dtype, unsigned flags, void *stream) {
  if (!grouped_ok(E_loc, R_cap, N, K) || a_rows < 0 || a_rows >= kMaxRows || (!row_index && a_rows < R_cap) ||
      (flags & ~MOE_MM_TRANSPOSED) != 0)
    return MOE_ERR_SHAPE;
  if ((tiles(R_cap, 32) + E_loc) * tiles(N, 32) > kMaxGrid) return MOE_ERR_SHAPE;
  if (!is_float(dtype) || !is_float(out_dtype) || (dtype == MOE_F32 && out_dtype != MOE_F32)) return MOE_ERR_DTYPE;
  if (R_cap == 0) return MOE_OK;
  if (a_rows == 0) return MOE_ERR_SHAPE;
  if (!a || !w || !offsets || !out) return MOE_ERR_NULL;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(offsets, 4) || !aligned(row_index, 4))
    return MOE_ERR_ALIGN;
  const size_t no = (size_t)R_cap * N * esize(out_dtype), e = esize(dtype);
  if (overlap(out, no, a, (size_t)a_rows * K * e) || overlap(out, no, w, (size_t)E_loc * N * K * e) ||
      overlap(out, no, offsets, (size_t)(E_loc + 1) * 4) || overlap(out, no, row_index, (size_t)R_cap * 4))
    return MOE_ERR_SHAPE;
  train::MmArgs m{};
  m.a = a;
  m.a_index = row_index;
  m.a_rows = a_rows;
  m.w = w;
  m.offsets = offsets;
  m.El = E_loc;
  m.R_cap = R_cap;
  m.N = N;
  m.K = K;
  m.out = out;
  m.bf16 = dtype == MOE_BF16;
  m.out_bf16 = out_dtype == MOE_BF16;
  m.kn = (flags & MOE_MM_TRANSPOSED) != 0;
  return hip_status(train::launch_grouped_mm(m, (hipStream_t)stream));
}

size_t moe_grouped_wgrad_workspace_size(int E_loc, int R_cap, int M, int N, int dtype) {
  if (!grouped_ok(E_loc, R_cap, M, N) || !is_float(dtype)) return 0;
  return train::wgrad_ws_bytes(E_loc, R_cap, M, N, dtype == MOE_BF16);
}

int moe_grouped_wgrad(const void *a, const int32_t *a_index, int a_rows, const void *b, const int32_t *b_index, int b_rows,
                      int dtype, const int32_t *offsets, int E_loc, int R_cap, int M, int N, void *dw, int dw_dtype,
                      void *workspace, size_t workspace_bytes, unsigned flags, void *stream) {
  if (!grouped_ok(E_loc, R_cap, M, N) || a_rows < 0 || a_rows >= kMaxRows || b_rows < 0 || b_rows >= kMaxRows ||
      (!a_index && a_rows < R_cap) || (!b_index && b_rows < R_cap) || (flags & ~MOE_WGRAD_ADD) != 0)
    return MOE_ERR_SHAPE;
  if ((long long)E_loc * tiles(M, 32) * tiles(N, 32) > kMaxGrid || (R_cap > 0 && (a_rows == 0 || b_rows == 0)))
    return MOE_ERR_SHAPE;
  if (!is_float(dtype) || !is_float(dw_dtype) || (dtype == MOE_F32 && dw_dtype != MOE_F32)) return MOE_ERR_DTYPE;
  if (!offsets || !dw || (R_cap > 0 && (!a || !b))) return MOE_ERR_NULL;
  const size_t need = moe_grouped_wgrad_workspace_size(E_loc, R_cap, M, N, dtype);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MOE_ERR_WORKSPACE;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(dw, 16) || !aligned(offsets, 4) || !aligned(a_index, 4) ||
      !aligned(b_index, 4) || (need > 0 && !aligned(workspace, 256)))
    return MOE_ERR_ALIGN;
  const size_t nd = (size_t)E_loc * M * N * esize(dw_dtype), e = esize(dtype);
  const void *ins[] = {a, b, offsets, a_index, b_index};
  const size_t bytes[] = {(size_t)a_rows * M * e, (size_t)b_rows * N * e, (size_t)(E_loc + 1) * 4, (size_t)R_cap * 4,
                          (size_t)R_cap * 4};
  for (int i = 0; i < 5; i++)
    if (overlap(dw, nd, ins[i], bytes[i]) || (need > 0 && overlap(workspace, need, ins[i], bytes[i]))) return MOE_ERR_SHAPE;
  if (need > 0 && overlap(workspace, need, dw, nd)) return MOE_ERR_SHAPE;
  train::WgradArgs g{};
  g.a = a;
  g.b = b;
  g.a_index = a_index;
  g.b_index = b_index;
  g.a_rows = a_rows;
  g.b_rows = b_rows;
  g.offsets = offsets;
  g.El = E_loc;
  g.R_cap = R_cap;
  g.M = M;
  g.N = N;
  g.dw = dw;
  g.bf16 = dtype == MOE_BF16;
  g.out_bf16 = dw_dtype == MOE_BF16;
  g.add = (flags & MOE_WGRAD_ADD) != 0;
  g.ws = workspace;
  return hip_status(train::launch_grouped_wgrad(g, (hipStream_t)stream));
}

int moe_swiglu(const void *gu, int dtype, const int32_t *offsets, const float *row_w, int E_loc, int R_cap, int I, void *h,
               void *stream) {
  if (!grouped_ok(offsets ? E_loc : 1, R_cap, 1, I)) return MOE_ERR_SHAPE;
  if (!is_float(dtype)) return MOE_ERR_DTYPE;
  if (R_cap == 0) return MOE_OK;
  if (!gu || !h) return MOE_ERR_NULL;
  if (!aligned(gu, 16) || !aligned(h, 16) || !aligned(offsets, 4) || !aligned(row_w, 4)) return MOE_ERR_ALIGN;
  const size_t nh = (size_t)R_cap * I * esize(dtype);
  if (overlap(h, nh, gu, 2 * nh) || overlap(h, nh, row_w, (size_t)R_cap * 4) ||
      overlap(h, nh, offsets, (size_t)(E_loc + 1) * 4))
    return MOE_ERR_SHAPE;
  train::SwigluArgs s{};
  s.gu = gu;
  s.offsets = offsets;
  s.row_w = row_w;
  s.El = E_loc;
  s.R_cap = R_cap;
  s.I = I;
  s.bf16 = dtype == MOE_BF16;
  s.h = h;
  return hip_status(train::launch_swiglu(s, (hipStream_t)stream));
}

int moe_swiglu_backward(const void *gu, const void *dh, int dtype, const int32_t *offsets, const float *row_w, int E_loc,
                        int R_cap, int I, void *dgu, void *h, float *d_row_w, void *stream) {
  if (!grouped_ok(offsets ? E_loc : 1, R_cap, 1, I)) return MOE_ERR_SHAPE;
  if (!is_float(dtype)) return MOE_ERR_DTYPE;
  if (R_cap == 0) return MOE_OK;
  if (!gu || !dh || !dgu) return MOE_ERR_NULL;
  if (!aligned(gu, 16) || !aligned(dh, 16) || !aligned(dgu, 16) || !aligned(h, 16) || !aligned(offsets, 4) ||
      !aligned(row_w, 4) || !aligned(d_row_w, 4))
    return MOE_ERR_ALIGN;
  const size_t n = (size_t)R_cap * I * esize(dtype), nr = (size_t)R_cap * 4, no = (size_t)(E_loc + 1) * 4;
  // dgu may be gu itself and h dh itself: a wave reads what it overwrites before it does, and nothing else reads it
  const void *outs[] = {dgu, h, d_row_w}, *ins[] = {gu, dh, row_w, offsets};
  const size_t ob[] = {2 * n, n, nr}, ib[] = {2 * n, n, nr, no};
  for (int i = 0; i < 3; i++) {
    for (int j = 0; j < 4; j++) {
      if ((i == 0 && j == 0 && dgu == gu) || (i == 1 && j == 1 && h == dh)) continue;
      if (overlap(outs[i], ob[i], ins[j], ib[j])) return MOE_ERR_SHAPE;
    }
    for (int j = 0; j < i; j++)
      if (overlap(outs[i], ob[i], outs[j], ob[j])) return MOE_ERR_SHAPE;
  }
  train::SwigluArgs s{};
  s.gu = gu;
  s.dh = dh;
  s.offsets = offsets;
  s.row_w = row_w;
  s.El = E_loc;
  s.R_cap = R_cap;
  s.I = I;
  s.bf16 = dtype == MOE_BF16;
  s.h = h;
  s.dgu = dgu;
  s.d_row_w = d_row_w;
  return hip_status(train::launch_swiglu_backward(s, (hipStream_t)stream));
}

int moe_route_backward(const int32_t *topk_ids, const float *topk_w, const float *d_topk_w, int T, int k, int E, int H,
                       const void *x, const void *w_router, int dtype, const int32_t *offsets, const int32_t *row_token,
                       const void *rows, int rows_dtype, const int32_t *rows_at, int R_cap, void *dx, int dx_dtype,
                       float *dw_router, float *d_bias, void *stream) {
  if (T < 0 || k < 1 || k > 32 || E < 1 || E > 1024 || k > E || H < 1 || H > (1 << 20) || (long long)T * k >= kMaxRows ||
      R_cap < 0 || R_cap >= kMaxRows)
    return MOE_ERR_SHAPE;
  if (!is_float(dtype) || (dx && !is_float(dx_dtype)) || (rows && !is_float(rows_dtype))) return MOE_ERR_DTYPE;
  const bool weights = dw_router || d_bias;
  if (!dx && !weights) return MOE_ERR_NULL;
  if (T > 0 && (!topk_ids || !topk_w || !d_topk_w || (dx && !w_router) || (dw_router && !x))) return MOE_ERR_NULL;
  if (weights && (!offsets || (T > 0 && !row_token))) return MOE_ERR_NULL;
  if (rows && dx && T > 0 && !rows_at) return MOE_ERR_NULL;
  if (!aligned(x, 16) || !aligned(w_router, 16) || !aligned(rows, 16) || !aligned(dx, 16) || !aligned(dw_router, 16) ||
      !aligned(topk_ids, 4) || !aligned(topk_w, 4) || !aligned(d_topk_w, 4) ||
      !aligned(offsets, 4) || !aligned(row_token, 4) || !aligned(rows_at, 4) || !aligned(d_bias, 4))
    return MOE_ERR_ALIGN;
  const size_t A = (size_t)T * k * 4, e = esize(dtype);
  const void *outs[] = {dx, dw_router, d_bias};
  const size_t ob[] = {(size_t)T * H * esize(dx_dtype), (size_t)E * H * 4, (size_t)E * 4};
  const void *ins[] = {topk_ids, topk_w, d_topk_w, x, w_router, offsets, row_token, rows, rows_at};
  const size_t ib[] = {A, A, A, (size_t)T * H * e, (size_t)E * H * e, (size_t)(E + 1) * 4, A,
                       (size_t)R_cap * H * esize(rows_dtype), A};
  for (int i = 0; i < 3; i++) {
    for (int j = 0; j < 9; j++)
      if (overlap(outs[i], ob[i], ins[j], ib[j])) return MOE_ERR_SHAPE;
    for (int j = 0; j < i; j++)
      if (overlap(outs[i], ob[i], outs[j], ob[j])) return MOE_ERR_SHAPE;
  }
  if (T == 0 && !weights) return MOE_OK;
  train::RouteGradArgs r{};
  r.ids = topk_ids;
  r.gates = topk_w;
  r.d_gates = d_topk_w;
  r.T = T;
  r.k = k;
  r.E = E;
  r.H = H;
  r.x = x;
  r.wr = w_router;
  r.bf16 = dtype == MOE_BF16;
  r.offsets = offsets;
  r.row_token = row_token;
  r.rows = rows;
  r.rows_bf16 = rows_dtype == MOE_BF16;
  r.rows_at = rows_at;
  r.R_cap = R_cap;
  r.dx = dx;
  r.dx_bf16 = dx_dtype == MOE_BF16;
  r.dwr = dw_router;
  r.dbias = d_bias;
  return hip_status(train::launch_route_grad(r, (hipStream_t)stream));
}

int moe_block_norm(const void *x, int x_dtype, const void *y, int y_dtype, const void *w_next, const void *w_post,
                   const void *gate, int w_dtype, int gate_kind, float scale, float eps, int T, int H, void *x_out, void *n,
                   float *rstd_next, float *rstd_post, void *stream) {
  if (!norm_sizes_ok(T, H) || !(eps > 0.0f) || gate_kind < 0 || gate_kind > 2) return MOE_ERR_SHAPE;
  // without a block's output there is nothing to add: the norm of x alone (arrays over no tokens may be NULL)
  if (T > 0 && ((gate != nullptr) != (gate_kind != 0) || (rstd_post && !w_post) ||
                (!y && (x_out || w_post || gate || rstd_post || scale != 1.0f))))
    return MOE_ERR_SHAPE;
  if (!is_float(x_dtype) || (y && !is_float(y_dtype)) || ((w_next || w_post || gate) && !is_float(w_dtype)))
    return MOE_ERR_DTYPE;
  if (T == 0) return MOE_OK;
  if (!x || (n != nullptr) != (w_next != nullptr) || (!n && !x_out)) return MOE_ERR_NULL;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(w_next, 16) || !aligned(w_post, 16) || !aligned(gate, 16) ||
      !aligned(x_out, 16) || !aligned(n, 16) || !aligned(rstd_next, 4) || !aligned(rstd_post, 4))
    return MOE_ERR_ALIGN;
  const size_t nx = (size_t)T * H * esize(x_dtype), w = esize(w_dtype);
  const void *outs[] = {x_out, n, rstd_next, rstd_post}, *ins[] = {x, y, w_next, w_post, gate};
  const size_t ob[] = {nx, nx, (size_t)T * 4, (size_t)T * 4};
  const size_t ib[] = {nx, (size_t)T * H * esize(y_dtype), H * w, H * w, (gate_kind == 2 ? T : H) * w};
  for (int i = 0; i < 4; i++) {
    for (int j = 0; j < 5; j++)  // the sum may replace the residual: a workgroup has read a row before it writes it
      if (!(i == 0 && j == 0 && x_out == x) && overlap(outs[i], ob[i], ins[j], ib[j])) return MOE_ERR_SHAPE;
    for (int j = 0; j < i; j++)
      if (overlap(outs[i], ob[i], outs[j], ob[j])) return MOE_ERR_SHAPE;
  }
  train::NormArgs a{};
  a.x = x;
  a.y = y;
  a.x_bf16 = x_dtype == MOE_BF16;
  a.y_bf16 = y_dtype == MOE_BF16;
  a.w_next = w_next;
  a.w_post = w_post;
  a.gate = gate;
  a.w_bf16 = w_dtype == MOE_BF16;
  a.gate_kind = gate_kind;
  a.scale = scale;
  a.eps = eps;
  a.T = T;
  a.H = H;
  a.x_out = x_out;
  a.n = n;
  a.rstd_next = rstd_next;
  a.rstd_post = rstd_post;
  return hip_status(train::launch_block_norm(a, (hipStream_t)stream));
}

size_t moe_block_norm_backward_workspace_size(int T, int H) { return norm_sizes_ok(T, H) ? train::norm_grad_ws_bytes(T, H) : 0; }

int moe_block_norm_backward(const void *x_out, int x_dtype, const void *y, int y_dtype, const void *w_next,
                            const void *w_post, const void *gate, int w_dtype, int gate_kind, float scale,
                            const float *rstd_next, const float *rstd_post, const void *dx_out, const void *dn, int T, int H,
                            void *dx, void *dy, int dy_dtype, float *dw_next, float *dw_post, float *d_gate, void *workspace,
                            size_t workspace_bytes, void *stream) {
  if (!norm_sizes_ok(T, H) || gate_kind < 0 || gate_kind > 2) return MOE_ERR_SHAPE;
  if (T > 0 && ((gate != nullptr) != (gate_kind != 0) || (!y && (w_post || gate || dy || scale != 1.0f)) ||
                (d_gate && !gate)))
    return MOE_ERR_SHAPE;
  if ((dw_next && !w_next) || (dw_post && !w_post)) return MOE_ERR_SHAPE;
  if (!is_float(x_dtype) || (y && !is_float(y_dtype)) || ((w_next || w_post || gate) && !is_float(w_dtype)))
    return MOE_ERR_DTYPE;
  if (dy && !is_float(dy_dtype)) return MOE_ERR_DTYPE;
  if (T > 0 && !dx && !dy && !dw_next && !dw_post && !d_gate) return MOE_ERR_NULL;
  if (T > 0 && ((!dn && !dx_out) || (dn && (!x_out || !w_next || !rstd_next)) || (w_post && !rstd_post))) return MOE_ERR_NULL;
  const bool columns = dw_next || dw_post || (d_gate && gate_kind == 1);
  const size_t need = moe_block_norm_backward_workspace_size(T, H);
  if (columns && need > 0 && (!workspace || workspace_bytes < need)) return MOE_ERR_WORKSPACE;
  if (!aligned(x_out, 16) || !aligned(y, 16) || !aligned(w_next, 16) || !aligned(w_post, 16) || !aligned(gate, 16) ||
      !aligned(dx_out, 16) || !aligned(dn, 16) || !aligned(dx, 16) || !aligned(dy, 16) || !aligned(dw_next, 16) ||
      !aligned(dw_post, 16) || !aligned(d_gate, 16) || !aligned(rstd_next, 4) || !aligned(rstd_post, 4) ||
      (columns && need > 0 && !aligned(workspace, 256)))
    return MOE_ERR_ALIGN;
  const size_t nx = (size_t)T * H * esize(x_dtype), ny = (size_t)T * H * esize(y_dtype), w = esize(w_dtype);
  const size_t ng = gate_kind == 2 ? T : H;
  const void *outs[] = {dx, dy, dw_next, dw_post, d_gate, columns && need > 0 ? workspace : nullptr};
  const size_t ob[] = {nx, (size_t)T * H * esize(dy_dtype), (size_t)H * 4, (size_t)H * 4, ng * 4, need};
  const void *ins[] = {x_out, y, w_next, w_post, gate, rstd_next, rstd_post, dx_out, dn};
  const size_t ib[] = {nx, ny, H * w, H * w, ng * w, (size_t)T * 4, (size_t)T * 4, nx, nx};
  for (int i = 0; i < 6; i++) {
    for (int j = 0; j < 9; j++)  // dx may replace dx_out or dn: a workgroup has read a row before it writes it
      if (!(i == 0 && j >= 7 && dx == ins[j]) && overlap(outs[i], ob[i], ins[j], ib[j])) return MOE_ERR_SHAPE;
    for (int j = 0; j < i; j++)
      if (overlap(outs[i], ob[i], outs[j], ob[j])) return MOE_ERR_SHAPE;
  }
  train::NormArgs a{};
  a.x = x_out;
  a.y = y;
  a.x_bf16 = x_dtype == MOE_BF16;
  a.y_bf16 = y_dtype == MOE_BF16;
  a.w_next = w_next;
  a.w_post = w_post;
  a.gate = gate;
  a.w_bf16 = w_dtype == MOE_BF16;
  a.gate_kind = gate_kind;
  a.scale = scale;
  a.T = T;
  a.H = H;
  a.rn = rstd_next;
  a.rp = rstd_post;
  a.dx_out = dx_out;
  a.dn = dn;
  a.dx = dx;
  a.dy = dy;
  a.dy_bf16 = dy_dtype == MOE_BF16;
  a.dw_next = dw_next;
  a.dw_post = dw_post;
  a.d_gate = d_gate;
  a.ws = columns ? workspace : nullptr;
  if (T == 0 && !columns) return MOE_OK;
  return hip_status(train::launch_block_norm_backward(a, (hipStream_t)stream));
}

}  // extern "C"
