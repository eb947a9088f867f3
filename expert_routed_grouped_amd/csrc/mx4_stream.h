// Weight-streaming core of the MXFP4 expert FFN for few rows per expert (grouped FFN of a small batch, the
// few-token layer).
//
// With a few rows per expert the work is one read of the active experts' weights, so the split is made for
// bytes in flight, not for reuse, and the weights are loaded non-temporally (64 tokens, 128 experts of 4096 x 1536:
// gate/up 137 -> 128 us or 6.7 TB/s, down 75 -> 72 us).
//
// Gate/up: a wave takes 16 rows of an expert x 32 intermediate columns (one block of the quantised
// intermediate): 32 gate and 32 up rows of the weights, through a ring of four 128-k steps (17 KB in flight per
// wave).  With few such tiles on the chip the contraction is split over S = 2, 4 or 8 waves of the
// workgroup in pieces of 512, joined through LDS in wave order.
//
// Down: one workgroup owns 16 output columns for every token; its waves take the experts' tiles of 8 rows in
// turn (few rows per expert leave most of a 16-row operand empty; eight rows load in full lines and reach their
// lanes through LDS, 88 -> 75 us), add gate * o into a sum per wave, token and column in LDS, and the sums are
// joined in wave order at the end.  Every byte of the down weights is read by one workgroup, nothing is added
// atomically, and y is written once, rounded once.  H / 16 workgroups fill the chip from H = 4096 on; with less, fewer
// compute units work (64 tokens, 128 experts of 2048 x 768: the whole FFN 81 us).
#pragma once
#include "mx4_common.h"

namespace mx4s {

using mx4::v8i_t;

constexpr int NW = 8, NTHR = 64 * NW;  // waves and threads of a workgroup
constexpr int TM = 16;                 // rows per gate/up tile
constexpr int TD = 8;                  // rows per down tile
constexpr int MAXT = kMx4StreamMaxT;   // tokens: the per-token sums of the down half fit LDS
constexpr int GP = 64 * 4;             // floats of one row group's partial sums of a wave
constexpr int RED_FLOATS = NW * 4 * GP;

struct Half {
  const uint8_t *a, *a_s;  // activations, row-major
  const uint8_t *w, *w_s;  // packed weights
};

// How many waves share a gate/up tile when ``tiles`` of them exist: as few as keep about six waves per compute
// unit busy (S is a power of two, at most one wave per 512 of the contraction).  Whole FFN of one token, eight experts of
// 4096 x 1536: 23.9 us; 25.3 with half as many waves, 26.4 with twice; from 8 tokens on all three alike.  The few-token
// layer knows its tiles; the grouped FFN gives the most that there can be, which on a share of the experts is more.
__host__ __device__ __forceinline__ int split_for(int tiles, int H) {
  int S = 1;
  while (S < NW && tiles * S < 1536 && S * 512 < H) S *= 2;
  return S;
}

// Rows [r0, r0 + rows) (rows <= 16) of expert e, intermediate columns [c0, c0 + 32): h rows r0 .. in
// MX format FA.  src(r) is the activation row of row r.  Wave s of the S that share the tile; red: RED_FLOATS
// floats of LDS.  Every thread of the workgroup calls it (with rows = 0 where it has no tile); there are two
// barriers inside if S > 1 and none otherwise.
template <int FA, typename SRC>
__device__ __forceinline__ void gate_up_tile(const Half &p, int H, int I, int e, int c0, int r0, int rows, int S,
                                             int s, SRC src, uint8_t *h, uint8_t *hs, float *red) {
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nstep = H / 128, nch = (nstep + 3) / 4;
  f32x4_t acc[4];
#pragma unroll
  for (int g = 0; g < 4; g++) acc[g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (rows > 0 && s < nch) {
    const size_t grp = ((size_t)e * 2 * I + c0) / 16;
    const size_t gc = mx4::group_codes(H), gs = mx4::group_scales(H);
    const uint8_t *wp[4], *sp[4];
#pragma unroll
    for (int g = 0; g < 4; g++) {
      const size_t gr = grp + (g & 1) + (size_t)(g >> 1) * (I / 16);
      wp[g] = p.w + gr * gc + lane * 16;
      sp[g] = p.w_s + gr * gs + lane * 4;
    }
    const size_t row = src(r0 + min(n, rows - 1));
    const uint8_t *arow = p.a + row * mx4::code_bytes<FA>(H), *asrow = p.a_s + row * (H / 32);
    u32x4_t w[4][4];
    v8i_t a[4];
    uint32_t as[4], ws[4], wsn[4];
    // steps past the end of a short last piece read its last step again and are not used
    auto load = [&](int j, int c) __attribute__((always_inline)) {
      const int st = min(4 * c + j, nstep - 1);
#pragma unroll
      for (int g = 0; g < 4; g++) w[j][g] = __builtin_nontemporal_load((const u32x4_t *)(wp[g] + (size_t)st * mx4::kBlk));
      a[j] = mx4::act_frag<FA>(arow, st, q);
      as[j] = mx4::act_scale(asrow, st, q);
    };
    auto step = [&](auto JC, int c) __attribute__((always_inline)) {
      constexpr int j = decltype(JC)::value;
      if (4 * c + j < nstep) {
#pragma unroll
        for (int g = 0; g < 4; g++) acc[g] = mx4::mfma<FA, j>(mx4::piece4(w[j][g]), a[j], acc[g], ws[g], as[j]);
      }
    };
#pragma unroll
    for (int g = 0; g < 4; g++) ws[g] = *(const uint32_t *)(sp[g] + (size_t)s * mx4::kSblk);
#pragma unroll
    for (int j = 0; j < 4; j++) load(j, s);
    int c = s;
    for (; c + S < nch; c += S) {  // compute piece c, fetching piece c + S into the steps it frees
#pragma unroll
      for (int g = 0; g < 4; g++) wsn[g] = *(const uint32_t *)(sp[g] + (size_t)(c + S) * mx4::kSblk);
      step(std::integral_constant<int, 0>{}, c);
      load(0, c + S);
      step(std::integral_constant<int, 1>{}, c);
      load(1, c + S);
      step(std::integral_constant<int, 2>{}, c);
      load(2, c + S);
      step(std::integral_constant<int, 3>{}, c);
      load(3, c + S);
#pragma unroll
      for (int g = 0; g < 4; g++) ws[g] = wsn[g];
    }
    step(std::integral_constant<int, 0>{}, c);
    step(std::integral_constant<int, 1>{}, c);
    step(std::integral_constant<int, 2>{}, c);
    step(std::integral_constant<int, 3>{}, c);
  }
  if (S > 1) {  // the partial sums of waves s > 0 go through LDS
    if (s > 0) {
#pragma unroll
      for (int g = 0; g < 4; g++) *(f32x4_t *)(red + (wave * 4 + g) * GP + lane * 4) = acc[g];
    }
    __syncthreads();
    if (s == 0) {
      for (int v = 1; v < S; v++) {
#pragma unroll
        for (int g = 0; g < 4; g++) acc[g] += *(const f32x4_t *)(red + ((wave + v) * 4 + g) * GP + lane * 4);
      }
    }
    __syncthreads();
  }
  if (s == 0 && rows > 0) {
    float v[2][4];
#pragma unroll
    for (int g = 0; g < 2; g++)
#pragma unroll
      for (int r = 0; r < 4; r++) v[g][r] = silu_fast(acc[g][r]) * acc[2 + g][r];
    const size_t r = (size_t)r0 + n;
    mx4::store_h_block<FA>(v, n < rows, h + r * mx4::code_bytes<FA>(I), hs + r * mx4::h_scale_stride(I), c0, q);
  }
}

struct DownArgs {
  const int32_t *offsets;  // [El+1]
  const int32_t *row_token;
  const float *row_w;
  int El, T, R_cap, H, I;
  Half p;                  // h rows and the down weights
  void *y;                 // [T, H], overwritten
  const int2 *tiles;       // its tiles {first row, expert | rows << 16}, or NULL: found from the offsets
  const int *ntiles;
  uint32_t *zero;          // n_zero words to zero for the next call, or NULL
  int n_zero;
};

// LDS of the down half: sums [NW][T][16], one staged operand piece per wave, tile list {first row, expert | rows
// << 16}, and every row's token and gate, so that the loop touches memory only for operands (a load of anything
// else would wait for all of them).
__host__ __device__ constexpr int max_tiles(int T, int El) { return El + T * 32 / TD; }  // k <= 32
template <int FA>
__host__ __device__ constexpr int stage_bytes() { return TD * (int)mx4::code_bytes<FA>(512); }
template <int FA>
__host__ __device__ constexpr size_t down_lds_bytes(int T, int El, int R_cap) {
  return (size_t)NW * (T * 16 * 4 + stage_bytes<FA>()) + (size_t)max_tiles(T, El) * 8 + (size_t)R_cap * 8;
}

template <int FA, bool BF16>
__global__ __launch_bounds__(NTHR) void down_sum_kernel(DownArgs a) {
  extern __shared__ __attribute__((aligned(16))) float lds[];
  __shared__ int s_tiles;
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cap = max_tiles(a.T, a.El);
  char *stage = (char *)(lds + NW * a.T * 16) + wave * stage_bytes<FA>();
  int2 *tiles = (int2 *)((char *)(lds + NW * a.T * 16) + NW * stage_bytes<FA>());
  int2 *rowinfo = tiles + cap;  // {token, gate bits}
  float *tot = lds + wave * a.T * 16;
  if (blockIdx.x == 0 && (int)threadIdx.x < a.n_zero) a.zero[threadIdx.x] = 0;
  for (int i = lane; i < a.T * 4; i += 64) *(f32x4_t *)(tot + 4 * i) = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int i = threadIdx.x; i < a.R_cap; i += NTHR) rowinfo[i] = make_int2(a.row_token[i], __float_as_int(a.row_w[i]));
  if (a.tiles) {
    const int nt = min(*a.ntiles, cap);
    for (int i = threadIdx.x; i < nt; i += NTHR) tiles[i] = a.tiles[i];
    if (threadIdx.x == 0) s_tiles = nt;
  } else if (wave == 0) {
    int n0 = 0;
    for (int b = 0; b < a.El; b += 64) {
      const int e = b + lane;
      const int beg = e < a.El ? max(a.offsets[e], 0) : 0;
      const int c = e < a.El ? min(min(a.offsets[e + 1], a.R_cap) - beg, a.T) : 0;  // at most one row per token
      const int t = c > 0 ? (c + TD - 1) / TD : 0;
      const int at = n0 + ffn::wave_incl_scan_i(t, lane) - t;
      for (int i = 0; i < t && at + i < cap; i++)
        tiles[at + i] = make_int2(beg + i * TD, e | min(TD, c - i * TD) << 16);
      n0 += ffn::wave_sum_i(t);
    }
    if (lane == 0) s_tiles = min(n0, cap);
  }
  __syncthreads();
  const int nt = __builtin_amdgcn_readfirstlane(s_tiles);
  const int K = a.I, nstep = K / 128, nch = (nstep + 3) / 4;
  const int mine = wave < nt ? (nt - wave + NW - 1) / NW : 0;
  const int nu = mine * nch;  // units: 512-long pieces of this wave's tiles
  const size_t gc = mx4::group_codes(K), gs = mx4::group_scales(K), hss = mx4::h_scale_stride(K);

  // Ring of units: codes and scales of the weights and of the tile's rows.  The rows' codes are staged in LDS in the
  // order [step][half][quarter][row] of 16-byte pieces (E2M1: no halves), in which a lane's operand reads are
  // free of conflicts; NA loads of 64 pieces fetch them, each touching eight rows a full line (E2M1: half a line) at a time.
  constexpr int D = 4, NA = stage_bytes<FA>() / 1024;
  struct Unit {
    u32x4_t w[4], a[NA];
    uint32_t ws, as;
  } ring[D];
  // cursors of the next unit to load and to compute: tile (of this wave) and piece
  int lt = 0, lc = 0, ct = 0, cc = 0;
  auto load = [&](Unit &u) __attribute__((always_inline)) {
    const int2 d = tiles[wave + lt * NW];
    const int beg = __builtin_amdgcn_readfirstlane(d.x), er = __builtin_amdgcn_readfirstlane(d.y);
    const int e = er & 0xffff, rows = er >> 16, c = lc;
    const size_t grp = (size_t)e * (a.H / 16) + blockIdx.x;
    const uint8_t *wp = a.p.w + grp * gc + lane * 16;
    u.ws = *(const uint32_t *)(a.p.w_s + grp * gs + (size_t)c * mx4::kSblk + lane * 4);
    u.as = *(const uint32_t *)(a.p.a_s + ((size_t)beg + min(n & 7, rows - 1)) * hss + (size_t)c * 16 + 4 * q);
    const int last = nstep - 1;  // steps past the end are read again and not used
#pragma unroll
    for (int j = 0; j < 4; j++) u.w[j] = __builtin_nontemporal_load((const u32x4_t *)(wp + (size_t)min(4 * c + j, last) * mx4::kBlk));
    const uint8_t *arow = a.p.a + ((size_t)beg + min(lane & 7, rows - 1)) * mx4::code_bytes<FA>(K);
#pragma unroll
    for (int i = 0; i < NA; i++) {
      const int st = min(4 * c + (FA == mx4::FP8 ? i : 2 * i + (lane >> 5)), last);
      u.a[i] = *(const u32x4_t *)(arow + (FA == mx4::FP8 ? (size_t)st * 128 + (lane >> 3) * 16
                                                         : (size_t)st * 64 + ((lane >> 3) & 3) * 16));
    }
    if (lc + 1 < nch) lc++;
    else if (lt + 1 < mine) { lc = 0; lt++; }  // past the last unit: it again, from cache
  };
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const Unit &u) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NA; i++) *(u32x4_t *)(stage + i * 1024 + lane * 16) = u.a[i];
    auto step = [&](auto JC) __attribute__((always_inline)) {
      constexpr int j = decltype(JC)::value;
      if (4 * cc + j < nstep) {
        const char *ap = stage + (FA == mx4::FP8 ? j * 1024 : j * 512) + q * 128 + (n & 7) * 16;
        v8i_t av;
        if constexpr (FA == mx4::FP8) av = mx4::piece8(*(const u32x4_t *)ap, *(const u32x4_t *)(ap + 512));
        else av = mx4::piece4(*(const u32x4_t *)ap);
        acc = mx4::mfma<FA, j, j>(mx4::piece4(u.w[j]), av, acc, u.ws, u.as);
      }
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
    if (++cc == nch) {  // the tile is done: add gate * o to its tokens' sums
      const int2 d = tiles[wave + ct * NW];
      if (n < (d.y >> 16)) {
        const int2 ri = rowinfo[d.x + n];
        if ((unsigned)ri.x < (unsigned)a.T) {
          f32x4_t *s = (f32x4_t *)(tot + ri.x * 16 + 4 * q);
          *s += acc * __int_as_float(ri.y);
        }
      }
      acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
      cc = 0;
      ct++;
    }
  };
  if (nu > 0) {
#pragma unroll
    for (int d = 0; d < D - 1; d++) {
      load(ring[d]);
      asm volatile("" ::: "memory");  // keeps the loads in unit order, so that a wait covers one unit
    }
    for (int i = 0; i < nu; i += D) {
#pragma unroll
      for (int d = 0; d < D; d++) {
        load(ring[(d + D - 1) % D]);
        asm volatile("" ::: "memory");
        if (i + d < nu) compute(ring[d]);
      }
    }
  }
  __syncthreads();
  // join the waves' sums in wave order: thread -> token, four columns
  const int nwv = min(NW, nt);
  for (int i = threadIdx.x; i < a.T * 4; i += NTHR) {
    f32x4_t s = {0.f, 0.f, 0.f, 0.f};
    for (int v = 0; v < nwv; v++) s += *(const f32x4_t *)(lds + v * a.T * 16 + 4 * i);
    mx4::store4<BF16>(a.y, (size_t)(i >> 2) * a.H + blockIdx.x * 16 + 4 * (i & 3), s);
  }
}

}  // namespace mx4s
