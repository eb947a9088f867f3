// Grouped expert FFN with MXFP4 weights (moe_grouped_ffn_mx4) for gfx950: the tile kernel.
//
// h = Q(silu(G) U), G, U = Wgu a; o = Wd h; y[t] = sum over t's rows of row_w o, in four launches: the
// activation scales into lane order (a byte per 32 values), gate/up, down (rows scaled by their gate into the
// workspace, in y's type) and the sum to token order, which adds a token's rows in slot order, so the result does
// not depend on scheduling.
//
// A tile is up to BM rows of one expert (equal tiles per expert, rounded to 32 rows) x 256 weight rows, eight
// waves as 2 (rows) x 4 (weight rows), K in steps of 128.  The weights are the first operand of
// v_mfma_scale_f32_16x16x128_f8f6f4, so an accumulator holds four neighbouring output columns of one token: the
// gate/up epilogue finds a 32-column block of h in four lanes, and the down epilogue stores neighbouring columns.
// Both operands go from memory to LDS by buffer loads (no registers, no address arithmetic in the loop) into a
// ring of RD slots, RD - 1 steps ahead; each slot holds them in the order in which the operand reads are
// contiguous, 1 KB pieces that one wave's load fills: packed weight blocks as they are, eight rows x 128 bytes
// of E4M3 rows, 16 rows x 64 bytes of E2M1 rows.  Scales go straight to registers, one dword per lane and 16 rows
// for four steps, a byte of it per step.  Every wave issues the same loads every step (past the last step they
// fetch it again into slots nobody reads), so the wait at the top of a step is a fixed count; one barrier per
// step.
//
// BM is 256, or 64 where an expert has few rows (the tile is then bound by the weights' bytes: a smaller
// activation slot leaves room for a deeper ring).
#include "mx4_common.h"

#include <utility>

namespace {

using ffn::TileParams;
using mx4::v8i_t;

constexpr int BN = 256, NTHR = 512, NWV = NTHR / 64;

struct Mx4Params {
  TileParams tp;               // offsets, row_token, row_w, El, H, I, R_cap, T; a / w / out: codes (out: rows for down)
  const uint8_t *a_scales;     // lane order, mx4::h_scale_stride(K) bytes a row
  const uint8_t *w_scales;     // packed
  uint8_t *out_scales;         // gate/up: h scales
};

typedef __attribute__((address_space(3))) void lds_void;
constexpr uint32_t kRsrcWord3 = 0x00020000;  // raw buffer, 32-bit data format

template <int FA, int BM>
struct Lay {
  static constexpr int AROW = FA == mx4::FP8 ? 128 : 64;     // activation bytes of a row and step
  static constexpr int A_BYTES = BM * AROW, W_BYTES = BN * 64;
  static constexpr int SLOT = A_BYTES + W_BYTES;
  static constexpr int RD = BM == 64 ? 6 : FA == mx4::FP8 ? 3 : 4;  // slots of the ring
  static constexpr int NA = (A_BYTES / 1024 + NWV - 1) / NWV, NL = NA + W_BYTES / 1024 / NWV;  // loads per wave and step
  static constexpr int BYTES = RD * SLOT;
  static_assert(BYTES <= 160 * 1024 && RD >= 3, "fits the LDS of one CU");
};

struct Src {
  __amdgpu_buffer_rsrc_t ra, rw, rsa, rsw;  // activations, this expert's weights, and their scales
  uint32_t off[6];                          // this lane's bytes of its wave's pieces at step 0, activations first
};

// Loads U0 .. U1 - 1 of the NL that this wave issues for step st into ring slot SLOTI (fewer activation pieces than
// waves: some are fetched twice).
template <int FA, int BM, int SLOTI, int U0, int U1>
__device__ __forceinline__ void load_pieces(const Src &src, int st, int wave, char *lds) {
  using L = Lay<FA, BM>;
  const uint32_t sa = (uint32_t)st * L::AROW, sw = (uint32_t)st * mx4::kBlk;
#pragma unroll
  for (int u = U0; u < U1; u++) {
    if (u < L::NA)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          src.ra, (lds_void *)(lds + SLOTI * L::SLOT + (wave + NWV * u) % (L::A_BYTES / 1024) * 1024), 16, src.off[u],
          sa, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          src.rw, (lds_void *)(lds + SLOTI * L::SLOT + L::A_BYTES + (wave + NWV * (u - L::NA)) * 1024), 16, src.off[u],
          sw, 0, 0);
  }
}

// MODE 0: gate/up + SwiGLU -> h.  MODE 1: down -> gated rows.  NB: 16-row blocks of this wave.
template <int MODE, int FA, bool BF16, int BM, int NB>
__device__ __forceinline__ void body(const Mx4Params &mp, const Src &src, int K, int nt, int rbase, int mvalid, int wave,
                                     int lane, int arow0, int wn, const uint32_t (&wgrp)[4], const uint32_t (&sao)[8],
                                     char *lds) {
  using L = Lay<FA, BM>;
  const TileParams &p = mp.tp;
  const int n = lane & 15, q = lane >> 4;
  const int nstep = K / 128, nch = (nstep + 3) / 4;
  f32x4_t acc[NB][4];
#pragma unroll
  for (int i = 0; i < NB; i++)
#pragma unroll
    for (int g = 0; g < 4; g++) acc[i][g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const uint32_t gs = (uint32_t)mx4::group_scales(K);
  uint32_t ws[4], as[NB], wsn[4], asn[NB];
  auto scales = [&](uint32_t(&w)[4], uint32_t(&a)[NB], int c) __attribute__((always_inline)) {
#pragma unroll
    for (int g = 0; g < 4; g++)
      w[g] = __builtin_amdgcn_raw_buffer_load_b32(src.rsw, lane * 4, (int)(wgrp[g] * gs + (uint32_t)c * mx4::kSblk), 0);
#pragma unroll
    for (int i = 0; i < NB; i++) a[i] = __builtin_amdgcn_raw_buffer_load_b32(src.rsa, (int)sao[i], c * 16, 0);
  };
  // LDS bytes of this lane's operands inside a slot
  const uint32_t wbase = L::A_BYTES + (uint32_t)wn * 4096u + lane * 16u;
  const uint32_t abase = FA == mx4::FP8
                             ? (uint32_t)(arow0 >> 3) * 1024u + (uint32_t)(n >> 3) * 1024u + q * 128u + (n & 7) * 16u
                             : (uint32_t)(arow0 >> 4) * 1024u + lane * 16u;
  scales(wsn, asn, 0);
  asm volatile("" ::: "memory");
  [&]<int... D>(std::integer_sequence<int, D...>) __attribute__((always_inline)) {
    (load_pieces<FA, BM, D, 0, L::NL>(src, min(D, nstep - 1), wave, lds), ...);
  }(std::make_integer_sequence<int, L::RD - 1>{});
  // step kt = IDX modulo PER: ring slot and scale byte are compile-time constants
  constexpr int PER = L::RD % 4 == 0 ? L::RD : L::RD % 2 == 0 ? 2 * L::RD : 4 * L::RD;
  auto step = [&](auto IC, int kt) __attribute__((always_inline)) {
    constexpr int IDX = decltype(IC)::value, j = IDX % 4, S = IDX % L::RD, SN = (IDX + L::RD - 1) % L::RD;
    if (kt >= nstep) return;
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L::NL *(L::RD - 2)) : "memory");
    asm volatile("s_barrier" ::: "memory");
    if constexpr (j == 0) {
#pragma unroll
      for (int g = 0; g < 4; g++) ws[g] = wsn[g];
#pragma unroll
      for (int i = 0; i < NB; i++) as[i] = asn[i];
      scales(wsn, asn, min((kt >> 2) + 1, nch - 1));
      asm volatile("" ::: "memory");
    }
    auto act = [&](int i) __attribute__((always_inline)) {
      if constexpr (FA == mx4::FP8)
        return mx4::piece8(*(const u32x4_t *)(lds + abase + (S * L::SLOT + i * 2048)),
                           *(const u32x4_t *)(lds + abase + (S * L::SLOT + i * 2048 + 512)));
      else
        return mx4::piece4(*(const u32x4_t *)(lds + abase + (S * L::SLOT + i * 1024)));
    };
    v8i_t w[4], a[2];
#pragma unroll
    for (int g = 0; g < 4; g++) w[g] = mx4::piece4(*(const u32x4_t *)(lds + wbase + (S * L::SLOT + g * 1024)));
    a[0] = act(0);
    const int stn = min(kt + L::RD - 1, nstep - 1);
    // block i: fetch the next operand and a share of the coming step, then multiply
    auto block = [&](auto I) __attribute__((always_inline)) {
      constexpr int i = decltype(I)::value;
      if constexpr (i + 1 < NB) a[(i + 1) & 1] = act(i + 1);
      load_pieces<FA, BM, SN, L::NL * i / NB, L::NL *(i + 1) / NB>(src, stn, wave, lds);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int g = 0; g < 4; g++) acc[i][g] = mx4::mfma<FA, j, j>(w[g], a[i & 1], acc[i][g], ws[g], as[i]);
    };
    [&]<int... I>(std::integer_sequence<int, I...>) __attribute__((always_inline)) {
      (block(std::integral_constant<int, I>{}), ...);
    }(std::make_integer_sequence<int, NB>{});
  };
  for (int kt = 0; kt < nstep; kt += PER)
    [&]<int... IDX>(std::integer_sequence<int, IDX...>) __attribute__((always_inline)) {
      (step(std::integral_constant<int, IDX>{}, kt + IDX), ...);
    }(std::make_integer_sequence<int, PER>{});
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS outlives the workgroup
  // acc[i][g][r]: tile row arow0 + 16 i + n, weight row 16 g + 4 q + r of this wave's 64
#pragma unroll
  for (int i = 0; i < NB; i++) {
    const int m = 16 * i + n;
    const bool on = m < mvalid;
    const size_t row = (size_t)(rbase + m);
    if constexpr (MODE == 0) {
      float v[2][4];
#pragma unroll
      for (int g = 0; g < 2; g++)
#pragma unroll
        for (int r = 0; r < 4; r++) v[g][r] = silu_fast(acc[i][g][r]) * acc[i][2 + g][r];
      mx4::store_h_block<FA>(v, on, (uint8_t *)p.out + row * mx4::code_bytes<FA>(p.I),
                             mp.out_scales + row * mx4::h_scale_stride(p.I), nt * 128 + wn * 32, q);
    } else if (on) {
      const float w = p.row_w[row];
#pragma unroll
      for (int g = 0; g < 4; g++) {
        const int col = nt * BN + wn * 64 + 16 * g + 4 * q;
        if (col < p.H) mx4::store4<BF16>(p.out, row * p.H + col, acc[i][g] * w);
      }
    }
  }
}

template <int MODE, int FA, bool BF16, int BM>
__global__ __launch_bounds__(NTHR, 1) void ffn_mx4_kernel(Mx4Params mp) {
  using L = Lay<FA, BM>;
  __shared__ __attribute__((aligned(1024))) char lds[L::BYTES];
  const TileParams &p = mp.tp;
  const int K = MODE == 0 ? p.H : p.I, Nw = MODE == 0 ? 2 * p.I : p.H;
  const int NT = MODE == 0 ? p.I / 128 : (p.H + BN - 1) / BN;
  int e, nt, mt, mtiles;
  if (!ffn::locate_tile<BM>(p, NT, e, nt, mt, mtiles)) return;
  e = __builtin_amdgcn_readfirstlane(e);  // the same in every lane: keep them scalar
  nt = __builtin_amdgcn_readfirstlane(nt);
  mt = __builtin_amdgcn_readfirstlane(mt);
  mtiles = __builtin_amdgcn_readfirstlane(mtiles);
  const int beg = p.offsets[e], cnt = p.offsets[e + 1] - beg;
  const int trows = __builtin_amdgcn_readfirstlane(min(BM, (((cnt + mtiles - 1) / mtiles) + 31) & ~31));
  const int r0 = beg + mt * trows;
  const int rows = min(trows, min(beg + cnt, p.R_cap) - r0);
  if (rows <= 0) return;
  const int half = trows >> 1;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3, n = lane & 15, q = lane >> 4;
  const int mvalid = min(rows - wm * half, half);

  const uint32_t arb = (uint32_t)mx4::code_bytes<FA>(K), ass = (uint32_t)mx4::h_scale_stride(K);
  const uint32_t gc = (uint32_t)mx4::group_codes(K);
  auto a_row = [&](int row) -> uint32_t {  // source row of tile row ``row`` (rows past the end repeat the last)
    const int r = r0 + min(row, rows - 1);
    return MODE == 0 ? min((uint32_t)p.row_token[r], (uint32_t)p.T - 1u) : (uint32_t)r;
  };
  auto w_group = [&](int i) -> uint32_t {  // weight group of LDS piece i
    if constexpr (MODE == 0) return (uint32_t)(nt * 8 + (i >> 2) * 2 + (i & 1) + ((i >> 1) & 1) * (p.I / 16));
    else return (uint32_t)min(nt * 16 + i, p.H / 16 - 1);
  };
  Src src;
  const uint32_t arows = MODE == 0 ? (uint32_t)p.T : (uint32_t)p.R_cap;
  const size_t wexp = (size_t)e * (Nw / 16);
  src.ra = __builtin_amdgcn_make_buffer_rsrc((void *)p.a, (short)0, (int)(arows * arb), kRsrcWord3);
  src.rsa = __builtin_amdgcn_make_buffer_rsrc((void *)mp.a_scales, (short)0, (int)(arows * ass), kRsrcWord3);
  src.rw = __builtin_amdgcn_make_buffer_rsrc((void *)((const char *)p.w + wexp * gc), (short)0, (int)(Nw / 16 * gc),
                                             kRsrcWord3);
  src.rsw = __builtin_amdgcn_make_buffer_rsrc((void *)(mp.w_scales + wexp * mx4::group_scales(K)), (short)0,
                                              (int)(Nw / 16 * mx4::group_scales(K)), kRsrcWord3);
#pragma unroll
  for (int u = 0; u < L::NA; u++) {
    const int b = (wave + NWV * u) % (L::A_BYTES / 1024);
    src.off[u] = FA == mx4::FP8 ? a_row(b * 8 + (lane & 7)) * arb + (uint32_t)(lane >> 3) * 16u
                                 : a_row(b * 16 + n) * arb + (uint32_t)q * 16u;
  }
#pragma unroll
  for (int u = 0; u < 2; u++) src.off[L::NA + u] = w_group(wave + NWV * u) * gc + (uint32_t)lane * 16u;
  const int arow0 = wm * half, rbase = r0 + arow0;
  uint32_t wgrp[4], sao[8];
#pragma unroll
  for (int g = 0; g < 4; g++) wgrp[g] = __builtin_amdgcn_readfirstlane(w_group(wn * 4 + g));
#pragma unroll
  for (int i = 0; i < BM / 32; i++) sao[i] = a_row(arow0 + 16 * i + n) * ass + 4u * q;
  const int nb = __builtin_amdgcn_readfirstlane(min(half >> 4, (max(mvalid, 1) + 15) >> 4));
#define MX4_BODY(NB) body<MODE, FA, BF16, BM, NB>(mp, src, K, nt, rbase, mvalid, wave, lane, arow0, wn, wgrp, sao, lds)
  if constexpr (BM == 64) {
    if (nb == 1) MX4_BODY(1);
    else MX4_BODY(2);
  } else {
    switch (nb) {
      case 1: MX4_BODY(1); break;
      case 2: MX4_BODY(2); break;
      case 3:
      case 4: MX4_BODY(4); break;
      case 5:
      case 6: MX4_BODY(6); break;
      default: MX4_BODY(8); break;
    }
  }
#undef MX4_BODY
}

// Activation scales [T, K/32] into lane order: dword q of piece c of a row has the scales 16c + 4j + q, j = 0 .. 3
// (0 past the end of the row).
__global__ __launch_bounds__(256) void lane_scales_kernel(const uint8_t *__restrict__ s, int T, int K,
                                                          uint32_t *__restrict__ out) {
  const int kb = K / 32, dw = (K + 511) / 512 * 4;
  const long long total = (long long)T * dw;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (long long)gridDim.x * blockDim.x) {
    const long long t = i / dw;
    const int d = (int)(i - t * dw), c = d >> 2, q = d & 3;
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int b = 16 * c + 4 * j + q;
      if (b < kb) w |= (uint32_t)s[t * kb + b] << (8 * j);
    }
    out[i] = w;
  }
}

// y[t] = sum of t's rows in slot order; a slot without a row (or with one out of range) adds nothing.
template <bool BF16>
__global__ __launch_bounds__(256) void sum_rows_kernel(const void *__restrict__ rows, const int32_t *__restrict__ token_row,
                                                       int T, int k, int R_cap, int H, void *__restrict__ y) {
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    for (int c = threadIdx.x * 4; c < H; c += blockDim.x * 4) {
      f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
      for (int j = 0; j < k; j++) {
        const int r = token_row[(size_t)t * k + j];
        if ((unsigned)r >= (unsigned)R_cap) continue;
        const size_t i = (size_t)r * H + c;
        if constexpr (BF16) {
          const uint2 v = *(const uint2 *)((const uint16_t *)rows + i);
          acc += f32x4_t{bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
        } else {
          acc += *(const f32x4_t *)((const float *)rows + i);
        }
      }
      mx4::store4<BF16>(y, (size_t)t * H + c, acc);
    }
  }
}

// Workspace: h codes [R_cap, I] (a byte each, half of it used by E2M1), h scales, and for the tile kernel the
// activation scales in lane order and the rows [R_cap, H].
size_t h_bytes(int R_cap, int I) { return align_up((size_t)R_cap * I, 256); }
size_t hs_bytes(int R_cap, int I) { return align_up((size_t)R_cap * mx4::h_scale_stride(I), 256); }
size_t as_bytes(int T, int H) { return align_up((size_t)T * mx4::h_scale_stride(H), 256); }

template <int FA, bool BF16, int BM>
hipError_t launch_tiles(const FfnMx4Args &a, hipStream_t s) {
  uint8_t *h = (uint8_t *)a.ws, *hs = h + h_bytes(a.R_cap, a.I), *as = hs + hs_bytes(a.R_cap, a.I);
  uint8_t *rows = as + as_bytes(a.T, a.H);
  const long long dwords = (long long)a.T * (mx4::h_scale_stride(a.H) / 4);
  hipLaunchKernelGGL(lane_scales_kernel, dim3((unsigned)(dwords < (1 << 20) ? (dwords + 255) / 256 : 4096)), dim3(256), 0,
                     s, a.a_s, a.T, a.H, (uint32_t *)as);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  Mx4Params p{};
  p.tp.offsets = a.offsets;
  p.tp.row_token = a.row_token;
  p.tp.row_w = a.row_w;
  p.tp.El = a.El;
  p.tp.H = a.H;
  p.tp.I = a.I;
  p.tp.R_cap = a.R_cap;
  p.tp.T = a.T;
  const long long mt1 = ((long long)a.R_cap + (long long)a.El * (BM - 1)) / BM;
  const long long mt2 = (long long)a.El * ceil_div_i(a.T, BM);
  const int mt = (int)(mt1 < mt2 ? mt1 : mt2);
  Mx4Params g = p;
  g.tp.a = a.a;
  g.a_scales = as;
  g.tp.w = a.wgu;
  g.w_scales = a.wgu_s;
  g.tp.out = h;
  g.out_scales = hs;
  hipLaunchKernelGGL((ffn_mx4_kernel<0, FA, false, BM>), dim3(mt * (a.I / 128)), dim3(NTHR), 0, s, g);
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  Mx4Params d = p;
  d.tp.a = h;
  d.a_scales = hs;
  d.tp.w = a.wd;
  d.w_scales = a.wd_s;
  d.tp.out = rows;
  hipLaunchKernelGGL((ffn_mx4_kernel<1, FA, BF16, BM>), dim3(mt * ceil_div_i(a.H, BN)), dim3(NTHR), 0, s, d);
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(sum_rows_kernel<BF16>, dim3(a.T < 16384 ? a.T : 16384), dim3(256), 0, s, rows, a.token_row, a.T,
                     a.k, a.R_cap, a.H, a.y);
  return hipGetLastError();
}

template <int FA, bool BF16>
hipError_t launch(const FfnMx4Args &a, hipStream_t s) {
  if ((long long)a.R_cap <= 64LL * a.El) return launch_tiles<FA, BF16, 64>(a, s);
  return launch_tiles<FA, BF16, 256>(a, s);
}

}  // namespace

size_t ffn_mx4_ws_bytes(int T, int R_cap, int H, int I, int y_bf16) {
  size_t b = h_bytes(R_cap, I) + hs_bytes(R_cap, I);
  if (T > kMx4StreamMaxT) b += as_bytes(T, H) + align_up((size_t)R_cap * H * (y_bf16 ? 2 : 4), 256);
  return b;
}

hipError_t launch_ffn_mx4(const FfnMx4Args &a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  if (a.T <= kMx4StreamMaxT) {
    uint8_t *h = (uint8_t *)a.ws;
    return launch_ffn_mx4_stream(a, h, h + h_bytes(a.R_cap, a.I), s);
  }
  if (a.a_fp4) return a.y_bf16 ? launch<mx4::FP4, true>(a, s) : launch<mx4::FP4, false>(a, s);
  return a.y_bf16 ? launch<mx4::FP8, true>(a, s) : launch<mx4::FP8, false>(a, s);
}
