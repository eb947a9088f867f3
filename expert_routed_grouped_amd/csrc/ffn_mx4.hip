// Grouped expert FFN with MXFP4 weights (moe_grouped_ffn_mx4) for gfx950: the tile kernel.
//
// h = Q(silu(G) U), G, U = Wgu a; o = Wd h; y[t] = sum over t's rows of row_w o, in four launches: the tile lists
// and the activation scales in lane order, gate/up, down (rows scaled by their gate into the workspace, in y's type)
// and the sum to token order, which adds a token's rows in slot order, so the result does not depend on scheduling.
//
// A tile is up to BM rows of one expert (equal tiles per expert, rounded to 32 rows) x 256 weight rows, K in steps of
// 128.  Eight waves multiply, as 2 (rows) x 4 (weight rows); the weights are the first operand of
// v_mfma_scale_f32_16x16x128_f8f6f4, so an accumulator holds four neighbouring output columns of one token: the
// gate/up epilogue finds a 32-column block of h in four lanes, and the down epilogue stores neighbouring columns.
// Four more waves load, from memory straight to LDS, into rings that run two to five steps ahead: packed weight blocks
// as they are, 128-byte lines of activation rows with their 16-byte chunks swizzled, and every four steps the scales
// of four steps.  Waves of their own for this, because a wave that multiplies and loads stalls its products at every
// load that finds the address unit busy, and waits for its stores before it can count its loads (6000 tokens with
// E2M1 activations: gate/up 430 us without, 375 with).  Every loading wave issues the same loads every step, so its wait
// at the top of a step is a fixed count; one barrier per step.
//
// One workgroup per compute unit works through a list of tiles (written by the launch before), and its loading
// waves run into the next tile while the others finish one.
//
// Times here and below are the shortest of 20 calls under a trace; medians are a few percent longer (6000 tokens: gate/up
// 538 us with E4M3 activations, 370 with E2M1, down 302 and 245).
//
// What bounds it (32 experts x 384 rows, K = 8192, 4096 weight rows): with E4M3 activations 292 us or 2.8 PFLOP/s,
// what a large fp8 library product reaches; the loads alone take 246 us, the products alone 239.  With E2M1 213 us or 3.9
// PFLOP/s, loads alone 190, products alone 161: the path from L2 and beyond to LDS, 42 KB per us and compute unit of
// the 47 that the Infinity Cache gives (135 when L2 holds everything).  Touching the weights' lines eight steps ahead
// made it slower (254 us), and so did weights laid out tile by tile (227 us) and two workgroups of 128 weight rows on a
// compute unit, which load more bytes per product (535 us instead of 440 for the 6000 tokens' gate/up).
#include "mx4_common.h"

#include <utility>

namespace {

using ffn::TileParams;
using mx4::v8i_t;

// Waves 0 .. 7 multiply, waves 8 .. 11 load.
constexpr int BN = 256, NC = 8, NP = 4, NTHR = (NC + NP) * 64, NCU = 256;

struct Mx4Params {
  TileParams tp;               // offsets, row_token, row_w, El, H, I, R_cap, T; a / w / out: codes (out: rows for down)
  const uint8_t *a_scales;     // lane order, mx4::h_scale_stride(K) bytes a row
  const uint8_t *w_scales;     // packed
  uint8_t *out_scales;         // gate/up: h scales
  const int4 *tiles;           // {expert, N tile, first row, rows | rows of a wave << 16}
  const int *ntiles;
};

typedef __attribute__((address_space(3))) void lds_void;
constexpr uint32_t kRsrcWord3 = 0x00020000;  // raw buffer, 32-bit data format

template <int FA, int BM>
struct Lay {
  // Activations come as 128 bytes of a row, a whole cache line: one step of E4M3, two of E2M1.  Of those, half the rows
  // come with one step's loads and half with the next's, a step ahead of the weights.
  static constexpr int PS = FA == mx4::FP8 ? 1 : 2;
  static constexpr int A_BYTES = BM * 128, W_BYTES = BN * 64;
  static constexpr int SSLOT = BM * 16 + BN / 16 * 256;      // scales of four steps
  static constexpr int ROWS = BM * 4;                        // a word per row: tokens (gate/up) or gates (down)
  static constexpr int a_slots(int rd) { return PS == 1 ? rd : rd / 2 + 1; }
  static constexpr int bytes(int rd) { return a_slots(rd) * A_BYTES + rd * W_BYTES + 2 * SSLOT + ROWS; }
  static constexpr int ring(int rd) { return bytes(rd) <= 163840 ? rd : ring(rd - PS); }
  static constexpr int RD = ring(6), RA = a_slots(RD);       // slots of the rings of weights and activations
  static constexpr int W0 = RA * A_BYTES, SCALES = W0 + RD * W_BYTES, ROW0 = SCALES + 2 * SSLOT, BYTES = ROW0 + ROWS;
  static constexpr int NA = A_BYTES / 1024 / NP / PS, NW = W_BYTES / 1024 / NP, NL = NA + NW;  // loads per loading wave and step
  static constexpr int SA = BM / 64, SP = SA + 4, NS = (SP + NP - 1) / NP;  // scale pieces: activations, all; loads a wave
  static_assert(RD >= 3 && A_BYTES % (1024 * NP * PS) == 0, "two steps ahead; whole pieces");
  // Steps that a tile takes.  A short one idles, so that loads reach only one tile ahead.
  static __host__ __device__ int steps(int nstep) {
    const int least = RD - 2 + PS, n = PS == 1 ? nstep : (nstep + 1) & ~1;
    return n > least ? n : least;
  }
  // Load u of a wave fetches scale piece scale_piece(wave, u); past the last one a weight piece again.
  static __device__ __forceinline__ int scale_piece(int pw, int u) {
    const int b = pw + NP * u;
    return b < SP ? b : SA + (b & 3);
  }
};

// 16 bytes per lane from memory to 1 KB of LDS.
__device__ __forceinline__ void dma(const __amdgpu_buffer_rsrc_t &r, char *to, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)to, 16, voff, soff, 0, 0);
}

// The same for lines that are read once.
__device__ __forceinline__ void dma_once(const __amdgpu_buffer_rsrc_t &r, char *to, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)to, 16, voff, soff, 0, 2);
}

// The workgroup's share of the tile list.  Workgroups go round-robin over the 8 XCDs: XCD x takes the x-th eighth of
// the list, its workgroups in turn, so that the tiles of one expert, which share operands, meet in one L2.  The
// list is read by scalar loads.
typedef int i32x4_t __attribute__((ext_vector_type(4)));
struct Share {
  const __attribute__((address_space(4))) i32x4_t *list;
  int at, end, per;
  __device__ __forceinline__ explicit Share(const Mx4Params &mp) {
    list = (const __attribute__((address_space(4))) i32x4_t *)(uintptr_t)mp.tiles;
    const int total = *(const __attribute__((address_space(4))) int *)(uintptr_t)mp.ntiles, xcd = blockIdx.x & 7;
    const int qt = total >> 3, rem = total & 7;
    per = gridDim.x >> 3;
    end = xcd * qt + min(xcd, rem) + qt + (xcd < rem ? 1 : 0);
    at = xcd * qt + min(xcd, rem) + (blockIdx.x >> 3);
  }
};

// ---------------------------------------------------------------- the loading waves
// A tile as one loading wave sees it.
template <int FA, int BM>
struct Source {
  __amdgpu_buffer_rsrc_t rw, rs[Lay<FA, BM>::NS];  // its expert's weights; the scales this wave fetches
  uint32_t off[Lay<FA, BM>::NA * Lay<FA, BM>::PS], woff[Lay<FA, BM>::NW];  // this lane's bytes of its wave's pieces at step 0
  uint32_t soff[Lay<FA, BM>::NS];                  // and of its scales
  int r0, rows;
};

template <int MODE, int FA, int BM>
__device__ __forceinline__ void load_tiles(const Mx4Params &mp, Share sh, int pw, int lane, char *lds) {
  using L = Lay<FA, BM>;
  const TileParams &p = mp.tp;
  const int K = MODE == 0 ? p.H : p.I, Nw = MODE == 0 ? 2 * p.I : p.H;
  const int nstep = K / 128, nch = (nstep + 3) / 4, nst = L::steps(nstep);
  const int n = lane & 15, q = lane >> 4;
  const uint32_t arb = (uint32_t)mx4::code_bytes<FA>(K), ass = (uint32_t)mx4::h_scale_stride(K);
  const uint32_t gc = (uint32_t)mx4::group_codes(K), gs = (uint32_t)mx4::group_scales(K);
  const uint32_t arows = MODE == 0 ? (uint32_t)p.T : (uint32_t)p.R_cap;
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc((void *)p.a, (short)0, (int)(arows * arb), kRsrcWord3);
  const __amdgpu_buffer_rsrc_t rsa =
      __builtin_amdgcn_make_buffer_rsrc((void *)mp.a_scales, (short)0, (int)(arows * ass), kRsrcWord3);
  const __amdgpu_buffer_rsrc_t rrow = __builtin_amdgcn_make_buffer_rsrc(
      MODE == 0 ? (void *)p.row_token : (void *)p.row_w, (short)0, p.R_cap * 4, kRsrcWord3);

  // What of a tile needs its description only.
  auto describe = [&](Source<FA, BM> &t, i32x4_t d) __attribute__((always_inline)) {
    const int nt = d.y;
    const size_t wexp = (size_t)d.x * (Nw / 16);
    t.r0 = d.z;
    t.rows = d.w & 0xffff;
    t.rw = __builtin_amdgcn_make_buffer_rsrc((void *)((const char *)p.w + wexp * gc), (short)0, (int)(Nw / 16 * gc),
                                             kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rsw =
        __builtin_amdgcn_make_buffer_rsrc((void *)(mp.w_scales + wexp * gs), (short)0, (int)(Nw / 16 * gs), kRsrcWord3);
    auto group = [&](int i) -> uint32_t {  // weight group of LDS piece i
      if constexpr (MODE == 0) return (uint32_t)(nt * 8 + (i >> 2) * 2 + (i & 1) + ((i >> 1) & 1) * (p.I / 16));
      else return (uint32_t)min(nt * 16 + i, p.H / 16 - 1);
    };
#pragma unroll
    for (int u = 0; u < L::NW; u++) t.woff[u] = group(pw + NP * u) * gc + (uint32_t)lane * 16u;
#pragma unroll
    for (int u = 0; u < L::NS; u++) {
      const int b = L::scale_piece(pw, u);
      t.rs[u] = b < L::SA ? rsa : rsw;
      if (b >= L::SA) t.soff[u] = group((b - L::SA) * 4 + q) * gs + (uint32_t)n * 16u;
    }
  };
  // A word per row of the tile to LDS, rows past its end as its last: the source rows' tokens or the gates.  Not into
  // registers: for such a load the compiler waits until nothing younger is under way either, i.e. for the whole ring.
  auto fetch_rows = [&](const Source<FA, BM> &t) __attribute__((always_inline)) {
    const int piece = pw % (BM / 64);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rrow, (lds_void *)(lds + L::ROW0 + piece * 256), 4,
                                             (t.r0 + min(piece * 64 + lane, t.rows - 1)) * 4, 0, 0, 0);
  };
  // What of a tile needs its rows' tokens: the bytes of this lane's activation pieces and scales.
  auto place = [&](Source<FA, BM> &t) __attribute__((always_inline)) {
    auto src = [&](int row) -> uint32_t {
      const uint32_t r = MODE == 0 ? *(const uint32_t *)(lds + L::ROW0 + row * 4) : (uint32_t)(t.r0 + min(row, t.rows - 1));
      return min(r, arows - 1);
    };
#pragma unroll
    for (int u = 0; u < L::NA * L::PS; u++) {
      const int row = (pw + NP * u) * 8 + (lane >> 3), chunk = (lane & 7) ^ (row >> 1 & 7);
      t.off[u] = src(row) * arb + (uint32_t)chunk * 16u;
    }
#pragma unroll
    for (int u = 0; u < L::NS; u++)
      if (L::scale_piece(pw, u) < L::SA) t.soff[u] = src(L::scale_piece(pw, u) * 64 + lane) * ass;
  };

  // The stream of loads runs RD - 1 steps ahead of the products (E2M1 activations: RD), into the next tile when a
  // tile's steps are all on their way.
  __amdgpu_buffer_rsrc_t rw;
  uint32_t off[L::NA * L::PS], woff[L::NW];
  int as = 0, ws = 0, aslot = 0, wslot = 0;  // steps of activations and weights so far; the slots they go to
  auto start_a = [&](const Source<FA, BM> &t) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < L::NA * L::PS; u++) off[u] = t.off[u];
    as = 0;
  };
  auto start_w = [&](const Source<FA, BM> &t) __attribute__((always_inline)) {
    rw = t.rw;
#pragma unroll
    for (int u = 0; u < L::NW; u++) woff[u] = t.woff[u];
    ws = 0;
  };
  auto load_a = [&]() __attribute__((always_inline)) {
    const bool second = L::PS == 2 && (as & 1);
    char *to = lds + aslot * L::A_BYTES + pw * 1024 + (second ? L::NA * NP * 1024 : 0);
    const uint32_t at = (uint32_t)min(as, nstep - 1) / L::PS * 128u;
#pragma unroll
    for (int u = 0; u < L::NA; u++)  // the second half of an odd row's last line may lie behind the buffer: it reads 0
      dma(ra, to + u * NP * 1024, (second ? off[(L::PS - 1) * L::NA + u] : off[u]) + at, 0);
    if (L::PS == 1 || second) aslot = aslot + 1 == L::RA ? 0 : aslot + 1;
    as++;
  };
  auto load_w = [&]() __attribute__((always_inline)) {
    char *to = lds + L::W0 + wslot * L::W_BYTES + pw * 1024;
    const uint32_t at = (uint32_t)min(ws, nstep - 1) * mx4::kBlk;
#pragma unroll
    for (int u = 0; u < L::NW; u++) {
      // Non-temporal where an expert has one tile of rows and its weights are read once (509 tokens: gate/up 143 -> 131 us,
      // down 86 -> 81); where two tiles share them it costs (6000 tokens, E2M1: 320 -> 332 us, 231 -> 241).
      if constexpr (BM == 64) dma_once(rw, to + u * NP * 1024, woff[u], at);
      else dma(rw, to + u * NP * 1024, woff[u], at);
    }
    wslot = wslot + 1 == L::RD ? 0 : wslot + 1;
    ws++;
  };
  auto load_scales = [&](const Source<FA, BM> &t, const Source<FA, BM> &other, bool same, int c, int sslot)
                         __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < L::NS; u++) {
      const int b = L::scale_piece(pw, u);
      dma(same ? t.rs[u] : other.rs[u], lds + L::SCALES + sslot * L::SSLOT + b * 1024, same ? t.soff[u] : other.soff[u],
          same ? c * (b < L::SA ? 16 : mx4::kSblk) : 0);
    }
  };

  Source<FA, BM> cur, nxt;
  describe(cur, sh.list[sh.at]);
  i32x4_t d = sh.list[sh.at + sh.per < sh.end ? sh.at + sh.per : sh.at];
  if constexpr (MODE == 0) {
    fetch_rows(cur);
    asm volatile("s_waitcnt vmcnt(0)\ns_barrier" ::: "memory");
  }
  place(cur);
  load_scales(cur, cur, true, 0, 0);
  start_a(cur);
  start_w(cur);
  if constexpr (L::PS == 2) load_a();
  for (int i = 0; i < L::RD - 1; i++) {
    load_a();
    load_w();
  }
  int sslot = 0;
  for (;;) {
    const bool more = sh.at + sh.per < sh.end;
    if (more) sh.at += sh.per;  // after the last tile: its own first steps again, which nobody reads
    describe(nxt, d);
    d = sh.list[sh.at + sh.per < sh.end ? sh.at + sh.per : sh.at];
    // After a tile whose last scale piece is short its successor's first scales are younger than the count below says.
    if ((nstep & 3) != 0) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    for (int kt = 0; kt < nst; kt++) {
      // What is read in this step was issued RD - 1 steps ago or earlier (the scales of a whole piece, four); newer are
      // the pieces of RD - 2 steps.
      asm volatile("s_waitcnt vmcnt(%0)\ns_barrier" ::"n"(L::NL *(L::RD - 2)) : "memory");
      if (kt == 0) fetch_rows(MODE == 0 ? nxt : cur);
      if ((kt & 3) == 0) {
        const int c = kt >> 2;
        if (c == max(nch - 2, 0)) {  // the rows came before step 0's pieces: they are there from step 4 on
          if (MODE == 0 && kt == 0) asm volatile("s_waitcnt vmcnt(0)\ns_barrier" ::: "memory");
          place(nxt);
        }
        if (c < nch) {
          sslot ^= 1;
          load_scales(cur, nxt, c + 1 < nch, c + 1, sslot);
        }
      }
      if (kt == nst - (L::RD - 2 + L::PS)) start_a(nxt);
      if (kt == nst - (L::RD - 1)) start_w(nxt);
      load_a();  // into slots read in the step before, or earlier
      load_w();
    }
    if (!more) break;
    cur = nxt;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS outlives the workgroup
}

// ---------------------------------------------------------------- the multiplying waves
// A tile as one of them sees it.
struct Tile {
  int col0, rbase, mvalid, arow0, nb;
};

// One tile: the K loop and the epilogue.  MODE 0: gate/up + SwiGLU -> h.  MODE 1: down -> gated rows.  NB: 16-row
// blocks of this wave.
template <int MODE, int FA, bool BF16, int BM, int NB>
__device__ __forceinline__ void multiply(const Mx4Params &mp, const Tile &t, int K, int wave, int lane, int &aslot,
                                         int &wslot, int &sslot, char *lds) {
  using L = Lay<FA, BM>;
  const TileParams &p = mp.tp;
  const int n = lane & 15, q = lane >> 4, wn = wave & 3;
  const int nstep = K / 128, nch = (nstep + 3) / 4;
  const int nst = L::steps(nstep);
  f32x4_t acc[NB][4];
#pragma unroll
  for (int i = 0; i < NB; i++)
#pragma unroll
    for (int g = 0; g < 4; g++) acc[i][g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // LDS bytes of this lane's operands inside their slots; of a row's eight 16-byte chunks c is at c ^ (row / 2 % 8),
  // so that 16 rows at one chunk meet all banks
  const uint32_t wbase = L::W0 + (uint32_t)wn * 4096u + lane * 16u;
  const uint32_t abase = (uint32_t)(t.arow0 + n) * 128u + (uint32_t)(q ^ (n >> 1)) * 16u;
  uint32_t ws[4], as[NB];
  auto step = [&](auto JC, int kt) __attribute__((always_inline)) {
    constexpr int j = decltype(JC)::value;
    if (kt >= nst) return;
    asm volatile("s_waitcnt lgkmcnt(0)\ns_barrier" ::: "memory");  // this wave is done with the slot before
    if constexpr (j == 0) {
      if (MODE == 0 && kt == 0 && nch <= 2) asm volatile("s_barrier" ::: "memory");  // the loading waves' extra one
      if (kt < nstep) {
        const char *sp = lds + L::SCALES + sslot * L::SSLOT;
#pragma unroll
        for (int g = 0; g < 4; g++) ws[g] = *(const uint32_t *)(sp + BM * 16 + (wn * 4 + g) * 256 + lane * 4);
#pragma unroll
        for (int i = 0; i < NB; i++) as[i] = *(const uint32_t *)(sp + (t.arow0 + 16 * i + n) * 16 + q * 4);
        sslot ^= 1;
      }
    }
    const uint32_t wb = wbase + (uint32_t)wslot * L::W_BYTES;
    const uint32_t ab = abase + (uint32_t)aslot * L::A_BYTES, ab4 = ab ^ 64u;  // chunk q, chunk q + 4
    auto act = [&](int i) __attribute__((always_inline)) {
      if constexpr (FA == mx4::FP8)
        return mx4::piece8(*(const u32x4_t *)(lds + ab + i * 2048), *(const u32x4_t *)(lds + ab4 + i * 2048));
      else
        return mx4::piece4(*(const u32x4_t *)(lds + (j & 1 ? ab4 : ab) + i * 2048));
    };
    if (kt < nstep) {
      v8i_t w[4], a[2];
#pragma unroll
      for (int g = 0; g < 4; g++) w[g] = mx4::piece4(*(const u32x4_t *)(lds + wb + g * 1024));
      a[0] = act(0);
#pragma unroll
      for (int i = 0; i < NB; i++) {
        if (i + 1 < NB) a[(i + 1) & 1] = act(i + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int g = 0; g < 4; g++) acc[i][g] = mx4::mfma<FA, j, j>(w[g], a[i & 1], acc[i][g], ws[g], as[i]);
      }
    }
    if (L::PS == 1 || (j & 1)) aslot = aslot + 1 == L::RA ? 0 : aslot + 1;
    wslot = wslot + 1 == L::RD ? 0 : wslot + 1;
  };
  for (int kt = 0; kt < nst; kt += 4) {
    step(std::integral_constant<int, 0>{}, kt);
    step(std::integral_constant<int, 1>{}, kt + 1);
    step(std::integral_constant<int, 2>{}, kt + 2);
    step(std::integral_constant<int, 3>{}, kt + 3);
  }
  // acc[i][g][r]: row rbase + 16 i + n, weight row 16 g + 4 q + r of this wave's 64
#pragma unroll
  for (int i = 0; i < NB; i++) {
    const int m = 16 * i + n;
    const bool on = m < t.mvalid;
    const size_t row = (size_t)(t.rbase + m);
    if constexpr (MODE == 0) {
      float v[2][4];
#pragma unroll
      for (int g = 0; g < 2; g++)
#pragma unroll
        for (int r = 0; r < 4; r++) v[g][r] = silu_fast(acc[i][g][r]) * acc[i][2 + g][r];
      mx4::store_h_block<FA>(v, on, (uint8_t *)p.out + row * mx4::code_bytes<FA>(p.I),
                             mp.out_scales + row * mx4::h_scale_stride(p.I), t.col0, q);
    } else if (t.col0 < p.H) {  // H is a multiple of 128: a wave's 64 columns are all there or none
      const float gate = *(const float *)(lds + L::ROW0 + (t.arow0 + m) * 4);
#pragma unroll
      for (int g = 0; g < 4; g += 2)
        mx4::store_pair<BF16>(p.out, row * p.H + t.col0 + 16 * g, q, acc[i][g] * gate, acc[i][g + 1] * gate, on);
    }
  }
  // Ends the stores' branches here.  Without it they end where the NB cases meet, which makes the ring's state, uniform
  // as it is, look different between lanes there: it would live in vector registers.
  asm volatile("; end of tile, %0 blocks" ::"n"(NB));
}

template <int MODE, int FA, bool BF16, int BM>
__global__ __launch_bounds__(NTHR, 3) void ffn_mx4_kernel(Mx4Params mp) {  // three waves per SIMD
  using L = Lay<FA, BM>;
  __shared__ __attribute__((aligned(1024))) char lds[L::BYTES];
  Share sh(mp);
  if (sh.at >= sh.end) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave >= NC) {
    load_tiles<MODE, FA, BM>(mp, sh, wave - NC, lane, lds);
    return;
  }
  const int wm = wave >> 2, wn = wave & 3, K = MODE == 0 ? mp.tp.H : mp.tp.I;
  if constexpr (MODE == 0) asm volatile("s_barrier" ::: "memory");  // the loading waves' extra one
  i32x4_t d = sh.list[sh.at];
  int aslot = 0, wslot = 0, sslot = 0;
  for (;;) {
    const int rows = d.w & 0xffff, part = d.w >> 16;
    Tile t;
    t.col0 = MODE == 0 ? d.y * 128 + wn * 32 : d.y * BN + wn * 64;
    t.arow0 = wm * part;
    t.rbase = d.z + t.arow0;
    t.mvalid = min(rows - t.arow0, part);
    t.nb = min(part >> 4, (max(t.mvalid, 1) + 15) >> 4);
    sh.at += sh.per;
    if (sh.at < sh.end) d = sh.list[sh.at];
#define MX4_BODY(NB) multiply<MODE, FA, BF16, BM, NB>(mp, t, K, wave, lane, aslot, wslot, sslot, lds)
    // the waves of a tile may take different cases: each meets the same barriers
    if constexpr (BM == 64) {
      if (t.nb == 1) MX4_BODY(1);
      else MX4_BODY(2);
    } else {
      if (t.nb <= 2) MX4_BODY(2);
      else if (t.nb <= 4) MX4_BODY(4);
      else if (t.nb == 5) MX4_BODY(5);  // three tiles for 385 to 480 rows: 3% of 6000 tokens; a case of 3 gave nothing
      else MX4_BODY(6);
    }
#undef MX4_BODY
    if (sh.at >= sh.end) break;
  }
}

// The tile list: expert by expert, then N tile by N tile, then M tile by M tile.  Workgroup ``part`` of ``parts``
// writes its share; each counts the M tiles of all experts for itself (a hand-over costs more than El loads do).  One
// workgroup writing all of it, a wave an expert, took 27 us, this 5.  cap: M tiles at most, as the workspace has room
// for.  smem: El + 1 ints, the first M tile of each expert.
template <int BM>
__device__ void list_tiles(const TileParams &p, int NT, int cap, int part, int parts, int4 *out, int *count, int *smem) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto rows_of = [&](int e) { return min(p.offsets[e + 1], p.R_cap) - max(p.offsets[e], 0); };
  for (int e = threadIdx.x; e < p.El; e += blockDim.x) {
    const int c = rows_of(e);
    smem[e] = c > 0 ? (c + BM - 1) / BM : 0;
  }
  __syncthreads();
  if (wave == 0) {
    int n0 = 0;
    for (int b = 0; b < p.El; b += 64) {
      const int t = b + lane < p.El ? smem[b + lane] : 0;
      const int incl = ffn::wave_incl_scan_i(t, lane);
      if (b + lane < p.El) smem[b + lane] = min(n0 + incl - t, cap);  // cap: whatever the offsets say
      n0 = min(n0 + __shfl(incl, 63, 64), cap);
    }
    if (lane == 0) smem[p.El] = n0;
  }
  __syncthreads();
  const int n = smem[p.El] * NT;
  if (part == 0 && threadIdx.x == 0) *count = n;
  for (int i = part * blockDim.x + threadIdx.x; i < n; i += parts * blockDim.x) {
    int e = 0;  // the last expert whose tiles start at or before i (an expert without tiles starts where the next does)
    for (int hi = p.El; hi - e > 1;) {
      const int mid = (e + hi) >> 1;
      if (smem[mid] * NT <= i) e = mid;
      else hi = mid;
    }
    const int c = rows_of(e), m = smem[e + 1] - smem[e], j = i - smem[e] * NT, nt = j / m, mt = j - nt * m;
    const int trows = min(BM, ((c + m - 1) / m + 31) & ~31);  // m * trows >= c; a last tile may have no rows left
    const int rows = max(min(trows, c - mt * trows), 0);
    out[i] = make_int4(e, nt, max(p.offsets[e], 0) + mt * trows, rows | (trows / 2) << 16);
  }
}

// What the tile kernels need first.  The first 2 ``parts`` workgroups: the tile lists of both halves.  The others:
// activation scales [T, K/32] into lane order: dword q of piece c of a row has the scales 16c + 4j + q, j = 0 .. 3 (0
// past the end of the row).
template <int BM>
__global__ __launch_bounds__(256) void prepare_kernel(TileParams p, int parts, int cap, int4 *gtiles,
                                                      int4 *dtiles, int *counts, const uint8_t *__restrict__ s,
                                                      uint32_t *__restrict__ out) {
  if ((int)blockIdx.x < 2 * parts) {
    __shared__ int smem[1024 + 1];
    const int part = blockIdx.x >> 1;
    if (blockIdx.x & 1) list_tiles<BM>(p, (p.H + BN - 1) / BN, cap, part, parts, dtiles, counts + 1, smem);
    else list_tiles<BM>(p, p.I / 128, cap, part, parts, gtiles, counts, smem);
    return;
  }
  const int K = p.H, kb = K / 32, dw = (K + 511) / 512 * 4, b0 = blockIdx.x - 2 * parts;
  const long long total = (long long)p.T * dw, stride = (long long)(gridDim.x - 2 * parts) * blockDim.x;
  for (long long i = (long long)b0 * blockDim.x + threadIdx.x; i < total; i += stride) {
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

// y[t] = sum of t's rows in slot order; a slot without a row (or with one out of range) adds nothing.  The rows come in y's
// type and are added in fp32.  With bf16 y a term is thus rounded to bf16 once before the sum: fp32 rows would take 872 ->
// 1040 us for 6000 tokens with E4M3 activations, 673 -> 821 with E2M1, and bring the error of the rounded y from 1.4
// roundings of it to one; who needs that asks for fp32 y.  A thread sums
// eight columns, the loads of eight slots in flight (509 tokens 18 -> 8 us) and non-temporal (6000 tokens 83 -> 70 us, 0.44
// GB at 6.3 TB/s; the same for the stores of the down launch costs that 15 us).
constexpr int SUM_THR = 256, SUM_COLS = 8;
template <bool BF16>
__global__ __launch_bounds__(SUM_THR) void sum_rows_kernel(const void *__restrict__ rows,
                                                           const int32_t *__restrict__ token_row, int T, int k,
                                                           int R_cap, int H, void *__restrict__ y) {
  const int c = (blockIdx.y * SUM_THR + threadIdx.x) * SUM_COLS;
  if (c >= H) return;  // H is a multiple of 128
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    f32x4_t lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
    for (int j0 = 0; j0 < k; j0 += 8) {
      u32x4_t v[8][BF16 ? 1 : 2];
      int r[8];
#pragma unroll
      for (int j = 0; j < 8; j++) {
        r[j] = j0 + j < k ? token_row[(size_t)t * k + j0 + j] : -1;
        if ((unsigned)r[j] >= (unsigned)R_cap) r[j] = -1;
      }
#pragma unroll
      for (int j = 0; j < 8; j++) {
        if (r[j] < 0) continue;
        const size_t i = (size_t)r[j] * H + c;
        if constexpr (BF16) {
          v[j][0] = __builtin_nontemporal_load((const u32x4_t *)((const uint16_t *)rows + i));
        } else {
          v[j][0] = __builtin_nontemporal_load((const u32x4_t *)((const float *)rows + i));
          v[j][1] = __builtin_nontemporal_load((const u32x4_t *)((const float *)rows + i + 4));
        }
      }
#pragma unroll
      for (int j = 0; j < 8; j++) {
        if (r[j] < 0) continue;
        if constexpr (BF16) {
          lo += f32x4_t{bf16_lo(v[j][0].x), bf16_hi(v[j][0].x), bf16_lo(v[j][0].y), bf16_hi(v[j][0].y)};
          hi += f32x4_t{bf16_lo(v[j][0].z), bf16_hi(v[j][0].z), bf16_lo(v[j][0].w), bf16_hi(v[j][0].w)};
        } else {
          lo += __builtin_bit_cast(f32x4_t, v[j][0]);
          hi += __builtin_bit_cast(f32x4_t, v[j][1]);
        }
      }
    }
    mx4::store4<BF16>(y, (size_t)t * H + c, lo);
    mx4::store4<BF16>(y, (size_t)t * H + c + 4, hi);
  }
}

// Workspace: h codes [R_cap, I] (a byte each, half of it used by E2M1), h scales, and for the tile kernels the
// activation scales in lane order, the tile lists and the rows [R_cap, H].
size_t h_bytes(int R_cap, int I) { return align_up((size_t)R_cap * I, 256); }
size_t hs_bytes(int R_cap, int I) { return align_up((size_t)R_cap * mx4::h_scale_stride(I), 256); }
size_t as_bytes(int T, int H) { return align_up((size_t)T * mx4::h_scale_stride(H), 256); }
// M tiles at most: one per started BM rows of each expert.
int max_mtiles(int T, int R_cap, int El, int BM) {
  const long long a = ((long long)R_cap + (long long)El * (BM - 1)) / BM, b = (long long)El * ceil_div_i(T, BM);
  return (int)(a < b ? a : b);
}
// Rows of a tile: 64 while R_cap / El, the most rows that an expert can have on average, is at most 40, else 192.  128
// experts, H = 4096, I = 1536, top 8, all local (us with 64-row tiles, with 192-row tiles in brackets), E4M3: 16 rows each
// 218 (243), 32 rows 230 (252), 40 rows 235 (257), 48 rows 242 (260), 64 rows 352 (278), 128 rows 493 (359); E2M1: 216
// (228), 225 (240), 229 (245), 233 (249), 321 (259), 436 (314).  Between 48 and 64 rows it depends on how many experts
// pass 64.  With El of E experts local, an expert has El / E of that on average: a share of 32 experts of 128 with 12 to 40
// rows each gets 192-row tiles, E4M3 77 us instead of 69 at 12 rows, 79 instead of 75 at 31, E2M1 within 1%.
// 128-row tiles in place of 192 gain 2% at 64 rows and lose 22% at 128, 7% at 375.
int tile_rows(int R_cap, int El) { return ceil_div_i(R_cap, El) <= 40 ? 64 : 192; }
size_t list_bytes(int T, int R_cap, int El, int H, int I) {
  const int m = max_mtiles(T, R_cap, El, tile_rows(R_cap, El));
  return 256 + align_up((size_t)m * (I / 128 + ceil_div_i(H, BN)) * sizeof(int4), 256);
}

template <int FA, bool BF16, int BM>
hipError_t launch_tiles(const FfnMx4Args &a, hipStream_t s) {
  uint8_t *h = (uint8_t *)a.ws, *hs = h + h_bytes(a.R_cap, a.I), *as = hs + hs_bytes(a.R_cap, a.I);
  uint8_t *list = as + as_bytes(a.T, a.H), *rows = list + list_bytes(a.T, a.R_cap, a.El, a.H, a.I);
  const int mt = max_mtiles(a.T, a.R_cap, a.El, BM), ntg = a.I / 128, ntd = ceil_div_i(a.H, BN);
  int *counts = (int *)list;
  int4 *gtiles = (int4 *)(list + 256), *dtiles = gtiles + (size_t)mt * ntg;
  Mx4Params p{};
  p.tp.offsets = a.offsets;
  p.tp.row_token = a.row_token;
  p.tp.row_w = a.row_w;
  p.tp.El = a.El;
  p.tp.H = a.H;
  p.tp.I = a.I;
  p.tp.R_cap = a.R_cap;
  p.tp.T = a.T;
  const long long dwords = (long long)a.T * (mx4::h_scale_stride(a.H) / 4);
  const int most = mt * (ntg > ntd ? ntg : ntd);
  const int parts = most < 64 * 256 ? ceil_div_i(most, 256) : 64;
  hipLaunchKernelGGL(prepare_kernel<BM>, dim3(2 * parts + (unsigned)(dwords < (1 << 20) ? (dwords + 255) / 256 : 4096)),
                     dim3(256), 0, s, p.tp, parts, mt, gtiles, dtiles, counts, a.a_s, (uint32_t *)as);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  Mx4Params g = p;
  g.tp.a = a.a;
  g.a_scales = as;
  g.tp.w = a.wgu;
  g.w_scales = a.wgu_s;
  g.tp.out = h;
  g.out_scales = hs;
  g.tiles = gtiles;
  g.ntiles = counts;
  hipLaunchKernelGGL((ffn_mx4_kernel<0, FA, false, BM>), dim3(NCU), dim3(NTHR), 0, s, g);
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  Mx4Params d = p;
  d.tp.a = h;
  d.a_scales = hs;
  d.tp.w = a.wd;
  d.w_scales = a.wd_s;
  d.tp.out = rows;
  d.tiles = dtiles;
  d.ntiles = counts + 1;
  hipLaunchKernelGGL((ffn_mx4_kernel<1, FA, BF16, BM>), dim3(NCU), dim3(NTHR), 0, s, d);
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(sum_rows_kernel<BF16>, dim3(a.T < 16384 ? a.T : 16384, ceil_div_i(a.H, SUM_THR * SUM_COLS)),
                     dim3(SUM_THR), 0, s, rows, a.token_row, a.T, a.k, a.R_cap, a.H, a.y);
  return hipGetLastError();
}

template <int FA, bool BF16>
hipError_t launch(const FfnMx4Args &a, hipStream_t s) {
  return tile_rows(a.R_cap, a.El) == 64 ? launch_tiles<FA, BF16, 64>(a, s) : launch_tiles<FA, BF16, 192>(a, s);
}

}  // namespace

size_t ffn_mx4_ws_bytes(int T, int R_cap, int El, int H, int I, int y_bf16) {
  size_t b = h_bytes(R_cap, I) + hs_bytes(R_cap, I);
  if (T > kMx4StreamMaxT)
    b += as_bytes(T, H) + list_bytes(T, R_cap, El, H, I) + align_up((size_t)R_cap * H * (y_bf16 ? 2 : 4), 256);
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
