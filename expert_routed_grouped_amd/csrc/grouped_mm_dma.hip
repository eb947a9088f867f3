// Products of rows grouped by expert on operands whose rows are whole 16-byte pieces: tiles that go from memory
// straight to LDS (moe_grouped_mm, moe_grouped_wgrad).
//
// One kernel for three products, by how an operand lies in memory.  A "k-major" operand has its contraction along its
// rows (activations; weights of a projection): its tile keeps rows of 64 values in LDS, 16-byte chunk c of row r in slot
// c ^ (r / 2 % 8), and a fragment of v_mfma_f32_32x32x16_bf16 is one 16-byte LDS read.  An "mn-major" operand has an output
// axis along its rows (weights for an input gradient; both operands of a weight gradient): its tile keeps whole k rows,
// and a fragment is two transposing 8-byte LDS reads, each four k rows of 16 columns.  The 32-byte pieces of a k row
// are turned (below), so that the four rows of two neighbouring pieces, which half a wave reads at once, meet all 64 banks.
//
// Large tiles are 256 x 256 outputs, eight waves of 128 x 64: rows times matrix take 64 values of the contraction a step, weight
// gradients 32.  6000 tokens x 8 of 128 experts, 1536 x 4096, take 639 to 662 us (0.91 to 0.945 PFLOP/s), weight gradients of the same
// size 716 to 765 (0.79 to 0.84; 1.6 GB of results).  Power holds the clock near 1.9 GHz, as in a dense library product; the matrix units are
// busy in 0.55 and 0.41 of the cycles (0.70 there), as all waves load, wait, multiply and store in step.  Few rows an expert take tiles
// of their own (mm_few_kernel; also fp32).
#include "grouped_tiles.h"

#include <algorithm>
#include <type_traits>

namespace {

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
typedef __attribute__((address_space(3))) void lds_void;
using train::MmTile;
using train::MmTiles;
constexpr uint32_t kRsrcWord3 = 0x00020000;  // raw buffer, 32-bit data format
constexpr uint32_t kNowhere = 0x80000000u;   // byte offset behind every buffer: such a load gives zeros

__device__ __forceinline__ void barrier_no_fence() { asm volatile("s_barrier" ::: "memory"); }

// Sixteen bytes a lane from memory to 1 KB of LDS at byte ``to``.  In assembly, because the compiler waits for every load to
// LDS that it knows of before a transposing LDS read (vmcnt(0) twice a step); nothing comes back in registers, and the waits
// for LDS are the kernel's own.  The five wait states are those between a scalar register that a vector instruction wrote (a
// spilled one, say) and a load that reads it, which the compiler does not see in here; M0 needs one.
typedef uint32_t rsrc_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void dma(rsrc_t r, uint32_t to, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(to), "v"(voff), "s"(r), "s"(soff)
               : "m0");
}
// The same for lines that are read once.
__device__ __forceinline__ void dma_once(rsrc_t r, uint32_t to, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds" ::"s"(to), "v"(voff), "s"(r),
               "s"(soff)
               : "m0");
}
// The same for four bytes a lane.
__device__ __forceinline__ void dma_words(rsrc_t r, uint32_t to, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(to), "v"(voff), "s"(r) : "m0");
}
// A buffer of ``bytes`` bytes.
__device__ __forceinline__ rsrc_t resource(const void *p, size_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  rsrc_t r;
  r.x = __builtin_amdgcn_readfirstlane((uint32_t)a);
  r.y = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32) & 0xffffu);
  r.z = __builtin_amdgcn_readfirstlane((uint32_t)bytes);
  r.w = kRsrcWord3;
  return r;
}
__device__ __forceinline__ uint32_t lds_at(const char *p) { return (uint32_t)(uintptr_t)(lds_void *)p; }

// Rows (output axis) and waves of a tile, slots of the two operands.
template <int BM_, int BN_, int BK_, int WM_, int WN_, int SA_, int SB_>
struct Cfg {
  static constexpr int BM = BM_, BN = BN_, BK = BK_, WM = WM_, WN = WN_, SA = SA_, SB = SB_;
  static constexpr int NW = WM * WN, NTHR = 64 * NW;
  static constexpr int MB = BM / WM / 32, NB = BN / WN / 32;       // 32-row blocks of a wave
  static constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2;
  static constexpr int NA = A_BYTES / 1024 / NW, NBL = B_BYTES / 1024 / NW;  // loads of a wave and step
  static constexpr int LDS = SA * A_BYTES + SB * B_BYTES;
  static_assert(NA >= 1 && NBL >= 1 && LDS <= 160 * 1024, "whole loads, one compute unit's LDS");
};

// Where an mn-major tile of R columns keeps the 32-byte piece p of k row k: at p ^ turn<R>(k).  Half a wave reads two
// neighbouring pieces of k rows 4c .. 4c + 3 (bit 3 of k is the same in it): with R >= 128 a row starts at bank 0, with
// R = 64 every other one does.
template <int R>
__device__ __forceinline__ constexpr int turn(int k) {
  return R >= 128 ? 2 * (k & 3) + ((k >> 3) & 1) : k & 2;
}

// What a wave loads of an operand: byte offsets of its N segments of 1 KB at step 0, and their advance.
template <int N, int NW>
struct Source {
  static constexpr int LOADS = N;  // loads of a step
  rsrc_t r;
  uint32_t off[N];
  uint32_t step;    // bytes from one step to the next
  uint32_t last;    // or-ed into a lane's offset in the last step: kNowhere where that is past the contraction's end
  __device__ __forceinline__ void start(int) {}
  // The first COUNT segments of step kt.
  template <int COUNT = N>
  __device__ __forceinline__ void load(uint32_t to, int wave, int, int kt, bool is_last, bool once = false) {
    const uint32_t so = (uint32_t)kt * step, m = is_last ? last : 0u;
    if (once) {
#pragma unroll
      for (int u = 0; u < COUNT; u++) dma_once(r, to + (wave + NW * u) * 1024, off[u] | m, so);
    } else {
#pragma unroll
      for (int u = 0; u < COUNT; u++) dma(r, to + (wave + NW * u) * 1024, off[u] | m, so);
    }
  }
  // k-major tile of 128 bytes a row and step: segment s holds rows 8s .. 8s + 7.  ``row`` gives the byte offset of segment u's
  // tile row.  ESZ: bytes of an element.
  template <int ESZ = 2, typename F>
  __device__ __forceinline__ void k_major(int wave, int lane, int K, F row) {
    static_assert(NW % 2 == 0, "a lane's chunk is the same in all of its segments");
    int chunk = 0;
#pragma unroll
    for (int u = 0; u < N; u++) {
      const int t = (wave + NW * u) * 8 + (lane >> 3);
      chunk = (lane & 7) ^ ((t >> 1) & 7);
      off[u] = row(u, t) + (uint32_t)chunk * 16u;
    }
    step = 128;
    const int tail = K & (128 / ESZ - 1);
    last = tail != 0 && chunk * (16 / ESZ) >= tail ? kNowhere : 0u;
  }
  // fp32 k rows of R columns, as they lie in memory (they are read word by word).
  template <int R, int BK>
  __device__ __forceinline__ void mn_words(int wave, int lane, uint32_t ld, uint32_t col) {
#pragma unroll
    for (int u = 0; u < N; u++)
      off[u] = (uint32_t)((wave + NW * u) * (256 / R) + lane / (R / 4)) * ld + col + (uint32_t)(lane % (R / 4)) * 16u;
    step = BK * ld;
    last = 0;
  }
  // mn-major tile of R columns from byte ``col`` of rows that lie ``ld`` bytes apart, BK k rows a step.
  template <int R, int BK>
  __device__ __forceinline__ void mn_major(int wave, int lane, uint32_t ld, uint32_t col) {
#pragma unroll
    for (int u = 0; u < N; u++) off[u] = (uint32_t)k_row<R>(wave + NW * u, lane) * ld + col + in_row<R>(wave + NW * u, lane);
    step = BK * ld;
    last = 0;
  }
  // A segment of an mn-major tile holds 512 / R k rows; a lane's k row, and its byte of it.
  template <int R>
  static __device__ __forceinline__ int k_row(int seg, int lane) {
    return seg * (512 / R) + lane / (R / 8);
  }
  template <int R>
  static __device__ __forceinline__ uint32_t in_row(int seg, int lane) {
    const int k = k_row<R>(seg, lane), slot = lane % (R / 8);
    return (uint32_t)((slot >> 1) ^ turn<R>(k)) * 32u + (uint32_t)(slot & 1) * 16u;
  }
};

// The same for an mn-major operand whose k rows are gathered, 32 a step.  The indexes of a step's rows go to LDS too, two
// steps before its rows do: a register load would have to be waited for with everything that is younger.
template <int N, int NW>
struct Gathered {
  using S = Source<N, NW>;
  static constexpr int LOADS = N + 1;
  rsrc_t r, ri;
  int rows, limit;
  uint32_t ld, at[N], words;  // words: LDS of this wave's indexes, two steps of 256 bytes
  int k[N];
  template <int R>
  __device__ __forceinline__ void mn_major(int wave, int lane, uint32_t ld_, uint32_t col) {
    ld = ld_;
#pragma unroll
    for (int u = 0; u < N; u++) k[u] = S::template k_row<R>(wave + NW * u, lane), at[u] = col + S::template in_row<R>(wave + NW * u, lane);
  }
  __device__ __forceinline__ void ahead(int lane, int kt) {
    dma_words(ri, words + (kt & 1) * 256, (uint32_t)min(kt * 32 + (lane & 31), rows - 1) * 4u);
  }
  __device__ __forceinline__ void start(int lane) {
    ahead(lane, 0);
    ahead(lane, 1);
  }
  __device__ __forceinline__ void load(uint32_t to, int wave, int lane, int kt, bool) {
    const __attribute__((address_space(3))) int *const w = (const __attribute__((address_space(3))) int *)(uintptr_t)(words + (kt & 1) * 256);
    uint32_t row[N];
#pragma unroll
    for (int u = 0; u < N; u++) row[u] = kt * 32 + k[u] < rows ? (uint32_t)min(max(w[k[u]], 0), limit - 1) * ld : kNowhere;
#pragma unroll
    for (int u = 0; u < N; u++) dma(r, to + (wave + NW * u) * 1024, row[u] + at[u], 0);
    ahead(lane, kt + 2);  // into the words that were just used
  }
};

// LDS bytes of a lane's fragments of blocks of 32 rows from row r0 on: of block b in slice kk of 16 values.
template <bool MN, int R, int B>
struct Frag {
  uint32_t base[MN ? B : 4];
  __device__ __forceinline__ Frag(int r0, int lane) {
    if constexpr (MN) {
      const int i = lane & 15, h = (lane >> 4) & 1, g = lane >> 5;
#pragma unroll
      for (int b = 0; b < B; b++)
        base[b] = (uint32_t)(8 * g + (i >> 2)) * (R * 2) + (uint32_t)((r0 / 16 + 2 * b + h) ^ turn<R>(8 * g + (i >> 2))) * 32u +
                  (uint32_t)(i & 3) * 8u;
    } else {
      const int n = lane & 31, g = lane >> 5;
#pragma unroll
      for (int kk = 0; kk < 4; kk++) base[kk] = (uint32_t)(r0 + n) * 128u + (uint32_t)((2 * kk + g) ^ ((n >> 1) & 7)) * 16u;
    }
  }
  // The same with kk known at run time only (base[kk] is base[0] ^ 32 kk).
  __device__ __forceinline__ bf16x8_t at(const char *slot, int kk, int b) const {
    if constexpr (MN) return get(slot + kk * 16 * (R * 2), 0, b);
    else return *(const bf16x8_t *)(slot + (base[0] ^ (uint32_t)(kk * 32)) + b * 4096);
  }
  __device__ __forceinline__ bf16x8_t get(const char *slot, int kk, int b) const {
    if constexpr (MN) {
      const char *p = slot + base[b] + kk * 16 * (R * 2);
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * (R * 2)));
      const uint2 x = __builtin_bit_cast(uint2, lo), y = __builtin_bit_cast(uint2, hi);
      return __builtin_bit_cast(bf16x8_t, u32x4_t{x.x, x.y, y.x, y.y});
    } else {
      return *(const bf16x8_t *)(slot + base[kk] + b * 4096);
    }
  }
};

// A wave's outputs, 32 rows of 128 bytes of LDS at a time, so that a store writes whole lines of a row: acc[i][j][r] at lane l
// is tile row m0 + 32 i + l % 32, column n0 + 32 j + 8 (r / 4) + 4 (l / 32) + r % 4.  Two-byte stores straight from the
// accumulators cost 440 of 1144 us of a weight gradient.  ADD: to what is there, in fp32.  ONCE: results that nobody reads
// soon, past the caches.  FULL: the tile lies inside the matrix; the stores are then as many as STORES says.  ``cols`` is a
// multiple of 8.
constexpr int kOutPitch = 144, kOutBytes = 32 * kOutPitch;
template <int MB, int NB, bool ADD, bool ONCE, bool FULL, typename TO, int MA>
__device__ __forceinline__ void store(const f32x16_t (&acc)[MA][NB], char *lds, TO *out, size_t ld, int m0, int n0, int rows,
                                      int cols, int lane) {
  using TS = std::conditional_t<ADD, float, TO>;  // a sum that is added to is not rounded before
  constexpr int JB = 4 / sizeof(TS), V = 16 / sizeof(TO), LR = JB * 32 / V;  // column blocks of a pass; lanes of a row
  static_assert(NB % JB == 0, "whole passes");
  char *const w = lds + (lane & 31) * kOutPitch + 4 * (lane >> 5) * (int)sizeof(TS);
  const char *const rd = lds + lane / LR * kOutPitch + lane % LR * V * (int)sizeof(TS);
  const uint32_t at_lane = ((uint32_t)(lane / LR) * (uint32_t)ld + (uint32_t)(lane % LR * V)) * (uint32_t)sizeof(TO);
#pragma unroll
  for (int i = 0; i < MB; i++)
#pragma unroll
    for (int j0 = 0; j0 < NB; j0 += JB) {
      constexpr int U = 32 * LR / 64;
      const int n = n0 + 32 * j0 + lane % LR * V;
      // a wave's own address and a lane's offset from it
      auto place = [&](int u) __attribute__((always_inline)) {
        return (TO *)((char *)(out + (size_t)(m0 + 32 * i + u * (64 / LR)) * ld + n0 + 32 * j0) + at_lane);
      };
      auto inside = [&](int u) __attribute__((always_inline)) {
        return FULL || (m0 + 32 * i + u * (64 / LR) + lane / LR < rows && n < cols);
      };
      // What is added to: all of a pass on its way at once, past the caches as the sums are (6000 tokens' fp32 gradients of 4096 x
      // 1536: one after the other 1753 us, 1495 at once, 1331 past the caches).
      u32x4_t old[ADD ? U : 1];
      if constexpr (ADD) {
#pragma unroll
        for (int u = 0; u < U; u++) old[u] = inside(u) ? __builtin_nontemporal_load((const u32x4_t *)place(u)) : u32x4_t{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int j = 0; j < JB; j++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const f32x16_t &c = acc[i][j0 + j];
          const float v[4] = {c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
          train::store_n<4>((TS *)(w + (32 * j + 8 * q) * (int)sizeof(TS)), v);
        }
      asm volatile("" ::: "memory");  // other lanes' values are read: the order of a wave's LDS accesses is the program's
#pragma unroll
      for (int u = 0; u < U; u++) {
        const char *const at = rd + u * (64 / LR) * kOutPitch;
        if (inside(u)) {
          if constexpr (ADD) {
            float x[V], y[V];
            train::load_n<V>((const float *)at, x);
            train::load_n<V>((const TO *)&old[u], y);
#pragma unroll
            for (int k = 0; k < V; k++) x[k] += y[k];
            u32x4_t v;
#pragma unroll
            for (int k = 0; k < 4; k++)
              v[k] = sizeof(TO) == 4 ? __float_as_uint(x[k]) : pack_bf16x2(x[2 * k % V], x[(2 * k + 1) % V]);
            __builtin_nontemporal_store(v, (u32x4_t *)place(u));
          } else {
            const u32x4_t v = *(const u32x4_t *)at;
            if constexpr (ONCE) __builtin_nontemporal_store(v, (u32x4_t *)place(u));
            else *(u32x4_t *)place(u) = v;
          }
        }
      }
      asm volatile("" ::: "memory");
    }
}
template <int MB, int NB, typename TO>
constexpr int STORES = MB * NB * 32 * 32 * sizeof(TO) / 1024;

constexpr int kWorkers = 256;  // one workgroup per compute unit, 32 to an XCD

// Rows times matrix.  The second operand, whose first touch comes from memory, is loaded two steps ahead through three
// slots, the rows one step ahead through two (160 KB of LDS).
using Mm = Cfg<256, 256, 64, 2, 4, 2, 3>;

template <bool KN, bool GATHER, typename TO>
__global__ __launch_bounds__(Mm::NTHR, 1) __attribute__((amdgpu_waves_per_eu(2, 2))) void mm_dma_kernel(train::MmArgs p) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the stub alone
  using C = Mm;
  __shared__ __attribute__((aligned(1024))) char lds[C::LDS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WN, n0 = wave % C::WN * (C::NB * 32), K = p.K, KT = (K + C::BK - 1) / C::BK;
  const MmTiles<C> tiles(p, lane);
  // Workgroups go round-robin over the 8 XCDs: XCD x takes the x-th eighth of the tiles, its workgroups in turn, so that
  // the tiles of an expert, which share operands, meet in one L2.
  const int xcd = blockIdx.x & 7, q = tiles.total >> 3, rem = tiles.total & 7;
  const int end = xcd * q + min(xcd, rem) + q + (xcd < rem ? 1 : 0);
  int L = xcd * q + min(xcd, rem) + (blockIdx.x >> 3);
  if (L >= end) return;
  char *const la = lds, *const lb = lds + C::SA * C::A_BYTES;
  const uint32_t ta = lds_at(la), tb = lds_at(lb);
  // Outputs go through the slots that the next tile's first loads leave free: the third of B, the second of A.
  constexpr int IN_B = C::B_BYTES / kOutBytes;
  static_assert(IN_B + C::A_BYTES / kOutBytes >= C::NW, "every wave's outputs fit");
  char *const stage = wave < IN_B ? lb + 2 * C::B_BYTES + wave * kOutBytes : la + C::A_BYTES + (wave - IN_B) * kOutBytes;

  Source<C::NA, C::NW> sa;
  Source<C::NBL, C::NW> sb;
  const uint32_t lda = (uint32_t)K * 2u;
  int src[C::NA];  // gathered: the tensor's rows of this lane's segments
  auto rows_of = [&](const MmTile &t) __attribute__((always_inline)) {
    if constexpr (GATHER) {
#pragma unroll
      for (int u = 0; u < C::NA; u++)  // rows past the end repeat the last one; nothing of them is stored
        src[u] = p.a_index[t.r0 + min((wave + C::NW * u) * 8 + (lane >> 3), t.rows - 1)];
    }
  };
  auto place = [&](const MmTile &t) __attribute__((always_inline)) {
    if constexpr (GATHER) sa.r = resource(p.a, (size_t)p.a_rows * lda);
    else sa.r = resource((const char *)p.a + (size_t)t.r0 * lda, (size_t)t.rows * lda);
    sa.k_major(wave, lane, K, [&](int u, int r) {
      if constexpr (GATHER) return (uint32_t)min(max(src[u], 0), p.a_rows - 1) * lda;
      else return (uint32_t)min(r, t.rows - 1) * lda;
    });
    sb.r = resource(t.w, (size_t)p.N * K * 2);
    if constexpr (KN) sb.template mn_major<C::BN, C::BK>(wave, lane, (uint32_t)p.N * 2u, t.nt * C::BN * 2u);
    else sb.k_major(wave, lane, K, [&](int, int r) { return (uint32_t)min(t.nt * C::BN + r, p.N - 1) * lda; });
  };
  // The loads that run ahead of a tile.  A matrix that one tile reads goes past the caches (512 tokens, 32 rows an expert: 308 us
  // without, 288; transposed 289 and 259), one that two tiles share does not (6000 tokens: 656 us, 701 with).
  auto first = [&](int trows, bool once) __attribute__((always_inline)) {
    if (trows > 192) sa.template load<4>(ta, wave, lane, 0, KT == 1);
    else if (trows > 128) sa.template load<3>(ta, wave, lane, 0, KT == 1);
    else if (trows > 64) sa.template load<2>(ta, wave, lane, 0, KT == 1);
    else sa.template load<1>(ta, wave, lane, 0, KT == 1);
    sb.load(tb, wave, lane, 0, KT == 1, once);
    if (KT > 1) sb.load(tb + C::B_BYTES, wave, lane, 1, KT == 2, once);
  };
  const Frag<KN, C::BN, C::NB> fb(n0, lane);
  f32x16_t acc[C::MB][C::NB];
  bool stored = false;  // exactly the stores of a whole tile are younger than the loads of this tile's first step

  // One tile of MB blocks of 32 rows for either half of the waves; the outputs are the caller's to store.
  auto contract = [&](auto MC, int m0, bool once) __attribute__((always_inline)) {
    constexpr int MB = decltype(MC)::value;
    const Frag<false, C::BM, MB> fa(m0, lane);
#pragma unroll
    for (int i = 0; i < MB; i++)
#pragma unroll
      for (int j = 0; j < C::NB; j++)
#pragma unroll
        for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;
    auto step = [&](auto PC, int kt) __attribute__((always_inline)) {
      constexpr int P = decltype(PC)::value, A0 = P % 2, B0 = P % 3, A1 = (P + 1) % 2, B2 = (P + 2) % 3;
      if (kt >= KT) return;
      // This wave's loads of the step have landed (within a step those of A are issued before those of B, one step younger),
      // and it has read its last fragments of the step before.
      if (kt + 1 >= KT) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      else if (P == 0 && kt == 0 && stored)
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(C::NBL + STORES<MB, C::NB, TO>) : "memory");
      else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(C::NBL) : "memory");
      barrier_no_fence();
      const char *a = la + A0 * C::A_BYTES, *b = lb + B0 * C::B_BYTES;
      bf16x8_t af[2][MB], bf[2][C::NB];
      auto frags = [&](int kk) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < C::NB; j++) bf[kk & 1][j] = fb.get(b, kk, j);
#pragma unroll
        for (int i = 0; i < MB; i++) af[kk & 1][i] = fa.get(a, kk, i);
      };
      frags(0);
#pragma unroll
      for (int kk = 0; kk < 4; kk++) {
        if (kk < 3) frags(kk + 1);
        if (kk == 0 && kt + 1 < KT) sa.template load<MB>(ta + A1 * C::A_BYTES, wave, lane, kt + 1, kt + 2 == KT);
        if (kk == 2 && kt + 2 < KT) sb.load(tb + B2 * C::B_BYTES, wave, lane, kt + 2, kt + 3 == KT, once);
#pragma unroll
        for (int i = 0; i < MB; i++)
#pragma unroll
          for (int j = 0; j < C::NB; j++)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[kk & 1][j], af[kk & 1][i], acc[i][j], 0, 0, 0);
      }
    };
    for (int kt = 0; kt < KT; kt += 6) {
      step(std::integral_constant<int, 0>{}, kt);
      step(std::integral_constant<int, 1>{}, kt + 1);
      step(std::integral_constant<int, 2>{}, kt + 2);
      step(std::integral_constant<int, 3>{}, kt + 3);
      step(std::integral_constant<int, 4>{}, kt + 4);
      step(std::integral_constant<int, 5>{}, kt + 5);
    }
  };

  MmTile t = tiles.at(L, p);
  rows_of(t);
  place(t);
  first(t.trows, t.once);
  for (;;) {
    const bool more = L + kWorkers / 8 < end;
    const MmTile tn = tiles.at(more ? L + kWorkers / 8 : L, p);
    rows_of(tn);
    const int m0 = wm * (t.trows >> 1), cols = p.N - t.nt * C::BN;
    TO *const out = (TO *)p.out + (size_t)t.r0 * p.N + t.nt * C::BN;
    const bool full = t.rows == t.trows && cols >= C::BN;
    auto body = [&](auto MC) __attribute__((always_inline)) {
      constexpr int MB = decltype(MC)::value;
      contract(MC, m0, t.once);
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // every wave has read its last fragments
      if (more) {
        place(tn);
        first(tn.trows, tn.once);
      }
      if (full) store<MB, C::NB, false, false, true>(acc, stage, out, p.N, m0, n0, t.rows, cols, lane);
      else store<MB, C::NB, false, false, false>(acc, stage, out, p.N, m0, n0, t.rows, cols, lane);
    };
    switch (t.trows >> 6) {
      case 1: body(std::integral_constant<int, 1>{}); break;
      case 2: body(std::integral_constant<int, 2>{}); break;
      case 3: body(std::integral_constant<int, 3>{}); break;
      default: body(std::integral_constant<int, 4>{}); break;
    }
    if (!more) break;
    stored = full && tn.trows == t.trows;
    L += kWorkers / 8;
    t = tn;
  }
#endif
}

// Few rows an expert: the matrices are read once, so what counts is how much of them is under way.  Tiles of up to 32 rows
// x 64 columns, 128 bytes of the contraction a step, six steps in LDS (72 KB, two workgroups on a compute unit); each of four
// waves multiplies a quarter of every step, and the quarters are joined at the end.  64 tokens x 8 of 128 experts, 1536 x 4096:
// 230 us, 6.9 TB/s.  fp32 operands go through the same tiles, 32 values a step, on v_mfma_f32_32x32x2_f32.
template <typename T>
struct Few {
  static constexpr int BM = 32, BN = 64, BK = 128 / sizeof(T), NW = 4, NTHR = 256, S = 6;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, LDS = S * (A_BYTES + B_BYTES);
  static constexpr int NA = A_BYTES / 1024 / NW, NBL = B_BYTES / 1024 / NW;
  static constexpr int PITCH = BN * 4 + 16;  // bytes between the rows of a quarter's sums
  static_assert(NW * BM * PITCH <= LDS, "the quarters fit");
};

template <typename T, bool KN, bool GATHER, typename TO>
__global__ __launch_bounds__(Few<T>::NTHR, 2) void mm_few_kernel(train::MmArgs p) {
#ifdef __HIP_DEVICE_COMPILE__
  using C = Few<T>;
  constexpr int ESZ = sizeof(T);
  constexpr bool F32 = ESZ == 4;
  __shared__ __attribute__((aligned(1024))) char lds[C::LDS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const MmTiles<C, ESZ> tiles(p, lane);
  const int wg = train::block_of();
  if (wg >= tiles.total) return;
  const int xcd = wg & 7, q = tiles.total >> 3, rem = tiles.total & 7;  // runs of tiles to an XCD
  const MmTile t = tiles.at(xcd * q + min(xcd, rem) + (wg >> 3), p);
  const int K = p.K, KT = (K + C::BK - 1) / C::BK, rows = t.rows;
  const uint32_t lda = (uint32_t)K * ESZ, ldn = (uint32_t)p.N * ESZ, col = (uint32_t)t.nt * C::BN * ESZ;
  Source<C::NA, C::NW> sa;
  Source<C::NBL, C::NW> sb;
  if constexpr (GATHER) sa.r = resource(p.a, (size_t)p.a_rows * lda);
  else sa.r = resource((const char *)p.a + (size_t)t.r0 * lda, (size_t)rows * lda);
  sa.template k_major<ESZ>(wave, lane, K, [&](int, int r) {
    const int at = min(r, rows - 1);  // rows past the end repeat the last one; nothing of them is stored
    return (uint32_t)(GATHER ? min(max(p.a_index[t.r0 + at], 0), p.a_rows - 1) : at) * lda;
  });
  sb.r = resource(t.w, (size_t)p.N * K * ESZ);
  if constexpr (KN && F32) sb.template mn_words<C::BN, C::BK>(wave, lane, ldn, col);
  else if constexpr (KN) sb.template mn_major<C::BN, C::BK>(wave, lane, ldn, col);
  else sb.template k_major<ESZ>(wave, lane, K, [&](int, int r) { return (uint32_t)min(t.nt * C::BN + r, p.N - 1) * lda; });
  const uint32_t to = lds_at(lds);
  // Step kt into its slot.  Steps past the end load nothing (every lane's offset is nowhere), so that the count below holds.
  int slot = 0;
  auto load = [&](int kt) __attribute__((always_inline)) {
    const uint32_t m = kt < KT ? (kt == KT - 1 ? sa.last : 0u) : kNowhere, at = to + slot * (C::A_BYTES + C::B_BYTES);
    const uint32_t mb = kt < KT ? (kt == KT - 1 ? sb.last : 0u) : kNowhere;
    const int k = min(kt, KT - 1);
#pragma unroll
    for (int u = 0; u < C::NA; u++) dma(sa.r, at + (wave + C::NW * u) * 1024, sa.off[u] | m, (uint32_t)k * sa.step);
    if (t.once) {
#pragma unroll
      for (int u = 0; u < C::NBL; u++) dma_once(sb.r, at + C::A_BYTES + (wave + C::NW * u) * 1024, sb.off[u] | mb, (uint32_t)k * sb.step);
    } else {
#pragma unroll
      for (int u = 0; u < C::NBL; u++) dma(sb.r, at + C::A_BYTES + (wave + C::NW * u) * 1024, sb.off[u] | mb, (uint32_t)k * sb.step);
    }
    slot = slot + 1 == C::S ? 0 : slot + 1;
  };
  for (int kt = 0; kt < C::S - 1; kt++) load(kt);
  const Frag<false, C::BM, 1> fa(0, lane);  // 16 bytes of a k-major row: eight bf16 or four fp32
  const Frag<KN && !F32, C::BN, 2> fb(0, lane);
  f32x16_t acc[2];
#pragma unroll
  for (int j = 0; j < 2; j++)
#pragma unroll
    for (int r = 0; r < 16; r++) acc[j][r] = 0.0f;
  int rd = 0;
  for (int kt = 0; kt < KT; kt++) {
    // the step's loads have landed; the slot that is filled next was read a step ago
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((C::NA + C::NBL) * (C::S - 2)) : "memory");
    const char *a = lds + rd * (C::A_BYTES + C::B_BYTES), *b = a + C::A_BYTES;
    if constexpr (F32) {  // this wave's eight values: instruction e takes 4g + e of lane group g
      const u32x4_t av = __builtin_bit_cast(u32x4_t, fa.at(a, wave, 0));
      u32x4_t bv[2];
#pragma unroll
      for (int j = 0; j < 2; j++) {
        if constexpr (KN) {
#pragma unroll
          for (int e = 0; e < 4; e++)
            bv[j][e] = *(const uint32_t *)(b + (8 * wave + 4 * (lane >> 5) + e) * (C::BN * 4) + (32 * j + (lane & 31)) * 4);
        } else bv[j] = __builtin_bit_cast(u32x4_t, fb.at(b, wave, j));
      }
      load(kt + C::S - 1);
#pragma unroll
      for (int e = 0; e < 4; e++)
#pragma unroll
        for (int j = 0; j < 2; j++)
          acc[j] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(bv[j][e]), __uint_as_float(av[e]), acc[j], 0, 0, 0);
    } else {
      const bf16x8_t af = fa.at(a, wave, 0), b0 = fb.at(b, wave, 0), b1 = fb.at(b, wave, 1);
      load(kt + C::S - 1);
      acc[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b0, af, acc[0], 0, 0, 0);
      acc[1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b1, af, acc[1], 0, 0, 0);
    }
    rd = rd + 1 == C::S ? 0 : rd + 1;
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  // acc[j][r] at lane l: row l % 32, column 32 j + 8 (r / 4) + 4 (l / 32) + r % 4
  char *const mine = lds + (wave * C::BM + (lane & 31)) * C::PITCH + 16 * (lane >> 5);
#pragma unroll
  for (int j = 0; j < 2; j++)
#pragma unroll
    for (int i = 0; i < 4; i++)
      *(float4 *)(mine + (32 * j + 8 * i) * 4) = make_float4(acc[j][4 * i], acc[j][4 * i + 1], acc[j][4 * i + 2], acc[j][4 * i + 3]);
  __syncthreads();
  const int cols = p.N - t.nt * C::BN, n = threadIdx.x % 16 * 4;
  if (n >= cols) return;
  TO *const out = (TO *)p.out + (size_t)t.r0 * p.N + t.nt * C::BN + n;
  for (int m = threadIdx.x / 16; m < rows; m += C::NTHR / 16) {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < C::NW; w++) {
      const float4 v = *(const float4 *)(lds + (w * C::BM + m) * C::PITCH + n * 4);
      s[0] += v.x, s[1] += v.y, s[2] += v.z, s[3] += v.w;
    }
    train::store_n<4>(out + (size_t)m * p.N, s);
  }
#endif
}

template <bool KN, bool GATHER, typename TO>
hipError_t launch(const train::MmArgs &a, hipStream_t s) {
  hipLaunchKernelGGL((mm_dma_kernel<KN, GATHER, TO>), dim3(kWorkers), dim3(Mm::NTHR), 0, s, a);
  return hipGetLastError();
}
template <typename T, bool KN, bool GATHER, typename TO>
hipError_t launch_few(const train::MmArgs &a, hipStream_t s) {
  using C = Few<T>;
  const long long mt = std::min(((long long)a.R_cap + (long long)a.El * (C::BM - 1)) / C::BM, (long long)a.R_cap);
  hipLaunchKernelGGL((mm_few_kernel<T, KN, GATHER, TO>), train::grid_of(mt * ceil_div_i(a.N, C::BN), C::NTHR), dim3(C::NTHR), 0, s, a);
  return hipGetLastError();
}
template <bool KN, bool GATHER>
hipError_t by_out(const train::MmArgs &a, bool few, hipStream_t s) {
  if (!a.bf16) return launch_few<float, KN, GATHER, float>(a, s);
  if (few) return a.out_bf16 ? launch_few<uint16_t, KN, GATHER, uint16_t>(a, s) : launch_few<uint16_t, KN, GATHER, float>(a, s);
  return a.out_bf16 ? launch<KN, GATHER, uint16_t>(a, s) : launch<KN, GATHER, float>(a, s);
}
template <bool KN>
hipError_t by_index(const train::MmArgs &a, bool few, hipStream_t s) {
  return a.a_index ? by_out<KN, true>(a, few, s) : by_out<KN, false>(a, few, s);
}

// Two workgroups of four waves on a compute unit, so that one multiplies while the other stores, took 809 us of the weight
// gradient's 748 (6000 tokens, 4096 x 1536): they load half as much again.  Without its stores it takes 556 us, 1.09 PFLOP/s.
using Wg = Cfg<256, 256, 32, 2, 4, 3, 3>;

// Weight gradients: the contraction is short (an expert's rows, 375 of 6000 tokens), so a workgroup works through a list
// of tiles and loads the next one's first two steps before it stores a tile.
template <bool GA, bool GB, bool ADD, typename TO>
__global__ __launch_bounds__(Wg::NTHR, 1) __attribute__((amdgpu_waves_per_eu(2, 2))) void wgrad_dma_kernel(train::WgradArgs p) {
#ifdef __HIP_DEVICE_COMPILE__
  using C = Wg;
  using SrcA = std::conditional_t<GA, Gathered<C::NA, C::NW>, Source<C::NA, C::NW>>;
  using SrcB = std::conditional_t<GB, Gathered<C::NBL, C::NW>, Source<C::NBL, C::NW>>;
  __shared__ __attribute__((aligned(1024))) char lds[C::LDS + C::NW * kOutBytes + (GA + GB) * C::NW * 512];
  const int MT = (p.M + C::BM - 1) / C::BM, NT = (p.N + C::BN - 1) / C::BN, per = MT * NT, total = p.El * per * p.splits;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m0 = wave / C::WN * (C::MB * 32), n0 = wave % C::WN * (C::NB * 32);
  // Workgroups go round-robin over the 8 XCDs: 32 neighbouring tiles, which share operands, run on one XCD at a time.
  int t = (blockIdx.x & 7) * (kWorkers / 8) + (blockIdx.x >> 3);
  if (t >= total) return;
  const auto *const off = (const __attribute__((address_space(4))) int *)(uintptr_t)p.offsets;  // scalar loads
  struct Tile {
    int e, mt, nt, s, r0, rows, KT;
  };
  auto tile = [&](int at) __attribute__((always_inline)) {
    Tile d;
    d.s = at / (p.El * per);
    at -= d.s * p.El * per;
    d.e = at / per;
    d.mt = (at - d.e * per) / NT;
    d.nt = at - d.e * per - d.mt * NT;
    train::clip_rows(off[d.e], off[d.e + 1], p.R_cap, d.r0, d.rows);
    if (p.splits > 1) train::part_of(d.s, p.splits, d.r0, d.rows);
    d.KT = (d.rows + C::BK - 1) / C::BK;
    return d;
  };
  SrcA sa;
  SrcB sb;
  char *const la = lds, *const lb = lds + C::SA * C::A_BYTES, *const stage = lds + C::LDS + wave * kOutBytes;
  const uint32_t ta = lds_at(la), tb = lds_at(lb);
  auto place = [&](const Tile &d) __attribute__((always_inline)) {
    const uint32_t lda = (uint32_t)p.M * 2u, ldb = (uint32_t)p.N * 2u, words = lds_at(lds) + C::LDS + C::NW * kOutBytes;
    if constexpr (GA) {
      sa.r = resource(p.a, (size_t)p.a_rows * lda);
      sa.ri = resource(p.a_index + d.r0, (size_t)d.rows * 4);
      sa.words = words + wave * 512;
      sa.rows = d.rows;
      sa.limit = p.a_rows;
      sa.template mn_major<C::BM>(wave, lane, lda, d.mt * C::BM * 2u);
    } else {
      sa.r = resource((const char *)p.a + (size_t)d.r0 * lda, (size_t)d.rows * lda);
      sa.template mn_major<C::BM, C::BK>(wave, lane, lda, d.mt * C::BM * 2u);
    }
    if constexpr (GB) {
      sb.r = resource(p.b, (size_t)p.b_rows * ldb);
      sb.ri = resource(p.b_index + d.r0, (size_t)d.rows * 4);
      sb.words = words + (GA * C::NW + wave) * 512;
      sb.rows = d.rows;
      sb.limit = p.b_rows;
      sb.template mn_major<C::BN>(wave, lane, ldb, d.nt * C::BN * 2u);
    } else {
      sb.r = resource((const char *)p.b + (size_t)d.r0 * ldb, (size_t)d.rows * ldb);
      sb.template mn_major<C::BN, C::BK>(wave, lane, ldb, d.nt * C::BN * 2u);
    }
  };
  auto first = [&](int KT) __attribute__((always_inline)) {  // the loads of a tile's first two steps
    if (KT == 0) return;
    sa.start(lane);
    sb.start(lane);
    if constexpr (GA || GB) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    sa.load(ta, wave, lane, 0, KT == 1);
    sb.load(tb, wave, lane, 0, KT == 1);
    if (KT > 1) {
      sa.load(ta + C::A_BYTES, wave, lane, 1, KT == 2);
      sb.load(tb + C::B_BYTES, wave, lane, 1, KT == 2);
    }
  };
  const Frag<true, C::BM, C::MB> fa(m0, lane);
  const Frag<true, C::BN, C::NB> fb(n0, lane);
  f32x16_t acc[C::MB][C::NB];
  constexpr int YOUNG = SrcA::LOADS + SrcB::LOADS, LATER = STORES<C::MB, C::NB, TO>;
  static_assert(C::SA == 3 && C::SB == 3 && YOUNG + LATER < 64, "two steps ahead; counts that a wait can name");

  Tile d = tile(t);
  place(d);
  first(d.KT);
  bool stored = false;  // exactly LATER stores are younger than the loads of this tile's first two steps
  for (;;) {
    const int tn = t + kWorkers;
    const bool more = tn < total;
    const Tile dn = tile(more ? tn : t);
    const int KT = d.KT;
#pragma unroll
    for (int i = 0; i < C::MB; i++)
#pragma unroll
      for (int j = 0; j < C::NB; j++)
#pragma unroll
        for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;
    auto step = [&](auto PC, int kt) __attribute__((always_inline)) {
      constexpr int P = decltype(PC)::value, P2 = (P + 2) % 3;
      if (kt >= KT) return;
      // this wave's loads of the step have landed, and it has read its last fragments of the step before
      if (kt + 1 >= KT) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      else if (P < 2 && kt < 2 && stored) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(YOUNG + LATER) : "memory");
      else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(YOUNG) : "memory");
      barrier_no_fence();
      const char *a = la + P * C::A_BYTES, *b = lb + P * C::B_BYTES;
      bf16x8_t af[2][C::MB], bf[2][C::NB];
      auto frags = [&](int kk) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < C::NB; j++) bf[kk & 1][j] = fb.get(b, kk, j);
#pragma unroll
        for (int i = 0; i < C::MB; i++) af[kk & 1][i] = fa.get(a, kk, i);
      };
      frags(0);
#pragma unroll
      for (int kk = 0; kk < C::BK / 16; kk++) {
        if (kk + 1 < C::BK / 16) frags(kk + 1);
        if (kk == 0 && kt + 2 < KT) sa.load(ta + P2 * C::A_BYTES, wave, lane, kt + 2, kt + 3 == KT);
        if (kk == 1 && kt + 2 < KT) sb.load(tb + P2 * C::B_BYTES, wave, lane, kt + 2, kt + 3 == KT);
#pragma unroll
        for (int i = 0; i < C::MB; i++)
#pragma unroll
          for (int j = 0; j < C::NB; j++)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[kk & 1][j], af[kk & 1][i], acc[i][j], 0, 0, 0);
      }
    };
    for (int kt = 0; kt < KT; kt += 3) {
      step(std::integral_constant<int, 0>{}, kt);
      step(std::integral_constant<int, 1>{}, kt + 1);
      step(std::integral_constant<int, 2>{}, kt + 2);
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // every wave has read its last fragments
    if (more) {
      place(dn);
      first(dn.KT);
    }
    TO *out = (TO *)p.dw + (((size_t)d.s * p.El + d.e) * p.M + d.mt * C::BM) * p.N + d.nt * C::BN;
    const int ms = p.M - d.mt * C::BM, ns = p.N - d.nt * C::BN;
    const bool full = ms >= C::BM && ns >= C::BN;
    if (ADD && KT == 0) {
    } else if (full) store<C::MB, C::NB, ADD, true, true>(acc, stage, out, p.N, m0, n0, ms, ns, lane);
    else store<C::MB, C::NB, ADD, true, false>(acc, stage, out, p.N, m0, n0, ms, ns, lane);
    if (!more) break;
    stored = !ADD && full;
    t = tn;
    d = dn;
  }
#endif
}

}  // namespace

// Rows of whole 16-byte pieces, every 32-bit byte offset below kNowhere.
bool train::mm_dma_fits(const MmArgs &a) {
  const long long lim = 1LL << 31, esz = a.bf16 ? 2 : 4, v = 16 / esz;
  return a.K % v == 0 && a.N % v == 0 && (long long)a.N * a.K * esz < lim &&
         (a.a_index ? (long long)a.a_rows * a.K * esz < lim : 256LL * a.K * esz < lim);
}
template <bool GA, bool GB, bool ADD>
static hipError_t wgrad_by_out(const train::WgradArgs &a, hipStream_t s) {
  const dim3 grid(kWorkers), block(Wg::NTHR);
  if (a.out_bf16) hipLaunchKernelGGL((wgrad_dma_kernel<GA, GB, ADD, uint16_t>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((wgrad_dma_kernel<GA, GB, ADD, float>), grid, block, 0, s, a);
  return hipGetLastError();
}
template <bool GA, bool GB>
static hipError_t wgrad_by_add(const train::WgradArgs &a, hipStream_t s) {
  return a.add ? wgrad_by_out<GA, GB, true>(a, s) : wgrad_by_out<GA, GB, false>(a, s);
}
bool train::wgrad_dma_fits(const WgradArgs &a) {
  const long long lim = 1LL << 31;
  return a.bf16 && a.M % 8 == 0 && a.N % 8 == 0 && a.M >= 128 && a.N >= 64 &&
         (long long)(a.a_index ? a.a_rows : a.R_cap) * a.M * 2 < lim && (long long)(a.b_index ? a.b_rows : a.R_cap) * a.N * 2 < lim;
}
hipError_t train::launch_wgrad_dma(const WgradArgs &a, hipStream_t s) {
  if (a.a_index) return a.b_index ? wgrad_by_add<true, true>(a, s) : wgrad_by_add<true, false>(a, s);
  return a.b_index ? wgrad_by_add<false, true>(a, s) : wgrad_by_add<false, false>(a, s);
}

hipError_t train::launch_mm_dma(const MmArgs &a, bool few, hipStream_t s) {
  return a.kn ? by_index<true>(a, few, s) : by_index<false>(a, few, s);
}
