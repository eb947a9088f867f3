// Products of rows grouped by expert, for every size and type (moe_grouped_mm, moe_grouped_wgrad).
//
//   rows times matrix    out[r, n] = sum_k a[r, k] w[e][n, k]      (w rows contiguous along k, or along n with KN)
//   weight gradient      dw[e][m, n] = sum over e's rows of a[r, m] b[r, n]
//
// Both are one kernel: an operand's tile is "k-major" (its contiguous axis is the contraction) or "mn-major" (its
// contiguous axis is an output axis).  Tiles of BM x 128 outputs, 128 bytes of contraction a step (32 fp32, 64 bf16),
// staged through registers into two LDS buffers; fp32 on v_mfma_f32_32x32x2_f32, whose products are fp32 throughout,
// bf16 on v_mfma_f32_32x32x16_bf16.  A k-major tile keeps its rows in LDS (144 bytes apart, so that 16 rows at one
// 16-byte piece meet all banks); an mn-major tile keeps its k rows, and bf16 operands are turned by the transposing
// LDS read.  What lies outside an expert's rows, N, M or K is stored as zero, in both operands, so that nothing
// outside can reach a product.  32 experts of 1024 x 2048 in fp32, 12000 rows: 505 us, 100 TFLOP/s, matrix units busy in 0.65 of the
// cycles, the rest their start and the last, partly idle round; gradients of 8 x 777 x 515 from 602 rows 21 us, latency.
#include "grouped_tiles.h"

#include <algorithm>

namespace {

constexpr int BN = 128, KB = 128, PITCH = KB + 16;  // bytes of a step; bytes between rows of a k-major tile
constexpr int NTHR = 256;

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

// One operand's tile: R rows (output axis) of KB bytes.
template <typename T, bool MN, int R>
struct Operand {
  static constexpr int KE = KB / sizeof(T);                      // contraction elements a step
  static constexpr int V = 16 / sizeof(T);                       // elements of a piece
  static constexpr int RP = R * sizeof(T) + 32;                  // mn-major: bytes between k rows
  static constexpr int BYTES = MN ? KE * RP : R * PITCH;
  static constexpr int NP = R * KB / 16 / NTHR;                  // pieces a thread and step
  static_assert(NP >= 1, "whole pieces");
  const T *base;        // first element of the expert's matrix or of the rows' tensor
  const int32_t *index; // row of the tensor for a row of the product, or NULL
  size_t ld;            // elements between rows of the tensor
  int row0, rows;       // first row of the product and how many (k-major A: the tile's; mn-major: the contraction's)
  int limit;            // rows of the tensor (index clamp)
  int col0, cols;       // mn-major: first output column of the tile and columns of the matrix
  int K;                // k-major: length of the contraction
  u32x4_t reg[NP];
  const T *src[MN ? 1 : NP];  // k-major: the rows of this thread's pieces, NULL past the last

  __device__ __forceinline__ const T *row(int r) const {
    if (index) r = min(max(index[r], 0), limit - 1);
    return base + (size_t)r * ld;
  }
  // The piece at p, of which the row has ``have`` elements.  Rows that are no whole pieces are loaded as whole ones too, at any
  // alignment (global memory allows it), their last piece element by element.
  template <bool VEC>
  __device__ __forceinline__ u32x4_t piece(const T *p, int have) const {
    if constexpr (VEC) return *(const u32x4_t *)p;
    else {
      u32x4_t v;
      if (have >= V) __builtin_memcpy(&v, p, 16);
      else {
        T e[V];
#pragma unroll
        for (int i = 0; i < V; i++) e[i] = i < have ? p[i] : T(0);
        v = __builtin_bit_cast(u32x4_t, e);
      }
      return v;
    }
  }
  __device__ __forceinline__ void start(int tid) {
    if constexpr (!MN) {
#pragma unroll
      for (int u = 0; u < NP; u++) {
        const int r = (tid + u * NTHR) / (KB / 16);
        src[u] = r < rows ? row(row0 + r) : nullptr;
      }
    }
  }
  template <bool VEC>
  __device__ __forceinline__ void fetch(int k0, int tid) {
#pragma unroll
    for (int u = 0; u < NP; u++) {
      const int c = tid + u * NTHR;
      if constexpr (!MN) {
        const int k = k0 + c % (KB / 16) * V;
        const int have = src[u] ? K - k : 0;
        reg[u] = have > 0 ? piece<VEC>(src[u] + k, have) : u32x4_t{0u, 0u, 0u, 0u};
      } else {
        constexpr int PR = R / V;  // pieces of a k row
        const int r = k0 + c / PR, n = col0 + c % PR * V;
        const int have = r < rows ? cols - n : 0;
        reg[u] = have > 0 ? piece<VEC>(row(row0 + r) + n, have) : u32x4_t{0u, 0u, 0u, 0u};
      }
    }
  }
  __device__ __forceinline__ void keep(char *lds, int tid) const {
#pragma unroll
    for (int u = 0; u < NP; u++) {
      const int c = tid + u * NTHR;
      if constexpr (!MN) *(u32x4_t *)(lds + c / (KB / 16) * PITCH + c % (KB / 16) * 16) = reg[u];
      else *(u32x4_t *)(lds + c / (R / V) * RP + c % (R / V) * 16) = reg[u];
    }
  }
};

// Operand registers of a 32-row block at row r0 for the q-th part of a step.  bf16: 16 contraction elements, lane
// (n, g) holds 8g .. 8g+7 of row n.  fp32: 8 elements, four instructions' worth: instruction j takes element 4g + j.
template <typename T, bool MN, int R>
__device__ __forceinline__ u32x4_t fragment(const char *lds, int r0, int q, int lane) {
  using O = Operand<T, MN, R>;
  const int n = lane & 31, g = lane >> 5;
  if constexpr (!MN) {
    return *(const u32x4_t *)(lds + (r0 + n) * PITCH + (2 * q + g) * 16);
  } else if constexpr (sizeof(T) == 4) {
    u32x4_t v;
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = *(const uint32_t *)(lds + (8 * q + 4 * g + j) * O::RP + (r0 + n) * 4);
    return v;
  } else {
    // lane i of 16 gives the address of k row i / 4, columns 4 (i % 4) ..; it gets four k rows of column i
    const int i = lane & 15;
    const char *p = lds + (16 * q + 8 * g + (i >> 2)) * O::RP + (r0 + (n & 16) + (i & 3) * 4) * 2;
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * O::RP));
    const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
    return u32x4_t{a.x, a.y, b.x, b.y};
  }
}

template <typename T>
__device__ __forceinline__ f32x16_t multiply(u32x4_t a, u32x4_t b, f32x16_t c) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 4; j++)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[j]), __uint_as_float(b[j]), c, 0, 0, 0);
    return c;
  } else {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0,
                                                   0, 0);
  }
}

// C tile of BM x BN: steps over the contraction, two LDS buffers, one barrier a step.
template <typename T, bool AMN, bool BMN, int BM, bool VA, bool VB, int MB, int NB>
__device__ __forceinline__ void tile(Operand<T, AMN, BM> &A, Operand<T, BMN, BN> &B, int K, int m0, int n0,
                                     f32x16_t (&acc)[MB][NB], char *lds) {
  using OA = Operand<T, AMN, BM>;
  using OB = Operand<T, BMN, BN>;
  constexpr int KE = OA::KE, BUF = OA::BYTES + OB::BYTES;
  const int tid = threadIdx.x, lane = tid & 63;
#pragma unroll
  for (int i = 0; i < MB; i++)
#pragma unroll
    for (int j = 0; j < NB; j++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;
  A.start(tid);
  B.start(tid);
  A.template fetch<VA>(0, tid);
  B.template fetch<VB>(0, tid);
  char *cur = lds, *nxt = lds + BUF;
  for (int k = 0; k < K; k += KE) {
    A.keep(cur, tid);
    B.keep(cur + OA::BYTES, tid);
    __syncthreads();  // the step is there; the buffer written next was read before the barrier
    if (k + KE < K) {
      A.template fetch<VA>(k + KE, tid);
      B.template fetch<VB>(k + KE, tid);
    }
#pragma unroll
    for (int q = 0; q < 4; q++) {
      u32x4_t a[MB], b[NB];
#pragma unroll
      for (int i = 0; i < MB; i++) a[i] = fragment<T, AMN, BM>(cur, m0 + i * 32, q, lane);
#pragma unroll
      for (int j = 0; j < NB; j++) b[j] = fragment<T, BMN, BN>(cur + OA::BYTES, n0 + j * 32, q, lane);
#pragma unroll
      for (int i = 0; i < MB; i++)
#pragma unroll
        for (int j = 0; j < NB; j++) acc[i][j] = multiply<T>(a[i], b[j], acc[i][j]);
    }
    char *t = cur;
    cur = nxt;
    nxt = t;
  }
}

// acc[i][j][r] at lane l: tile row m0 + 32 i + 8 (r / 4) + 4 (l / 32) + r % 4, column n0 + 32 j + l % 32.
template <int MB, int NB, typename F>
__device__ __forceinline__ void each(const f32x16_t (&acc)[MB][NB], int m0, int n0, F f) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < MB; i++)
#pragma unroll
    for (int j = 0; j < NB; j++)
#pragma unroll
      for (int r = 0; r < 16; r++)
        f(m0 + 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3), n0 + 32 * j + (lane & 31), acc[i][j][r]);
}

template <int BM>
struct Waves {  // BM = 128: 2 x 2 waves of 64 x 64 outputs; 64: 2 x 2 of 32 x 64; 32: 1 x 4 of 32 x 32
  static constexpr int MB = BM == 128 ? 2 : 1, NB = BM >= 64 ? 2 : 1;
  static __device__ __forceinline__ int m0(int w) { return BM >= 64 ? (w >> 1) * (BM / 2) : 0; }
  static __device__ __forceinline__ int n0(int w) { return BM >= 64 ? (w & 1) * 64 : w * 32; }
};

// Rows of a tile: fp32 products are slow enough that small tiles cost nothing, and they fill the chip more evenly.
template <typename T>
constexpr int kRows = sizeof(T) == 4 ? 64 : 128;

template <int BM_>
struct Shape {
  static constexpr int BM = BM_, BN = ::BN;
};

template <typename T, typename TO, bool KN, int BM, bool VA, bool VB>
__global__ __launch_bounds__(NTHR) void mm_kernel(train::MmArgs p) {
  using OA = Operand<T, false, BM>;
  using OB = Operand<T, KN, BN>;
  using Wv = Waves<BM>;
  __shared__ __attribute__((aligned(16))) char lds[2 * (OA::BYTES + OB::BYTES)];
  const train::MmTiles<Shape<BM>, sizeof(T)> tiles(p, threadIdx.x & 63);
  const int b = train::block_of();
  if (b >= tiles.total) return;
  const int xcd = b & 7, q = tiles.total >> 3, rem = tiles.total & 7;  // runs of tiles to an XCD
  const train::MmTile t = tiles.at(xcd * q + min(xcd, rem) + (b >> 3), p);
  const int nt = t.nt, r0 = t.r0, rows = t.rows;
  OA A{};
  A.base = (const T *)p.a;
  A.index = p.a_index;
  A.ld = p.K;
  A.row0 = r0;
  A.rows = rows;
  A.limit = p.a_rows;
  A.K = p.K;
  OB B{};
  B.base = (const T *)t.w;
  if constexpr (KN) {
    B.ld = p.N;
    B.rows = p.K;
    B.col0 = nt * BN;
    B.cols = p.N;
  } else {
    B.ld = p.K;
    B.row0 = nt * BN;
    B.rows = p.N - nt * BN;
    B.K = p.K;
  }
  const int wave = threadIdx.x >> 6, m0 = Wv::m0(wave), n0 = Wv::n0(wave);
  f32x16_t acc[Wv::MB][Wv::NB];
  tile<T, false, KN, BM, VA, VB>(A, B, p.K, m0, n0, acc, lds);
  TO *out = (TO *)p.out + (size_t)r0 * p.N + nt * BN;
  const int cols = p.N - nt * BN;
  each(acc, m0, n0, [&](int m, int n, float v) {
    if (m < rows && n < cols) train::put(out + (size_t)m * p.N + n, v);
  });
}

template <typename T, typename TO, bool VA, bool VB>
__global__ __launch_bounds__(NTHR) void wgrad_kernel(train::WgradArgs p) {
  constexpr int BM = kRows<T>;
  using OA = Operand<T, true, BM>;
  using OB = Operand<T, true, BN>;
  using Wv = Waves<BM>;
  __shared__ __attribute__((aligned(16))) char lds[2 * (OA::BYTES + OB::BYTES)];
  const int MT = (p.M + BM - 1) / BM, NT = (p.N + BN - 1) / BN;
  // Workgroups go round-robin over the 8 XCDs: runs of tiles to an XCD, so that the lines that two tiles of an odd row share
  // meet in one L2 (8 x 777 x 515 fp32 from 602 rows 25.3 us in launch order, 20.9 so; bf16 1021 x 1023, 12000 rows 115 and 87).
  const int G = p.splits * p.El * MT * NT, wg = train::block_of(), each_xcd = G >> 3, more = G & 7, xcd = wg & 7;
  if (wg >= G) return;
  const int at = xcd * each_xcd + min(xcd, more) + (wg >> 3);
  const int s = at / (MT * NT * p.El), b = at % (MT * NT * p.El);
  const int e = b / (MT * NT), mt = b / NT % MT, nt = b % NT;
  int r0, rows;
  train::clip_rows(p.offsets[e], p.offsets[e + 1], p.R_cap, r0, rows);
  if (p.splits > 1) train::part_of(s, p.splits, r0, rows);
  // No rows: nothing to add, or zeros, 16 bytes a lane (6 tokens, 123 experts x 1301 x 1210 fp32: 169 us through the products, 143).
  if (rows == 0) {
    if (p.add) return;
    constexpr int V = 16 / sizeof(TO), LR = BN / V;  // lanes of a row
    const int ms = min(p.M - mt * BM, BM), n = nt * BN + threadIdx.x % LR * V;
    for (int m = threadIdx.x / LR; m < ms; m += NTHR / LR) {
      TO *const o = (TO *)p.dw + (((size_t)s * p.El + e) * p.M + mt * BM + m) * p.N + n;
      if (n + V <= p.N) {
        const u32x4_t zeros = {0u, 0u, 0u, 0u};
        __builtin_memcpy(o, &zeros, 16);
      } else {
        for (int i = 0; n + i < p.N; i++) o[i] = TO(0);
      }
    }
    return;
  }
  OA A{};
  A.base = (const T *)p.a;
  A.index = p.a_index;
  A.ld = p.M;
  A.row0 = r0;
  A.rows = rows;
  A.limit = p.a_rows;
  A.col0 = mt * BM;
  A.cols = p.M;
  OB B{};
  B.base = (const T *)p.b;
  B.index = p.b_index;
  B.ld = p.N;
  B.row0 = r0;
  B.rows = rows;
  B.limit = p.b_rows;
  B.col0 = nt * BN;
  B.cols = p.N;
  const int wave = threadIdx.x >> 6, m0 = Wv::m0(wave), n0 = Wv::n0(wave);
  f32x16_t acc[Wv::MB][Wv::NB];
  tile<T, true, true, BM, VA, VB>(A, B, rows, m0, n0, acc, lds);
  TO *out = (TO *)p.dw + (((size_t)s * p.El + e) * p.M + mt * BM) * p.N + nt * BN;
  const int ms = p.M - mt * BM, ns = p.N - nt * BN;
  const bool add = p.add;
  each(acc, m0, n0, [&](int m, int n, float v) {
    if (m < ms && n < ns) {
      TO *o = out + (size_t)m * p.N + n;
      train::put(o, add ? train::to_f32(*o) + v : v);
    }
  });
}

// Sums of the parts, in their order.
template <typename TO>
__global__ __launch_bounds__(256) void join_kernel(const float *ws, int splits, long long n, int add, TO *dw) {
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
    float v = 0.0f;
#pragma unroll 4
    for (int s = 0; s < splits; s++) v += ws[s * n + i];
    train::put(dw + i, add ? train::to_f32(dw[i]) + v : v);
  }
}

template <typename T, typename TO, bool KN, int BM>
hipError_t launch_mm(const train::MmArgs &a, hipStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const bool va = a.K % V == 0, vb = (KN ? a.N : a.K) % V == 0;
  // worst-case tiles: sum of ceil(c / BM) <= (R + El (BM - 1)) / BM
  const long long mt = std::min(((long long)a.R_cap + (long long)a.El * (BM - 1)) / BM, (long long)a.R_cap);
  const dim3 grid = train::grid_of(mt * ceil_div_i(a.N, BN), NTHR);
  if (va && vb) hipLaunchKernelGGL((mm_kernel<T, TO, KN, BM, true, true>), grid, dim3(NTHR), 0, s, a);
  else if (va) hipLaunchKernelGGL((mm_kernel<T, TO, KN, BM, true, false>), grid, dim3(NTHR), 0, s, a);
  else if (vb) hipLaunchKernelGGL((mm_kernel<T, TO, KN, BM, false, true>), grid, dim3(NTHR), 0, s, a);
  else hipLaunchKernelGGL((mm_kernel<T, TO, KN, BM, false, false>), grid, dim3(NTHR), 0, s, a);
  return hipGetLastError();
}

template <typename T, typename TO>
hipError_t pick_mm(const train::MmArgs &a, hipStream_t s) {
  const bool few = (long long)a.R_cap <= 32LL * a.El;
  if (a.kn) return few ? launch_mm<T, TO, true, 32>(a, s) : launch_mm<T, TO, true, kRows<T>>(a, s);
  return few ? launch_mm<T, TO, false, 32>(a, s) : launch_mm<T, TO, false, kRows<T>>(a, s);
}

template <typename T, typename TO>
hipError_t launch_wgrad(const train::WgradArgs &a, hipStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const dim3 grid = train::grid_of((long long)a.splits * a.El * ceil_div_i(a.M, kRows<T>) * ceil_div_i(a.N, BN), NTHR);
  const bool va = a.M % V == 0, vb = a.N % V == 0;
  if (va && vb) hipLaunchKernelGGL((wgrad_kernel<T, TO, true, true>), grid, dim3(NTHR), 0, s, a);
  else if (va) hipLaunchKernelGGL((wgrad_kernel<T, TO, true, false>), grid, dim3(NTHR), 0, s, a);
  else if (vb) hipLaunchKernelGGL((wgrad_kernel<T, TO, false, true>), grid, dim3(NTHR), 0, s, a);
  else hipLaunchKernelGGL((wgrad_kernel<T, TO, false, false>), grid, dim3(NTHR), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t train::launch_grouped_mm(const MmArgs &a, hipStream_t s) {
  if (mm_dma_fits(a)) {
    // Tiles for few rows an expert on average.  128 experts of 1536 x 4096, top 8, us with those and with the large tiles: 64
    // tokens 230 and 255, 256 243 and 259, 384 248 and 273, 512 296 and 274; transposed 8 tokens 114 and 127, 24 200 and 207, 64
    // 244 and 233, 512 342 and 259.  fp32, 32 experts of 1024 x 2048, top 4: 200 tokens 73 and 92, 300 84 and 89.
    bool few = a.R_cap <= (a.bf16 ? (a.kn ? 2LL : 24LL) : 40LL) * a.El;
    // And where the large tiles would leave most of the chip idle: 4 experts x 3000 rows, 64 x 2048, 13 and 44 us; the tiles of
    // this file where those for few rows would be very many (8 x 375 rows, 1024 x 1024: 18 us, 24 with those, 25 large).
    const int bm = a.bf16 ? 256 : kRows<float>, bn = a.bf16 ? 256 : BN;
    const long long large = (long long)a.El * ceil_div_i(ceil_div_i(a.R_cap, a.El), bm) * ceil_div_i(a.N, bn);
    const long long small = (a.R_cap / 32 + (long long)a.El) * ceil_div_i(a.N, 64);
    if (large <= 96) few = few || small <= 768;
    if (few || (a.bf16 && large > 96)) return launch_mm_dma(a, few, s);
  }
  if (!a.bf16) return pick_mm<float, float>(a, s);
  return a.out_bf16 ? pick_mm<uint16_t, uint16_t>(a, s) : pick_mm<uint16_t, float>(a, s);
}

// Parts of an expert's rows, each with sums of its own: where the tiles are fewer than half the compute units and an expert has
// 512 rows or more on average, as many as fill the chip, of 256 rows or more (4 experts of 256 x 256, 3000 rows each: 65 us in
// one part, 22 in eleven).
static int wgrad_splits(int El, int R_cap, int M, int N) {
  const long long tiles = (long long)El * ceil_div_i(M, 128) * ceil_div_i(N, 128), avg = R_cap / El;
  if (tiles > 128 || avg < 512) return 1;
  return (int)std::min({256 / tiles, avg / 256, 32LL});
}

size_t train::wgrad_ws_bytes(int El, int R_cap, int M, int N, int bf16) {
  const int splits = wgrad_splits(El, R_cap, M, N);
  return splits > 1 ? align_up((size_t)splits * El * M * N * sizeof(float), 256) : 0;
}

static hipError_t wgrad_parts(const train::WgradArgs &a, hipStream_t s) {
  if (train::wgrad_dma_fits(a)) return train::launch_wgrad_dma(a, s);
  if (!a.bf16) return launch_wgrad<float, float>(a, s);
  return a.out_bf16 ? launch_wgrad<uint16_t, uint16_t>(a, s) : launch_wgrad<uint16_t, float>(a, s);
}

hipError_t train::launch_grouped_wgrad(const WgradArgs &args, hipStream_t s) {
  WgradArgs a = args;
  a.splits = wgrad_splits(a.El, a.R_cap, a.M, a.N);
  if (a.splits == 1) return wgrad_parts(a, s);
  a.dw = a.ws;
  a.out_bf16 = a.add = 0;
  const hipError_t err = wgrad_parts(a, s);
  if (err != hipSuccess) return err;
  const long long n = (long long)a.El * a.M * a.N;
  const dim3 grid((unsigned)std::min((n + 255) / 256, 4096LL));
  if (args.out_bf16) hipLaunchKernelGGL((join_kernel<uint16_t>), grid, dim3(256), 0, s, (const float *)a.ws, a.splits, n, args.add, (uint16_t *)args.dw);
  else hipLaunchKernelGGL((join_kernel<float>), grid, dim3(256), 0, s, (const float *)a.ws, a.splits, n, args.add, (float *)args.dw);
  return hipGetLastError();
}
