// The whole MoE layer of a few tokens with MXFP4 experts in two launches (moe_decode_layer_mx4).
//
// Launch 1 routes, groups and computes the intermediate h; launch 2 is the down half of mx4_stream.h, which also
// sums to token order.  In launch 1 the resident workgroups draw tickets.  The first T * ceil(E / 64) tickets are
// routing items (token t, 64 experts): the row of x is widened into LDS (the item of the first experts also
// quantises it to MXFP8 for the experts' products) and one wave computes 64 logits, one lane each, with the
// library's fp32 chain over ascending h.  The last item to finish takes the top k of every token, groups the
// assignments by expert, lists the experts' tiles and raises a flag.  A workgroup whose ticket is past the routing
// items waits for the flag (its wait is for workgroups that drew earlier tickets, so they run; it is bounded
// all the same) and then takes its share of the gate/up tiles.
//
// What bounds it: at one token the chain, H dependent additions whose order is the routing contract (about 3 ns
// each), then the weights' bytes.  Against instruction issue the chain has the packed fp32 router (no unpacking), its
// x operand broadcast inside rows of 16 lanes by the FMA itself (DPP), so 16 steps cost 16 FMAs, four loads and
// one LDS read; and the matrix is touched by the idle waves beforehand, so that the loads find it in L2.
#include "mx4_stream.h"
#include "permute_dev.h"
#include "route_dev.h"

#include <mutex>

namespace {

constexpr int NTHR = mx4s::NTHR, NW = mx4s::NW;
constexpr uint32_t kSpinLimit = 1u << 22;  // polls of the routed flag before giving up (seconds)

// control words
enum : int { kTicket = 0, kDone = 1, kRouted = 2, kExit = 3, kError = 4, kTiles = 5, kCtlBytes = 256 };

struct Params {
  const uint16_t *x;   // [T, H] bf16
  const float *wr;     // [H/4, E, 4] fp32
  const float *bias;   // [E] or NULL
  int T, H, E, k, lo, El, I, nbits, R_cap, n_route;
  int32_t *ids;
  float *gates;
  uint32_t *ctl;
  float *logits;       // [T, 64 EC]
  uint8_t *xq, *xs;    // x as MXFP8
  int32_t *counts, *offsets, *row_token, *token_row;
  float *row_w;
  int2 *tiles;         // {first row, expert | rows << 16}
  const uint8_t *wgu, *wgu_s;
  uint8_t *h, *hs;
};

__device__ __forceinline__ uint32_t ld_agent(const uint32_t *p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// acc += x[h] w[h] for 16 steps in order: lane l holds x[h0 + l % 16], w[i] the weights of steps 4i .. 4i+3.  The FMA
// takes its x from lane i of each row of 16 (DPP); the leading wait is what DPP needs after a VALU write of x.
__device__ __forceinline__ float chain16(float acc, float xv, const f32x4_t (&w)[4]) {
#define CHAIN(i, n) "v_fmac_f32_dpp %0, %1, %" #n " row_newbcast:" #i " row_mask:0xf bank_mask:0xf\n"
  asm("s_nop 1\n" CHAIN(0, 2) CHAIN(1, 3) CHAIN(2, 4) CHAIN(3, 5) CHAIN(4, 6) CHAIN(5, 7) CHAIN(6, 8) CHAIN(7, 9)
          CHAIN(8, 10) CHAIN(9, 11) CHAIN(10, 12) CHAIN(11, 13) CHAIN(12, 14) CHAIN(13, 15) CHAIN(14, 16) CHAIN(15, 17)
      : "+v"(acc)
      : "v"(xv), "v"(w[0][0]), "v"(w[0][1]), "v"(w[0][2]), "v"(w[0][3]), "v"(w[1][0]), "v"(w[1][1]), "v"(w[1][2]),
        "v"(w[1][3]), "v"(w[2][0]), "v"(w[2][1]), "v"(w[2][2]), "v"(w[2][3]), "v"(w[3][0]), "v"(w[3][1]), "v"(w[3][2]),
        "v"(w[3][3]));
#undef CHAIN
  return acc;
}

// Routing item: 64 logits of token t (experts 64c ..); with c == 0 also x[t] as MXFP8.
__device__ __forceinline__ void route_item(const Params &p, int t, int c, int EP, float *xf) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int H = p.H;
  uint32_t touch = 0;
  if (wave > 0) {  // the chain's 1 KB lines, one access per 128 bytes
    const char *base = (const char *)p.wr + (size_t)c * 1024;
    const int width = min(p.E - 64 * c, 64) * 16;  // bytes of a 4-wide h group in this item's slice
    const int per = (width + 127) / 128, n = H / 4 * per;
    for (int i = threadIdx.x - 64; i < n; i += NTHR - 64)
      touch |= *(const volatile uint32_t *)(base + (size_t)(i / per) * p.E * 16 + min((i % per) * 128, width - 4));
  }
  for (int v = threadIdx.x; v < H / 8; v += NTHR) {
    const u32x4_t r = *((const u32x4_t *)(p.x + (size_t)t * H) + v);
    const float f[8] = {bf16_lo(r.x), bf16_hi(r.x), bf16_lo(r.y), bf16_hi(r.y),
                        bf16_lo(r.z), bf16_hi(r.z), bf16_lo(r.w), bf16_hi(r.w)};
    *(f32x4_t *)(xf + 8 * v) = f32x4_t{f[0], f[1], f[2], f[3]};
    *(f32x4_t *)(xf + 8 * v + 4) = f32x4_t{f[4], f[5], f[6], f[7]};
    if (c == 0) {  // H is a multiple of 128: the four lanes of a block loop together
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; j++) m = max(m, mx4::abs_bits(f[j]));
      m = max(m, (uint32_t)__shfl_xor((int)m, 1, 64));
      m = max(m, (uint32_t)__shfl_xor((int)m, 2, 64));
      const uint32_t s = mx4::scale_of_bits<8>(m);
      float u[8];
#pragma unroll
      for (int j = 0; j < 8; j++) u[j] = ldexpf(f[j], 127 - (int)s);
      const uint32_t lo = mx4::e4m3_quad(u[0], u[1], u[2], u[3]), hi = mx4::e4m3_quad(u[4], u[5], u[6], u[7]);
      *(uint2 *)(p.xq + (size_t)t * H + 8 * v) = s == 255 ? make_uint2(0, 0) : make_uint2(lo, hi);
      if ((v & 3) == 0) p.xs[(size_t)t * (H / 32) + (v >> 2)] = (uint8_t)s;
    }
  }
  __syncthreads();
  if (wave == 0) {
    const int e = 64 * c + lane;
    // buffer loads: the lane's offset fixed, the advance along h a scalar
    const __amdgpu_buffer_rsrc_t rw =
        __builtin_amdgcn_make_buffer_rsrc((void *)p.wr, (short)0, p.E * H * 4, 0x00020000);
    const int voff = min(e, p.E - 1) * 16, step = p.E * 16;
    constexpr int NS = 8;  // ring of 16-h stages; H is a multiple of 128
    f32x4_t w[NS][4];
    float xv[NS];
    const int n = H / 16;
    auto load = [&](f32x4_t(&d)[4], float &x, int s) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 4; i++)
        d[i] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, voff, (4 * s + i) * step, 0));
      x = xf[16 * s + (lane & 15)];
    };
#pragma unroll
    for (int s = 0; s < NS - 1; s++) {
      load(w[s], xv[s], s);
      asm volatile("" ::: "memory");  // keeps the loads in order, so that a wait covers one stage
    }
    float acc = 0.0f;
    for (int s = 0; s < n; s += NS) {
#pragma unroll
      for (int j = 0; j < NS; j++) {
        load(w[(j + NS - 1) % NS], xv[(j + NS - 1) % NS], min(s + j + NS - 1, n - 1));
        asm volatile("" ::: "memory");
        acc = chain16(acc, xv[j], w[j]);
      }
    }
    if (e < p.E) p.logits[(size_t)t * EP + e] = p.bias ? acc + p.bias[e] : acc;
  }
  asm volatile("" ::"v"(touch));  // keeps the warm-up loads
}

// After every logit: top k and gates, the grouping, the tile list, the flag.
template <int EC>
__device__ __forceinline__ void group_all(const Params &p, int *smem) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int t = wave; t < p.T; t += NW)
    rt::topk_token<EC>(p.logits + (size_t)t * 64 * EC, p.E, p.k, lane, p.ids + (size_t)t * p.k, p.gates + (size_t)t * p.k);
  __syncthreads();
  perm::permute_block<NW>(p.ids, p.gates, p.T * p.k, p.k, p.lo, p.El, p.nbits, p.R_cap, p.counts, p.offsets,
                          p.row_token, p.row_w, p.token_row, smem);
  __syncthreads();
  if (wave == 0) {
    int n0 = 0;
    for (int b = 0; b < p.El; b += 64) {
      const int e = b + lane;
      const int beg = e < p.El ? p.offsets[e] : 0, cnt = e < p.El ? p.offsets[e + 1] - beg : 0;
      const int t = (cnt + mx4s::TM - 1) / mx4s::TM;
      const int incl = ffn::wave_incl_scan_i(t, lane), at = n0 + incl - t;
      for (int i = 0; i < t; i++)
        p.tiles[at + i] = make_int2(beg + i * mx4s::TM, e | min(mx4s::TM, cnt - i * mx4s::TM) << 16);
      n0 += __shfl(incl, 63, 64);
    }
    if (lane == 0) p.ctl[kTiles] = (uint32_t)n0;
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
  __syncthreads();
  if (threadIdx.x == 0) __hip_atomic_store(p.ctl + kRouted, 1u, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT);
}

template <int EC>
__global__ __launch_bounds__(NTHR, 2) void decode_route_gate_up_kernel(Params p) {  // two waves per SIMD
  extern __shared__ __attribute__((aligned(16))) float lds[];
  __shared__ int s_item;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int item;
  for (;;) {
    if (threadIdx.x == 0) s_item = (int)atomicAdd(p.ctl + kTicket, 1u);
    __syncthreads();
    item = __builtin_amdgcn_readfirstlane(s_item);
    __syncthreads();  // everyone has the item before thread 0 may draw the next one
    if (item >= p.n_route) break;
    route_item(p, item / EC, item % EC, 64 * EC, lds);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");  // logits and x codes before the count
    __syncthreads();
    if (threadIdx.x == 0) s_item = atomicAdd(p.ctl + kDone, 1u) == (uint32_t)p.n_route - 1u;
    __syncthreads();
    if (__builtin_amdgcn_readfirstlane(s_item)) {
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      group_all<EC>(p, (int *)lds);
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    int ok = 0;
    for (uint32_t i = 0; i < kSpinLimit; i++) {
      if (ld_agent(p.ctl + kRouted) != 0) {
        ok = 1;
        break;
      }
      __builtin_amdgcn_s_sleep(2);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");  // this CU's L1 and this XCD's L2 let go of older copies
    if (!ok) atomicOr(p.ctl + kError, 1u);
    s_item = ok ? (int)ld_agent(p.ctl + kTiles) : 0;
  }
  __syncthreads();
  const int nt = __builtin_amdgcn_readfirstlane(s_item), fid = item - p.n_route;
  const int ncb = p.I / 32, S = mx4s::split_for(nt * ncb, p.H), per = NW / S, nb = (ncb + per - 1) / per;
  for (int i = fid; i < nt * nb; i += gridDim.x) {
    const int ti = i / nb;
    const int2 d = p.tiles[ti];
    const int r0 = __builtin_amdgcn_readfirstlane(d.x), er = __builtin_amdgcn_readfirstlane(d.y);
    const int cb = (i - ti * nb) * per + wave / S;
    mx4s::gate_up_tile<mx4::FP8>(mx4s::Half{p.xq, p.xs, p.wgu, p.wgu_s}, p.H, p.I, er & 0xffff, cb * 32, r0,
                                 cb < ncb ? er >> 16 : 0, S, wave & (S - 1), [&](int r) { return (size_t)p.row_token[r]; },
                                 p.h, p.hs, lds);
  }
  __syncthreads();
  if (threadIdx.x == 0 && atomicAdd(p.ctl + kExit, 1u) == gridDim.x - 1u) {
    // every other workgroup has left: zero the control words for the next call (not the error word)
    for (int i = 0; i < kError; i++) __hip_atomic_store(p.ctl + i, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}

// Workgroups the device holds at once, per device and kernel instance (queried once).
template <typename K>
int resident_blocks(K kernel, size_t shm) {
  static std::mutex mu;
  static int cache[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (cache[dev] == 0) {
    int per_cu = 0, cus = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, kernel, NTHR, shm) != hipSuccess ||
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
      return 0;
    cache[dev] = per_cu * cus;
  }
  return cache[dev];
}

// LDS of launch 1: the widened row of x, the grouping's scratch or the partial sums, whichever is largest
// (the same for every call, so that the resident count is too).
constexpr size_t kLds = sizeof(float) * (kDecodeMx4MaxH > mx4s::RED_FLOATS ? kDecodeMx4MaxH : mx4s::RED_FLOATS);
static_assert(kLds >= sizeof(int) * (NW + 1) * kDecodeMx4MaxE, "the grouping's scratch fits");

template <int EC>
hipError_t launch(const Params &p, hipStream_t s) {
  auto kernel = decode_route_gate_up_kernel<EC>;
  const int resident = resident_blocks(kernel, kLds);
  if (resident <= 0) return hipErrorInvalidConfiguration;
  const int tiles = p.R_cap < p.El + p.R_cap / mx4s::TM ? p.R_cap : p.El + p.R_cap / mx4s::TM;
  const long long most = p.n_route + (long long)tiles * (p.I / 32);
  hipLaunchKernelGGL(kernel, dim3((unsigned)(most < resident ? most : resident)), dim3(NTHR), kLds, s, p);
  return hipGetLastError();
}

// Workspace pieces after the control words, each 256-byte aligned.
struct Layout {
  size_t logits, xq, xs, counts, offsets, row_token, token_row, row_w, tiles, h, hs, end;
  Layout(int T, int k, int El, int H, int I) {
    const size_t R = (size_t)T * (k < El ? k : El);
    size_t at = kCtlBytes;
    auto take = [&](size_t n) {
      const size_t o = at;
      at = align_up(at + n, 256);
      return o;
    };
    logits = take((size_t)T * kDecodeMx4MaxE * 4);
    xq = take((size_t)T * H);
    xs = take((size_t)T * (H / 32));
    counts = take((size_t)El * 4);
    offsets = take((size_t)(El + 1) * 4);
    row_token = take(R * 4);
    token_row = take((size_t)T * k * 4);
    row_w = take(R * 4);
    tiles = take((El + R / mx4s::TM) * sizeof(int2));
    h = take(R * I);
    hs = take(R * mx4::h_scale_stride(I));
    end = at;
  }
};

}  // namespace

size_t decode_layer_mx4_ws_bytes(int T, int k, int El, int H, int I) { return Layout(T, k, El, H, I).end; }

hipError_t launch_decode_layer_mx4(const DecodeMx4Args &a, hipStream_t s) {
  const Layout l(a.T, a.k, a.El, a.H, a.I);
  char *ws = (char *)a.ws;
  const int ec = ceil_div_i(a.E, 64), EC = ec <= 2 ? ec : 4;
  Params p{};
  p.x = (const uint16_t *)a.x;
  p.wr = a.wr;
  p.bias = a.bias;
  p.T = a.T;
  p.H = a.H;
  p.E = a.E;
  p.k = a.k;
  p.lo = a.lo;
  p.El = a.El;
  p.I = a.I;
  while ((1 << p.nbits) < a.El) p.nbits++;
  p.R_cap = a.T * (a.k < a.El ? a.k : a.El);
  p.n_route = a.T * EC;
  p.ids = a.ids;
  p.gates = a.gates;
  p.ctl = (uint32_t *)ws;
  p.logits = (float *)(ws + l.logits);
  p.xq = (uint8_t *)(ws + l.xq);
  p.xs = (uint8_t *)(ws + l.xs);
  p.counts = (int32_t *)(ws + l.counts);
  p.offsets = (int32_t *)(ws + l.offsets);
  p.row_token = (int32_t *)(ws + l.row_token);
  p.token_row = (int32_t *)(ws + l.token_row);
  p.row_w = (float *)(ws + l.row_w);
  p.tiles = (int2 *)(ws + l.tiles);
  p.wgu = a.wgu;
  p.wgu_s = a.wgu_s;
  p.h = (uint8_t *)(ws + l.h);
  p.hs = (uint8_t *)(ws + l.hs);
  const hipError_t err = EC == 1 ? launch<1>(p, s) : EC == 2 ? launch<2>(p, s) : launch<4>(p, s);
  if (err != hipSuccess) return err;
  FfnMx4Args d{};
  d.offsets = p.offsets;
  d.row_token = p.row_token;
  d.row_w = p.row_w;
  d.El = a.El;
  d.T = a.T;
  d.R_cap = p.R_cap;
  d.H = a.H;
  d.I = a.I;
  d.wd = a.wd;
  d.wd_s = a.wd_s;
  d.y = a.y;
  d.y_bf16 = a.y_bf16;
  return launch_down_sum_mx4(d, p.h, p.hs, s);
}
