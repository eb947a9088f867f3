// The whole MoE layer of a few tokens with MXFP4 experts in two launches (moe_decode_layer_mx4).
//
// Launch 1 routes, groups and computes the intermediate h; launch 2 is the down half of mx4_stream.h, which also
// sums to token order (and zeroes the control words).  In launch 1 the resident workgroups draw tickets.  The
// first T * ceil(E / 64) tickets are routing items (token t, 64 experts): the row of x is widened into LDS (the item
// of the first experts also quantises it to MXFP8 for the experts' products), one wave computes 64 logits, one
// lane each, with the library's fp32 chain over ascending h, and counts itself done.  A workgroup whose ticket is
// past the routing items waits for that count (for workgroups that drew earlier tickets, so they run; the wait is
// bounded all the same).  Then every workgroup takes the top k of every token and groups the assignments for
// itself, in LDS, rather than wait for one that does it and hands it out (a hand-over between workgroups on
// different XCDs costs about 5 us; one token 52 -> 37 us), the one with the first free ticket writes down what
// launch 2 needs, and all share the gate/up tiles.
//
// What bounds it: at one token the chain, H dependent additions whose order is the routing contract (3.0 ns each),
// then the weights' bytes.  Against instruction issue the chain has the packed fp32 router (no unpacking)
// and its x operand broadcast inside rows of 16 lanes by the FMA itself (DPP), so 16 steps cost 16 FMAs, four loads
// and one LDS read: 16 us of 4096 steps (12.4 for the FMAs alone, 10.2 without DPP).  Touching the matrix beforehand
// with the idle waves made it slower, 23 us.  Launch 1 takes 38 us for one token of 128 experts of 4096 x 1536, top 8
// (routing item 20, hand-over 3, top k and grouping 4, gate/up 11), 63 for five, 141 for 24, and 82 for 64 tokens and 32
// local experts (23, 7, 14, 38).
#include "mx4_stream.h"
#include "route_dev.h"

#include <mutex>

namespace {

constexpr int NTHR = mx4s::NTHR, NW = mx4s::NW;
constexpr uint32_t kSpinLimit = 1u << 22;  // polls of the count before giving up (seconds)

// control words
enum : int { kTicket = 0, kDone = 1, kError = 4, kCtlBytes = 256 };

struct Params {
  const uint16_t *x;   // [T, H] bf16
  const float *wr;     // [H/4, E, 4] fp32
  const float *bias;   // [E] or NULL
  int T, H, E, k, lo, El, I, R_cap, n_route;
  int32_t *ids;
  float *gates;
  uint32_t *ctl;
  float *logits;       // [T, 64 EC]
  uint8_t *xq, *xs;    // x as MXFP8
  int2 *dtiles;        // the down half's tiles {first row, expert | rows << 16}
  int *ndtiles;
  int32_t *row_token;
  float *row_w;
  const uint8_t *wgu, *wgu_s;
  uint8_t *h, *hs;
};

// What a routing item hands to other workgroups is stored at agent scope, i.e. through to memory, so that nothing
// has to be written back before it counts itself done.
__device__ __forceinline__ void st_agent(uint32_t *p, uint32_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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
  for (int v = threadIdx.x; v < H / 8; v += NTHR) {
    const u32x4_t r = *((const u32x4_t *)(p.x + (size_t)t * H) + v);
    const float f[8] = {bf16_lo(r.x), bf16_hi(r.x), bf16_lo(r.y), bf16_hi(r.y),
                        bf16_lo(r.z), bf16_hi(r.z), bf16_lo(r.w), bf16_hi(r.w)};
    *(f32x4_t *)(xf + 8 * v) = f32x4_t{f[0], f[1], f[2], f[3]};
    *(f32x4_t *)(xf + 8 * v + 4) = f32x4_t{f[4], f[5], f[6], f[7]};
    if (c == 0) {  // H is a multiple of 128: 16 neighbouring lanes loop together
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; j++) m = max(m, mx_abs_bits(f[j]));
      m = max(m, (uint32_t)__shfl_xor((int)m, 1, 64));
      m = max(m, (uint32_t)__shfl_xor((int)m, 2, 64));
      const uint32_t s = mx_scale_of_bits<8>(m);
      float u[8];
#pragma unroll
      for (int j = 0; j < 8; j++) u[j] = ldexpf(f[j], 127 - (int)s);
      const uint32_t lo = mx4::e4m3_quad(u[0], u[1], u[2], u[3]), hi = mx4::e4m3_quad(u[4], u[5], u[6], u[7]);
      uint32_t *xq = (uint32_t *)(p.xq + (size_t)t * H + 8 * v);
      st_agent(xq, s == 255 ? 0u : lo);
      st_agent(xq + 1, s == 255 ? 0u : hi);
      // the scale bytes of four blocks (16 lanes) as one dword
      uint32_t w = s << (8 * ((v >> 2) & 3));
      w |= (uint32_t)__shfl_xor((int)w, 4, 64);
      w |= (uint32_t)__shfl_xor((int)w, 8, 64);
      if ((v & 15) == 0) st_agent((uint32_t *)(p.xs + (size_t)t * (H / 32) + (v >> 2)), w);
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
    if (e < p.E) st_agent((uint32_t *)p.logits + (size_t)t * EP + e, __float_as_uint(p.bias ? acc + p.bias[e] : acc));
  }
}

// LDS after the partial sums (which the widened row of x shares): the grouping.  With at most 64 tokens, each on
// distinct experts, an expert's rows are a 64-bit set of tokens: its count is the set's, a row's place in the
// expert's group (token order) the number of lower members.
struct Groups {
  unsigned long long *set;  // [El]
  int2 *sel;                // [T, k] {local expert or -1, gate}
  int2 *tiles;              // {first row, expert | rows << 16}
  int *first;               // [El] first row of an expert
  int *token;               // [R_cap] token of a row
  __device__ Groups(const Params &p, char *at) {
    set = (unsigned long long *)at;
    sel = (int2 *)(set + p.El);
    tiles = sel + p.T * p.k;
    first = (int *)(tiles + p.El + p.R_cap / mx4s::TM);
    token = first + p.El;
  }
};
constexpr size_t kGroupBytes = kDecodeMx4MaxE * 20 + kMx4StreamMaxT * 32 * 12 + kMx4StreamMaxT * 32 / mx4s::TM * 8;

// Top k and gates, the grouping and the tile list; ``write``: also to memory.  Returns the number of tiles.
template <int EC>
__device__ __forceinline__ int group_all(const Params &p, const Groups &g, bool write, int *s_n, float *scratch) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), N = p.T * p.k;
  for (int e = threadIdx.x; e < p.El; e += NTHR) g.set[e] = 0;
  // the logits in one go, so that a wave's tokens do not wait for memory one after the other
  const bool staged = p.T * 64 * EC <= mx4s::RED_FLOATS;
  if (staged)
    for (int i = threadIdx.x; i < p.T * 16 * EC; i += NTHR) *((f32x4_t *)scratch + i) = *((const f32x4_t *)p.logits + i);
  __syncthreads();
  // A wave's tokens are wave, wave + NW, ...; four at a time when it has more than one (64 tokens, 32 local experts:
  // 83.5 -> 80 us).
  auto pick = [&](auto NC, int t0) __attribute__((always_inline)) {
    constexpr int N = decltype(NC)::value;
    const float *l[N];
    int e[N];
    float w[N];
#pragma unroll
    for (int i = 0; i < N; i++) l[i] = (staged ? scratch : p.logits) + (size_t)min(t0 + i * NW, p.T - 1) * 64 * EC;
    rt::topk_lanes<EC, N>(l, p.E, p.k, lane, e, w);
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int t = t0 + i * NW;
      if (lane >= p.k || t >= p.T) continue;
      if (write) {
        p.ids[(size_t)t * p.k + lane] = e[i];
        p.gates[(size_t)t * p.k + lane] = w[i];
      }
      const int el = (unsigned)(e[i] - p.lo) < (unsigned)p.El ? e[i] - p.lo : -1;
      if (el >= 0) atomicOr(g.set + el, 1ull << t);
      g.sel[t * p.k + lane] = make_int2(el, __float_as_int(w[i]));
    }
  };
  if (p.T <= NW) {
    if (wave < p.T) pick(std::integral_constant<int, 1>{}, wave);
  } else {
    for (int t = wave; t < p.T; t += 4 * NW) pick(std::integral_constant<int, 4>{}, t);
  }
  __syncthreads();
  if (wave == 0) {
    int n0 = 0, t0 = 0, d0 = 0;
    for (int b = 0; b < p.El; b += 64) {
      const int e = b + lane, cnt = e < p.El ? __popcll(g.set[e]) : 0, t = (cnt + mx4s::TM - 1) / mx4s::TM;
      const int ci = ffn::wave_incl_scan_i(cnt, lane), ti = ffn::wave_incl_scan_i(t, lane);
      const int beg = n0 + ci - cnt;
      if (e < p.El) g.first[e] = beg;
      if (write) {  // the down half's tiles
        const int dt = (cnt + mx4s::TD - 1) / mx4s::TD, di = ffn::wave_incl_scan_i(dt, lane);
        for (int i = 0; i < dt; i++)
          p.dtiles[d0 + di - dt + i] = make_int2(beg + i * mx4s::TD, e | min(mx4s::TD, cnt - i * mx4s::TD) << 16);
        d0 += __shfl(di, 63, 64);
      }
      for (int i = 0; i < t; i++)
        g.tiles[t0 + ti - t + i] = make_int2(beg + i * mx4s::TM, e | min(mx4s::TM, cnt - i * mx4s::TM) << 16);
      n0 += __shfl(ci, 63, 64);
      t0 += __shfl(ti, 63, 64);
    }
    if (lane == 0) {
      if (write) *p.ndtiles = d0;
      *s_n = t0;
    }
  }
  __syncthreads();
  for (int a = threadIdx.x; a < N; a += NTHR) {
    const int2 d = g.sel[a];
    const int t = a / p.k;
    if (d.x < 0) continue;
    const int r = g.first[d.x] + __popcll(g.set[d.x] & ((1ull << t) - 1));
    g.token[r] = t;
    if (write) {
      p.row_token[r] = t;
      p.row_w[r] = __int_as_float(d.y);
    }
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(*s_n);
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
    __builtin_amdgcn_s_waitcnt(0);  // this wave's stores have reached memory
    __syncthreads();
    if (threadIdx.x == 0) __hip_atomic_fetch_add(p.ctl + kDone, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // Closes thread 0's part before the next ticket.  Without it the compiler joins the two conditionals across the
    // loop's back edge, and the other lanes of its wave go round the loop without it, for ever on the old ticket.
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    int ok = 0;
    for (uint32_t i = 0; i < kSpinLimit && !ok; i++) {
      ok = __hip_atomic_load(p.ctl + kDone, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) >= (uint32_t)p.n_route;
      if (!ok) __builtin_amdgcn_s_sleep(1);
    }
    if (!ok) atomicOr(p.ctl + kError, 1u);
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");  // this CU's L1 and this XCD's L2 let go of older copies
  }
  __syncthreads();
  const int fid = item - p.n_route;
  const Groups g(p, (char *)(lds + mx4s::RED_FLOATS));
  const int nt = group_all<EC>(p, g, fid == 0, &s_item, lds);
  const int ncb = p.I / 32, S = mx4s::split_for(nt * ncb, p.H), per = NW / S, nb = (ncb + per - 1) / per;
  for (int i = fid; i < nt * nb; i += gridDim.x) {
    const int ti = i / nb;
    const int2 d = g.tiles[ti];
    const int r0 = __builtin_amdgcn_readfirstlane(d.x), er = __builtin_amdgcn_readfirstlane(d.y);
    const int cb = (i - ti * nb) * per + wave / S;
    mx4s::gate_up_tile<mx4::FP8>(mx4s::Half{p.xq, p.xs, p.wgu, p.wgu_s}, p.H, p.I, er & 0xffff, cb * 32, r0,
                                 cb < ncb ? er >> 16 : 0, S, wave & (S - 1), [&](int r) { return (size_t)g.token[r]; },
                                 p.h, p.hs, lds);
  }
}

// Workgroups the device holds at once, per device and kernel (queried once; every call has the same LDS).
template <auto KERNEL>
int resident_blocks(size_t shm) {
  static std::mutex mu;
  static int cache[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (cache[dev] == 0) {
    int per_cu = 0, cus = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, KERNEL, NTHR, shm) != hipSuccess ||
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
      return 0;
    cache[dev] = per_cu * cus;
  }
  return cache[dev];
}

// LDS of launch 1, the same for every call, so that the resident count is too.
static_assert(kDecodeMx4MaxH <= mx4s::RED_FLOATS, "the widened row of x fits where the partial sums go");
constexpr size_t kLds = sizeof(float) * mx4s::RED_FLOATS + kGroupBytes;

template <int EC>
hipError_t launch(const Params &p, hipStream_t s) {
  constexpr auto kernel = decode_route_gate_up_kernel<EC>;
  const int resident = resident_blocks<kernel>(kLds);
  if (resident <= 0) return hipErrorInvalidConfiguration;
  const int tiles = p.R_cap < p.El + p.R_cap / mx4s::TM ? p.R_cap : p.El + p.R_cap / mx4s::TM;
  const long long most = p.n_route + (long long)tiles * (p.I / 32);
  hipLaunchKernelGGL(kernel, dim3((unsigned)(most < resident ? most : resident)), dim3(NTHR), kLds, s, p);
  return hipGetLastError();
}

// Workspace pieces after the control words, each 256-byte aligned.
struct Layout {
  size_t logits, xq, xs, dtiles, ndtiles, row_token, row_w, h, hs, end;
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
    dtiles = take((size_t)mx4s::max_tiles(T, El) * sizeof(int2));
    ndtiles = take(sizeof(int));
    row_token = take(R * 4);
    row_w = take(R * 4);
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
  p.R_cap = a.T * (a.k < a.El ? a.k : a.El);
  p.n_route = a.T * EC;
  p.ids = a.ids;
  p.gates = a.gates;
  p.ctl = (uint32_t *)ws;
  p.logits = (float *)(ws + l.logits);
  p.xq = (uint8_t *)(ws + l.xq);
  p.xs = (uint8_t *)(ws + l.xs);
  p.dtiles = (int2 *)(ws + l.dtiles);
  p.ndtiles = (int *)(ws + l.ndtiles);
  p.row_token = (int32_t *)(ws + l.row_token);
  p.row_w = (float *)(ws + l.row_w);
  p.wgu = a.wgu;
  p.wgu_s = a.wgu_s;
  p.h = (uint8_t *)(ws + l.h);
  p.hs = (uint8_t *)(ws + l.hs);
  const hipError_t err = EC == 1 ? launch<1>(p, s) : EC == 2 ? launch<2>(p, s) : launch<4>(p, s);
  if (err != hipSuccess) return err;
  FfnMx4Args d{};
  d.tiles = p.dtiles;
  d.ntiles = p.ndtiles;
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
  d.zero = p.ctl;
  d.n_zero = kDone + 1;
  return launch_down_sum_mx4(d, p.h, p.hs, s);
}
