// layer.cu -- a whole mixture-of-experts layer for a few tokens (T <= 32) in
// two launches, on NF4 or MXFP4 expert weights.
//
//   l[t, e] = sum_k x[t, k] Wr[e, k] (+ b[e]); ids, w = the k largest and their
//   softmax weights (route.cuh); per slot (t, s) with e = ids[t, s]:
//     h = silu(x Wg_e^T) * (x Wu_e^T),  y = h Wd_e^T;   out[t] = sum_s w y
//
// Kernel 1 (moe_router): the router logits, one CTA per expert and 8 tokens,
// fp32 chains of at most H / 256 products; it also zeroes kernel 2's counters.
// Kernel 2 (moe_experts), one CTA per SM, launched early behind kernel 1
// (programmatic dependent launch: its codebook table is built meanwhile):
//   every CTA chooses the experts itself from the logits (no third kernel);
//   phase A  gate_up + SwiGLU in units of (expert, 8 gate rows + the matching
//            8 up rows), h written as bf16 high and low parts;
//   phase B  down in units of (16 rows, expert), y in fp32; the CTA that
//            finishes a tile's last expert combines the tile's slots in slot
//            order (no sum depends on the order of arrival).
//   Between the phases a CTA waits until all of phase A is done.  Shares of
//   both phases are claimed from counters, and a CTA waits only once no share
//   of phase A is unclaimed, so every share waited for is held by a running
//   CTA: the wait ends whether or not all CTAs are resident at a time, also
//   with other kernels on the device.
//
// Bound: the active experts' packed bytes from HBM, and the decode's
// instructions.  16 warps each own a ring of four 2 KB stages (16 weight rows
// x 256 k) filled by cp.async three stages ahead -- across the wait between
// the phases too: the next phase's weights do not depend on it.  A packed byte
// becomes two bf16 values by one conflict-free table lookup and goes straight
// into mma.sync m16n8k16 as the A operand (weights are M, tokens N), 64 k of
// one scale block at a time; block sums are scaled in fp32.  The low part of h
// keeps the down projection's input at 16 bits of mantissa, at one more mma
// and no conversion.  A unit's K is split over several warps (joined through
// shared memory in a fixed order) when a CTA has fewer units than warps.
#include <algorithm>

#include "common.cuh"
#include "launch.cuh"
#include "route.cuh"

namespace gbw {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxE = 1024;
constexpr int kMaxP = 512;
constexpr int kRows = 8;           // most rows of a group: rows of one expert that share a decode
constexpr int CKB = 128;           // bytes per weight row and stage: 256 k
constexpr int D = 4;               // stages per warp
constexpr int kStage = 16 * CKB;   // 2 KB
constexpr int kScStage = 256;      // scales of a stage

// Shared memory by address in the shared window (dynamic shared memory starts
// at 1 KB).  The table lies at 64 KB: entry b of lane l at 65536 + b * 256 +
// l * 4, so that one byte permute of a packed word gives the whole address.
// The other half of each 256 bytes holds partial sums: two pieces per warp of
// up to 8 rows of 32 floats.  The warps' rings lie on both sides of it.
static_assert(kWarps * 2 * 8 <= 256, "partial sums fit beside the table");
constexpr int kLowWarps = 7;
struct Smem {
  static constexpr int ids = 1024;               // [kMaxP] int
  static constexpr int wts = ids + 4 * kMaxP;    // [kMaxP] float
  static constexpr int rows = wts + 4 * kMaxP;   // [kMaxP] uint16 slot of sorted row
  static constexpr int active = rows + 2 * kMaxP;  // [kMaxP] uint16 expert
  static constexpr int misc = active + 2 * kMaxP;  // 16 ints
  static constexpr int part = misc + 64;           // [kWarps] scan parts
  static constexpr int low_end = part + 4 * kWarps;
  static constexpr int table = 65536;
  static constexpr int ring_low = table - kLowWarps * D * kStage;
  static constexpr int ring_high = 2 * table;
  static constexpr int scales = ring_high + (kWarps - kLowWarps) * D * kStage;
  static constexpr int first = scales + kWarps * D * kScStage;  // [kMaxP + 4] int first sorted row
  static constexpr int count = first + 4 * (kMaxP + 4);  // [kMaxE] int: token bits, then first row
  static constexpr int end = count + 4 * kMaxE;
};
static_assert(Smem::low_end <= Smem::ring_low, "the small arrays fit below the rings");
static_assert(Smem::end <= 232448, "shared memory exceeds the 227 KB a CTA can have");

struct LayerArgs {
  LayerProblem p;
  float* logits;      // [T, E]
  uint16_t* hhi;      // [P, I] bf16
  uint16_t* hlo;      // [P, I] bf16
  float* y;           // [P, H]
  int* counters;      // claimA, claimB, doneA, then one per 16 columns of H
};

constexpr int kCounters = 4;

// ----------------------------------------------------------------------
// kernel 1
// ----------------------------------------------------------------------

constexpr int kRouterThreads = 512;  // at most; H / 8 rounded up to warps else
constexpr int kRouterTokens = 8;

__global__ void __launch_bounds__(kRouterThreads) moe_router(const LayerArgs a) {
  const LayerProblem& p = a.p;
  __shared__ float part[kRouterThreads / 32][kRouterTokens];
  grid_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < kCounters + (int)(p.H / 16); i += blockDim.x) a.counters[i] = 0;
  const int e = blockIdx.x, t0 = blockIdx.y * kRouterTokens;
  const int n = min(kRouterTokens, (int)p.T - t0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int U = (int)(p.H / 8);
  const uint4* w = reinterpret_cast<const uint4*>(p.rw + (int64_t)e * p.H);
  float acc[kRouterTokens] = {};
  for (int u = threadIdx.x; u < U; u += blockDim.x) {
    const uint4 wv = __ldg(w + u);
    const uint32_t wx[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int j = 0; j < kRouterTokens; ++j) {
      if (j < n) {
        const uint4 xv = __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)(t0 + j) * p.H) + u);
        const uint32_t xx[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[j] = fmaf(__uint_as_float(wx[i] << 16), __uint_as_float(xx[i] << 16), acc[j]);
          acc[j] = fmaf(__uint_as_float(wx[i] & 0xFFFF0000u), __uint_as_float(xx[i] & 0xFFFF0000u),
                        acc[j]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kRouterTokens; ++j) {
    if (j < n) {
      const float v = warp_sum(acc[j]);
      if (lane == 0) part[warp][j] = v;
    }
  }
  __syncthreads();
  if (threadIdx.x < (unsigned)n) {
    float v = 0.0f;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) v += part[i][threadIdx.x];
    if (p.rb) v += __ldg(p.rb + e);
    a.logits[(int64_t)(t0 + threadIdx.x) * p.E + e] = v;
  }
}

// ----------------------------------------------------------------------
// kernel 2
// ----------------------------------------------------------------------

// The NF4 levels enter the table times this, and the scales times its inverse:
// of the factors in [1, 2) it is the one whose products with the 16 levels
// round to bf16 with the least error, 6.3e-4 of their root mean square (1.1e-3
// without it).
constexpr float kLevelScale = 1.437f;

// Codebook value q as its bf16 bit pattern (a select tree: an indexed array
// would live in local memory).
template <Fmt F>
__device__ __forceinline__ uint32_t code_bf16(int q) {
  float v;
  if (F == Fmt::NF4) {
    const float a0 = q & 1 ? -0.6961928009986877f : -1.0f;
    const float a1 = q & 1 ? -0.39491748809814453f : -0.5250730514526367f;
    const float a2 = q & 1 ? -0.18477343022823334f : -0.28444138169288635f;
    const float a3 = q & 1 ? 0.0f : -0.09105003625154495f;
    const float a4 = q & 1 ? 0.16093020141124725f : 0.07958029955625534f;
    const float a5 = q & 1 ? 0.33791524171829224f : 0.24611230194568634f;
    const float a6 = q & 1 ? 0.5626170039176941f : 0.44070982933044434f;
    const float a7 = q & 1 ? 1.0f : 0.7229568362236023f;
    const float b0 = q & 2 ? a1 : a0, b1 = q & 2 ? a3 : a2, b2 = q & 2 ? a5 : a4, b3 = q & 2 ? a7 : a6;
    const float c0 = q & 4 ? b1 : b0, c1 = q & 4 ? b3 : b2;
    v = __fmul_rn(q & 8 ? c1 : c0, kLevelScale);
  } else {
    // e2m1: 0, 1/2, then (1 + m / 2) 2^(x - 1)
    const int x = (q >> 1) & 3, m = q & 1;
    v = x ? (float)((2 + m) << (x - 1)) * 0.5f : 0.5f * m;
    v = q & 8 ? -v : v;
  }
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// D = A (16 x 16, row) * B (16 x 8, col) (+ D), bf16 in, fp32 out.
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A table entry: the table does not change after the block has built it, so
// the load may be moved freely (its address comes from data read later).
__device__ __forceinline__ uint32_t lds_table(uint32_t addr) {
  uint32_t v;
  asm("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}

__device__ __forceinline__ int ld_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// 16-byte unit u of row r of a stage is stored at u ^ swizzle(r): the rows'
// lanes then read different banks (NF4: 8 bytes a lane, 4 rows a wavefront;
// MXFP4: 4 bytes a lane, 8 rows).
template <Fmt F>
__device__ __forceinline__ uint32_t swizzle(int r) {
  return F == Fmt::NF4 ? 2u * (r & 3) : (uint32_t)(r & 7);
}

// One phase's share of this CTA: units [u0, u0 + n) of nc chunks (256 k)
// each.  Warp w multiplies chunks [w L / 16, (w + 1) L / 16) of the L = n * nc,
// so that all warps have the same work; a unit that ends up in several warps
// is joined from their partial sums in order.
struct Share {
  int phase;  // 0: gate_up, 1: down
  int u0, n, nc;
  __device__ __forceinline__ int begin(int w) const { return (w * n * nc) / kWarps; }
};

// A lane's place in its warp's stream of chunks to load.
struct Cursor {
  int phase, left;          // chunks left of this share's range
  int ai, tile, c;          // group, output tile and chunk of the unit
  const uint8_t* w;         // this lane's first 16 code bytes of the chunk
  const uint8_t* sc;        // this lane's first scale of the chunk
};

template <Fmt F, int NPL>
__global__ void __launch_bounds__(kThreads, 1) moe_experts(const LayerArgs a, const int aligned) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const LayerProblem& p = a.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int T = (int)p.T, E = p.E, k = p.k, P = T * k;
  const int H = (int)p.H, I = (int)p.I;
  uint8_t* smem = smem_raw - smem_u32(smem_raw);  // indexed by shared address
  int* ids = reinterpret_cast<int*>(smem + Smem::ids);
  float* wts = reinterpret_cast<float*>(smem + Smem::wts);
  uint16_t* rows = reinterpret_cast<uint16_t*>(smem + Smem::rows);
  uint16_t* active = reinterpret_cast<uint16_t*>(smem + Smem::active);
  int* first = reinterpret_cast<int*>(smem + Smem::first);
  volatile int* misc = reinterpret_cast<volatile int*>(smem + Smem::misc);
  int* part = reinterpret_cast<int*>(smem + Smem::part);
  int* count = reinterpret_cast<int*>(smem + Smem::count);
  if (smem_u32(smem_raw) > Smem::ids) {  // (the layout above takes 1 KB as given)
    raise_error(p.err, GBW_DEVERR_TIMEOUT);
    return;
  }
  // misc: 0 claim A, 1 claim B, 2 next claim, 3 abort, 4 groups, 5 last of a tile,
  // 6 rows of the largest expert

  {
    // warp w writes the 16 bytes of high nibble w: lane l holds level l & 15
    const uint32_t level = code_bf16<F>(lane & 15), top = code_bf16<F>(warp);
#pragma unroll
    for (int l = 0; l < 16; ++l) {
      const uint32_t low = __shfl_sync(0xffffffffu, level, l);
      sts32(Smem::table + (warp * 16 + l) * 256 + lane * 4,
            F == Fmt::NF4 ? top | (low << 16) : low | (top << 16));
    }
  }
  for (int e = threadIdx.x; e < E; e += kThreads) count[e] = 0;
  if (threadIdx.x == 0) misc[3] = misc[6] = 0;
  __syncthreads();
  grid_dependency_wait();
  if (threadIdx.x == 0) {
    misc[0] = atomicAdd(&a.counters[0], 1);
    misc[1] = atomicAdd(&a.counters[1], 1);
  }

  // ---- the choice of experts, the same in every CTA
  for (int t = warp; t < T; t += kWarps) {
    int id = 0;
    float w = 0.0f;
    choose<LogitL2, NPL>(reinterpret_cast<const LogitL2*>(a.logits) + (int64_t)t * E, E, k, p.renorm,
                         lane, id, w);
    if (lane < k) {
      ids[t * k + lane] = id;
      wts[t * k + lane] = w;
      atomicOr(&count[id], 1 << t);
    }
  }
  __syncthreads();
  // rows sorted by expert and cut into groups of at most kRows rows of one
  // expert: two packed scans (rows below, groups below), two experts per thread.
  // count[e] holds the tokens of expert e as bits (T <= 32), so a slot's place
  // among its expert's rows is the number of lower bits: the same in every
  // CTA, as it must be for the groups to hold the same rows everywhere.
  {
    static_assert(kMaxP <= kThreads, "one slot per thread");
    const int e0 = threadIdx.x * 2;
    const int c0 = e0 < E ? __popc(count[e0]) : 0, c1 = e0 + 1 < E ? __popc(count[e0 + 1]) : 0;
    const int slot = threadIdx.x, id = slot < P ? ids[slot] : 0;
    const int at = slot < P ? __popc(count[id] & ((1 << (slot / k)) - 1)) : 0;
    const int g0 = (c0 + kRows - 1) / kRows, g1 = (c1 + kRows - 1) / kRows;
    const int v = (c0 + c1) | ((g0 + g1) << 16);
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int s = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += s;
    }
    if (lane == 31) part[warp] = incl;
    const int top = __reduce_max_sync(0xffffffffu, max(c0, c1));
    if (lane == 0) atomicMax(const_cast<int*>(&misc[6]), top);
    __syncthreads();
    int below = incl - v;
    for (int i = 0; i < warp; ++i) below += part[i];
    const int r0 = below & 0xFFFF, a0 = below >> 16;
    for (int j = 0; j < g0; ++j) {
      active[a0 + j] = (uint16_t)e0;
      first[a0 + j] = r0 + j * kRows;
    }
    for (int j = 0; j < g1; ++j) {
      active[a0 + g0 + j] = (uint16_t)(e0 + 1);
      first[a0 + g0 + j] = r0 + c0 + j * kRows;
    }
    if (threadIdx.x == kThreads - 1) {
      misc[4] = (below + v) >> 16;
      first[(below + v) >> 16] = P;
    }
    __syncthreads();
    if (e0 < E) count[e0] = r0;
    if (e0 + 1 < E) count[e0 + 1] = r0 + c0;
    __syncthreads();
    if (slot < P) rows[count[id] + at] = (uint16_t)slot;
  }
  __syncthreads();
  const int A = misc[4];  // groups
  const int G = gridDim.x;
  int next_a = misc[0], next_b = misc[1];
  const int tiles_a = I / 8, tiles_b = H / 16;

  // Column tiles of 8: phase A, up to 8 rows of a group are one tile; phase B,
  // 4 rows a tile, the high parts of h in columns 0..3, the low ones in 4..7.
  const bool two_tiles = misc[6] > 4;  // some group has more than 4 rows
  auto make_share = [&](int phase, int idx) __attribute__((always_inline)) -> Share {
    Share s;
    s.phase = phase;
    const int tiles = phase ? tiles_b : tiles_a;
    // phase B, aligned: whole tiles, so that no tile is shared between CTAs
    const int per = phase && aligned ? A : 1;
    const unsigned total = (unsigned)(per > 1 ? tiles : tiles * A);
    const unsigned q = total / (unsigned)G, r = total - q * (unsigned)G;
    s.u0 = (int)(q * idx + min((unsigned)idx, r)) * per;
    s.n = idx < G ? (int)(q + (idx < (int)r)) * per : 0;
    s.nc = ((phase ? I : H) + 255) >> 8;
    return s;
  };

  // (group, output tile) of unit u, and of the one after it
  auto unit_of = [&](int phase, int u, int& ai, int& tile) __attribute__((always_inline)) {
    const int d = phase ? A : tiles_a, q = u / d, r = u - q * d;
    ai = phase ? r : q;
    tile = phase ? q : r;
  };
  auto next_unit = [&](int phase, int& ai, int& tile) __attribute__((always_inline)) {
    if (phase) {
      if (++ai == A) { ai = 0; ++tile; }
    } else {
      if (++tile == tiles_a) { tile = 0; ++ai; }
    }
  };

  constexpr int kScChunk = F == Fmt::NF4 ? 16 : 8;                // scale bytes per row and chunk
  const int kb_a = H / 2, kb_b = I / 2;                           // bytes of codes per row
  const int sr_a = F == Fmt::NF4 ? H / 16 : H / 32;               // scale bytes per row
  const int sr_b = F == Fmt::NF4 ? I / 16 : I / 32;

  // cp.async: this lane copies 16-byte unit my_unit of rows my_row + 4 j
  const int my_row = lane >> 3, my_unit = lane & 7;
  const int sc_row = lane >> 1, sc_half = lane & 1;  // and two scale words of row sc_row

  // Points cur's lane pointers at its chunk.  Rows 8 .. 15 of a gate_up unit
  // are the up rows, I - 8 further.
  auto point = [&](Cursor& cur) __attribute__((always_inline)) {
    const int e = active[cur.ai];
    if (cur.phase) {
      const int64_t row = (int64_t)e * H + cur.tile * 16;
      cur.w = p.dn + (row + my_row) * kb_b + cur.c * CKB + my_unit * 16;
      cur.sc = static_cast<const uint8_t*>(p.dn_scale) + (row + sc_row) * sr_b + cur.c * kScChunk +
               sc_half * (kScChunk / 2);
    } else {
      const int64_t row = (int64_t)e * 2 * I + cur.tile * 8;
      cur.w = p.gu + (row + my_row) * kb_a + cur.c * CKB + my_unit * 16;
      cur.sc = static_cast<const uint8_t*>(p.gu_scale) +
               (row + sc_row + (sc_row >= 8 ? I - 8 : 0)) * sr_a + cur.c * kScChunk +
               sc_half * (kScChunk / 2);
    }
  };

  // this warp's ring, as shared addresses
  const uint32_t ring = warp < kLowWarps ? Smem::ring_low + warp * (D * kStage)
                                         : Smem::ring_high + (warp - kLowWarps) * (D * kStage);
  const uint32_t ring_s = Smem::scales + warp * (D * kScStage);
  const uint32_t put_w0 = ring + my_row * CKB + (my_unit ^ swizzle<F>(my_row)) * 16;
  const uint32_t put_w1 = ring + (my_row + 4) * CKB + (my_unit ^ swizzle<F>(my_row + 4)) * 16;
  const uint32_t put_s = ring_s + sc_row * 16 + sc_half * 8;
  uint32_t sv0 = 0, sv1 = 0;  // scales loaded for the stage before
  uint32_t sv_to = 0;         // their place, or 0: none pending

  auto put_scales = [&]() __attribute__((always_inline)) {
    if (sv_to == 0) return;
    if (F == Fmt::NF4) {
      sv0 = __float_as_uint(__uint_as_float(sv0) * (1.0f / kLevelScale));
      sv1 = __float_as_uint(__uint_as_float(sv1) * (1.0f / kLevelScale));
    } else {
      // e8m0 byte s -> bf16 bits of 2^(s - 127): s << 7, but 0 and 255
      const uint32_t v = prmt(sv0, sv1, 0x5410u);
      sv0 = prmt(v, 0u, 0x4140u) << 7;
      sv1 = prmt(v, 0u, 0x4342u) << 7;
      const uint32_t zero = (v - 0x01010101u) & ~v, ones = (~v - 0x01010101u) & v;
      if ((zero | ones) & 0x80808080u) {  // a byte of 0 or 255 among them
        auto fix = [](uint32_t h) -> uint32_t { return h == 0u ? 0x40u : h == 0x7F80u ? 0x7FC0u : h; };
        sv0 = fix(sv0 & 0xFFFFu) | (fix(sv0 >> 16) << 16);
        sv1 = fix(sv1 & 0xFFFFu) | (fix(sv1 >> 16) << 16);
      }
    }
    sts64(sv_to, sv0, sv1);
    sv_to = 0;
  };

  // ---- the warp's stream of chunks: share A, then share B
  Share sa = make_share(0, next_a), sb = make_share(1, next_b);
  uint32_t q_in = 0, q_out = 0;  // ring slots of the next chunk to load and to multiply
  Cursor pc{};                   // next chunk to load, if pc.left > 0
  auto enter = [&](const Share& s) __attribute__((always_inline)) {
    const int f = s.begin(warp);
    pc.phase = s.phase;
    pc.left = s.begin(warp + 1) - f;
    if (pc.left > 0) {
      const int u = f / s.nc;
      pc.c = f - u * s.nc;
      unit_of(s.phase, s.u0 + u, pc.ai, pc.tile);
      point(pc);
    }
  };
  // Loads the next chunk into its ring slot; its scales reach shared memory
  // with the call after this one, two calls before they are read.
  auto issue = [&]() __attribute__((always_inline)) {
    put_scales();
    if (pc.left == 0 && pc.phase == 0) enter(sb);
    if (pc.left > 0) {
      const int kb = pc.phase ? kb_b : kb_a;
      const int bytes = kb - pc.c * CKB;  // of a row, from this chunk on
      const uint32_t slot = q_in * kStage;
      const uint8_t* up = pc.w + (int64_t)(pc.phase ? 8 : I) * kb;
      if (my_unit * 16 < bytes) {
        cp_async_16(put_w0 + slot, pc.w);
        cp_async_16(put_w1 + slot, pc.w + 4 * kb);
        cp_async_16(put_w0 + slot + 8 * CKB, up);
        cp_async_16(put_w1 + slot + 8 * CKB, up + 4 * kb);
      }
      const int words = (bytes >> 5) - sc_half * 2;  // scale words left: one per 64 k
      if (F == Fmt::NF4) {
        if (words > 0) sv0 = __ldg(reinterpret_cast<const uint32_t*>(pc.sc));
        if (words > 1) sv1 = __ldg(reinterpret_cast<const uint32_t*>(pc.sc) + 1);
      } else {
        if (words > 0) sv0 = __ldg(reinterpret_cast<const uint16_t*>(pc.sc));
        if (words > 1) sv1 = __ldg(reinterpret_cast<const uint16_t*>(pc.sc) + 1);
      }
      sv_to = put_s + q_in * kScStage;
      q_in = (q_in + 1) & (D - 1);
      --pc.left;
      ++pc.c;
      if (bytes > CKB) {
        pc.w += CKB;
        pc.sc += kScChunk;
      } else {
        pc.c = 0;
        next_unit(pc.phase, pc.ai, pc.tile);
        if (pc.left > 0) point(pc);
      }
    }
    cp_async_commit();
  };

  const int g = lane >> 2, t4 = lane & 3;
  const uint32_t lut = Smem::table | (uint32_t)lane * 4u;

  constexpr int kSecond = F == Fmt::NF4 ? 8 : 32;  // distance of a lane's second 8 k

  // This lane's column in column tile i of a group (r0, cnt), at its first k of
  // a stage.  Columns past the group's rows repeat its last row; nothing reads
  // them.
  auto column = [&](int phase, int r0, int cnt, int i) __attribute__((always_inline)) -> const uint16_t* {
    const int row = min(phase ? i * 4 + (g & 3) : i * 8 + g, cnt - 1);
    const int slot = rows[r0 + row], k0 = t4 * (F == Fmt::NF4 ? 16 : 8);
    if (phase == 0) return p.x + (int64_t)(slot / k) * H + k0;
    return (g < 4 ? a.hhi : a.hlo) + (int64_t)slot * I + k0;
  };
  // plain loads: h was written by other CTAs of this launch, before the wait
  auto load_x = [&](const uint16_t* xp, uint4& x0, uint4& x1) __attribute__((always_inline)) {
    x0 = *reinterpret_cast<const uint4*>(xp);
    x1 = *reinterpret_cast<const uint4*>(xp + kSecond);
  };
  // Weight fragments of block b of a stage: the lane's 16 weights of rows g and
  // g + 8 (same swizzle).  NF4, one scale block: bytes 8 t4 .. of its 32;
  // MXFP4, two blocks of 16 bytes: 4 bytes of each, so that every mma stays
  // inside a scale block.  `st` is this lane's address in block 0; the blocks
  // differ in address bits 5 and 6 alone.
  const uint32_t get_w = ring + g * CKB + (F == Fmt::NF4 ? ((t4 >> 1) ^ swizzle<F>(g)) * 16 + (t4 & 1) * 8
                                                         : swizzle<F>(g) * 16 + t4 * 4);
  const uint32_t get_s = ring_s + g * 16;
  auto decode = [&](uint32_t st, int b, uint32_t (&fa)[8], uint32_t (&fb)[8]) __attribute__((always_inline)) {
    uint2 wa, wb;
    const uint8_t* at = smem + (st ^ (b * 32));
    if (F == Fmt::NF4) {
      wa = *reinterpret_cast<const uint2*>(at);
      wb = *reinterpret_cast<const uint2*>(at + 8 * CKB);
    } else {
      const uint8_t* au = smem + (st ^ (b * 32 + 16));
      wa.x = *reinterpret_cast<const uint32_t*>(at);
      wa.y = *reinterpret_cast<const uint32_t*>(au);
      wb.x = *reinterpret_cast<const uint32_t*>(at + 8 * CKB);
      wb.y = *reinterpret_cast<const uint32_t*>(au + 8 * CKB);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // byte i & 3 to address bits 8 .. 15, the table's base and the lane around
      const uint32_t sel = 0x7604u | ((uint32_t)(i & 3) << 4);
      fa[i] = lds_table(prmt(i < 4 ? wa.x : wa.y, lut, sel));
      fb[i] = lds_table(prmt(i < 4 ? wb.x : wb.y, lut, sel));
    }
  };
  // acc += block b (scale words sg, sh of rows g, g + 8) times the lane's x
  auto mma_block = [&](float (&acc)[4], const uint32_t (&fa)[8], const uint32_t (&fb)[8],
                       const uint4& x0, const uint4& x1, uint32_t sg, uint32_t sh) __attribute__((always_inline)) {
    const uint32_t xb[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
    constexpr int kPer = F == Fmt::NF4 ? 4 : 2;  // mma of one scale block
#pragma unroll
    for (int m0 = 0; m0 < 4; m0 += kPer) {
      float d[4];
#pragma unroll
      for (int m = m0; m < m0 + kPer; ++m) {
        if (m == m0)
          mma16816_zero(d, fa[2 * m], fb[2 * m], fa[2 * m + 1], fb[2 * m + 1], xb[2 * m], xb[2 * m + 1]);
        else
          mma16816(d, fa[2 * m], fb[2 * m], fa[2 * m + 1], fb[2 * m + 1], xb[2 * m], xb[2 * m + 1]);
      }
      const uint32_t wg = F == Fmt::NF4 ? sg : m0 ? sg & 0xFFFF0000u : sg << 16;
      const uint32_t wh = F == Fmt::NF4 ? sh : m0 ? sh & 0xFFFF0000u : sh << 16;
      acc[0] = fmaf(d[0], __uint_as_float(wg), acc[0]);
      acc[1] = fmaf(d[1], __uint_as_float(wg), acc[1]);
      acc[2] = fmaf(d[2], __uint_as_float(wh), acc[2]);
      acc[3] = fmaf(d[3], __uint_as_float(wh), acc[3]);
    }
  };

  // Waits for the chunk to multiply; its stage's offset in the ring.
  auto wait_stage = [&]() __attribute__((always_inline)) -> uint32_t {
    cp_async_wait_group<D - 1>();
    __syncwarp();
    const uint32_t slot = q_out;
    q_out = (q_out + 1) & (D - 1);
    return slot;
  };
  // One column tile, the `nb` blocks of one chunk: x holds the columns of its
  // first two blocks; at the end those at nsrc, the next ones the warp needs.
  auto step_one = [&](uint4 (&x)[2][2], const uint16_t* src, int nb, const uint16_t* nsrc, int nnb,
                      float (&acc)[4]) __attribute__((always_inline)) {
    issue();
    uint4 y[2][2];
    auto load_cols = [&](uint4 (&v)[2][2], const uint16_t* from, int n) __attribute__((always_inline)) {
      if (n > 0) load_x(from, v[0][0], v[0][1]);
      if (n > 1) load_x(from + 64, v[1][0], v[1][1]);
    };
    load_cols(y, src + 128, nb - 2);
    const uint32_t slot = wait_stage();
    const uint32_t st = get_w + slot * kStage;
    const uint4 s0 = *reinterpret_cast<const uint4*>(smem + get_s + slot * kScStage);
    const uint4 s1 = *reinterpret_cast<const uint4*>(smem + get_s + slot * kScStage + 8 * 16);
    auto block = [&](int b, const uint4 (&v)[2], uint32_t sg, uint32_t sh) __attribute__((always_inline)) {
      uint32_t fa[8], fb[8];
      decode(st, b, fa, fb);
      mma_block(acc, fa, fb, v[0], v[1], sg, sh);
    };
    if (nb >= 4) {
      block(0, x[0], s0.x, s1.x);
      block(1, x[1], s0.y, s1.y);
      load_cols(x, nsrc, nnb);
      block(2, y[0], s0.z, s1.z);
      block(3, y[1], s0.w, s1.w);
    } else {
      block(0, x[0], s0.x, s1.x);
      if (nb > 1) block(1, x[1], s0.y, s1.y);
      load_cols(x, nsrc, nnb);
      if (nb > 2) block(2, y[0], s0.z, s1.z);
    }
    __syncwarp();
  };
  // Phase B, two column tiles: the columns are loaded a block ahead.
  auto step_two = [&](uint4 (&x)[2][2][2], const uint16_t* s0, const uint16_t* s1, int left,
                      float (&acc)[2][4]) __attribute__((always_inline)) {
    issue();
    const uint32_t slot = wait_stage();
    const uint32_t st = get_w + slot * kStage;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (b < left) {
        if (b + 1 < left) {
          load_x(s0 + b * 64 + 64, x[(b + 1) & 1][0][0], x[(b + 1) & 1][0][1]);
          load_x(s1 + b * 64 + 64, x[(b + 1) & 1][1][0], x[(b + 1) & 1][1][1]);
        }
        const uint32_t sg = *reinterpret_cast<const uint32_t*>(smem + get_s + slot * kScStage + b * 4);
        const uint32_t sh = *reinterpret_cast<const uint32_t*>(smem + get_s + slot * kScStage + 128 + b * 4);
        uint32_t fa[8], fb[8];
        decode(st, b, fa, fb);
        mma_block(acc[0], fa, fb, x[b & 1][0][0], x[b & 1][0][1], sg, sh);
        mma_block(acc[1], fa, fb, x[b & 1][1][0], x[b & 1][1][1], sg, sh);
      }
    }
    __syncwarp();
  };

  // Writes one column tile of a finished unit: h (phase A) or y (phase B).
  auto finish = [&](int phase, const float (&d)[4], int cnt, int r0, int tile, int nt) __attribute__((always_inline)) {
    if (phase == 0) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = nt * 8 + 2 * t4 + j;
        if (c < cnt) {
          const int slot = rows[r0 + c];
          const float h = __fdiv_rn(d[j], 1.0f + expf(-d[j])) * d[2 + j];
          const __nv_bfloat16 hi = __float2bfloat16_rn(h);
          // an infinite high part keeps a zero low part (inf - inf is NaN)
          const float low = h - __bfloat162float(hi);
          const __nv_bfloat16 lo = __float2bfloat16_rn(isfinite(low) ? low : 0.0f);
          a.hhi[(int64_t)slot * I + tile * 8 + g] = __bfloat16_as_ushort(hi);
          a.hlo[(int64_t)slot * I + tile * 8 + g] = __bfloat16_as_ushort(lo);
        }
      }
    } else {
      // high and low parts of a row: columns c and c + 4, lanes t4 and t4 + 2
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = d[j] + __shfl_xor_sync(0xffffffffu, d[j], 2);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = nt * 4 + 2 * t4 + j;
        if (t4 < 2 && c < cnt) {
          float* y = a.y + (int64_t)rows[r0 + c] * H + tile * 16 + g;
          y[0] = v[j];
          y[8] = v[2 + j];
        }
      }
    }
  };

  float* parts = reinterpret_cast<float*>(smem + Smem::table + 128);  // row i at i * 64
  // A share: this warp's range of chunks, then the units that several warps
  // shared, joined in order.
  auto run_share = [&](const Share& s) __attribute__((always_inline)) {
    const int nc = s.nc, K = s.phase ? I : H, nbk = K >> 6;  // blocks of a unit
    const bool wide = s.phase && two_tiles;
    const int rows4 = wide ? 8 : 4;                          // part rows of a piece
    int f = s.begin(warp);
    const int f1 = s.begin(warp + 1);
    if (f < f1) {
      const int u0 = f / nc;
      int u = u0, c = f - u0 * nc, ai, tile;
      unit_of(s.phase, s.u0 + u, ai, tile);
      int r0 = first[ai], cnt = first[ai + 1] - r0;
      const uint16_t* src = column(s.phase, r0, cnt, 0) + c * 256;
      uint4 x[2][2];
      if (!wide) {
        load_x(src, x[0][0], x[0][1]);
        if (nbk - c * 4 > 1) load_x(src + 64, x[1][0], x[1][1]);
      }
#pragma unroll 1
      for (;;) {
        // the piece: chunks [c, c1) of unit u; then the next unit's first
        const int c1 = min(nc, c + f1 - f);
        const bool more = f + (c1 - c) < f1;
        int nai = ai, ntile = tile;
        if (more) next_unit(s.phase, nai, ntile);
        const int nr0 = first[nai], ncnt = first[nai + 1] - nr0;
        const uint16_t* nsrc = column(s.phase, nr0, ncnt, 0);
        float acc[2][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[0][j] = acc[1][j] = 0.0f;
        const bool whole = c == 0 && c1 == nc;
        f += c1 - c;
        if (!wide) {
#pragma unroll 1
          for (; c < c1; ++c, src += 256) {
            const bool last = c + 1 == c1;
            step_one(x, src, nbk - c * 4, last ? nsrc : src + 256, last ? nbk : nbk - c * 4 - 4, acc[0]);
          }
        } else {
          const uint16_t* src1 = column(1, r0, cnt, cnt > 4 ? 1 : 0) + c * 256;
          uint4 y[2][2][2];
          load_x(src, y[0][0][0], y[0][0][1]);
          load_x(src1, y[0][1][0], y[0][1][1]);
#pragma unroll 1
          for (; c < c1; ++c, src += 256, src1 += 256)
            step_two(y, src, src1, c + 1 < c1 ? nbk - c * 4 : min(4, nbk - c * 4), acc);
        }
        if (whole) {
          finish(s.phase, acc[0], cnt, r0, tile, 0);
          if (wide && cnt > 4) finish(1, acc[1], cnt, r0, tile, 1);
        } else {
          // a warp's first piece in its first slot, its last in the second
          float* to = parts + ((warp * 2 + (u != u0)) * rows4) * 64 + lane;
#pragma unroll
          for (int j = 0; j < 4; ++j) to[j * 64] = acc[0][j];
          if (wide)
#pragma unroll
            for (int j = 0; j < 4; ++j) to[(4 + j) * 64] = acc[1][j];
        }
        if (!more) break;
        ++u;
        ai = nai;
        tile = ntile;
        r0 = nr0;
        cnt = ncnt;
        src = nsrc;
        c = 0;
      }
    }
    __syncthreads();
    // units cut by a warp's border: warp w joins the one that begins in its
    // range and goes on behind it
    const int e = s.begin(warp + 1);
    if (s.begin(warp) < e && e % nc) {
      const int u = e / nc;
      if (u * nc >= s.begin(warp)) {
        int ai, tile;
        unit_of(s.phase, s.u0 + u, ai, tile);
        const int r0 = first[ai], cnt = first[ai + 1] - r0;
        for (int i = 0; i < (wide && cnt > 4 ? 2 : 1); ++i) {
          float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          for (int w = warp; w < kWarps && s.begin(w) < (u + 1) * nc; ++w) {
            if (s.begin(w) == s.begin(w + 1)) continue;
            const float* from = parts + ((w * 2 + (s.begin(w) / nc != u)) * rows4 + i * 4) * 64 + lane;
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j] += from[j * 64];
          }
          finish(s.phase, d, cnt, r0, tile, i);
        }
      }
    }
  };

  // Waits until every share of phase A is done.
  auto wait_a = [&]() __attribute__((always_inline)) {
    if (threadIdx.x == 0) {
      const uint64_t t0 = globaltimer_ns();
      while (ld_acquire(&a.counters[2]) < G) {
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
          misc[3] = 1;
          raise_error(p.err, GBW_DEVERR_TIMEOUT);
          break;
        }
      }
      __threadfence();
    }
    __syncthreads();
  };
  // Combines the slots of output tile `tile` in slot order.
  auto combine = [&](int tile) __attribute__((always_inline)) {
    for (int i = threadIdx.x; i < T * 16; i += kThreads) {
      const int t = i >> 4, n = tile * 16 + (i & 15);
      float v = 0.0f;
      for (int s = 0; s < k; ++s) {
        const float w = wts[t * k + s];
        if (w != 0.0f) v = fmaf(w, __ldcg(a.y + (int64_t)(t * k + s) * H + n), v);
      }
      p.out[(int64_t)t * H + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
  };

  bool in_a = next_a < G, fresh = true, waited = in_a;
#pragma unroll 1
  for (;;) {
    if (fresh) {
      fresh = false;
      enter(sa);
#pragma unroll 1
      for (int i = 0; i < D - 1; ++i) issue();
    }
    if (!waited) {
      waited = true;
      wait_a();
    }
    if (!in_a && (next_b >= G || misc[3])) break;
    const Share cur = in_a ? sa : sb;
    run_share(cur);
    if (threadIdx.x == 0) misc[2] = atomicAdd(&a.counters[in_a ? 0 : 1], 1);
    if (in_a || !aligned) __threadfence();
    __syncthreads();
    const int next = misc[2];
    if (in_a) {
      if (threadIdx.x == 0) atomicAdd(&a.counters[2], 1);
    } else if (cur.n > 0) {
      // tiles that this share touches: an aligned share holds all of a tile's
      // experts; else the CTA that brings the tile's count to A combines it
      const int last_tile = (cur.u0 + cur.n - 1) / A;
      for (int tile = cur.u0 / A; tile <= last_tile; ++tile) {
        if (aligned) {
          combine(tile);
        } else {
          if (threadIdx.x == 0) {
            const int mine = min(cur.u0 + cur.n, (tile + 1) * A) - max(cur.u0, tile * A);
            misc[5] = atomicAdd(&a.counters[kCounters + tile], mine) + mine == A;
            __threadfence();
          }
          __syncthreads();
          if (misc[5]) combine(tile);
          __syncthreads();
        }
      }
    }
    if (next < G) {
      // another share of this phase is unclaimed (some CTAs have not started):
      // drop what is in flight and start the stream again
      cp_async_wait_group<0>();
      __syncthreads();  // before misc[2], the rings and the part rows are written again
      if (in_a) {
        sa = make_share(0, next);
      } else {
        sa.n = 0;  // (enter: no chunks of share A)
        sb = make_share(1, next);
      }
      q_in = q_out = sv_to = 0;
      fresh = true;
    } else if (in_a) {
      in_a = waited = false;
    } else {
      break;
    }
  }
  cp_async_wait_group<0>();
}

struct Layout {
  int64_t logits, hhi, hlo, y, counters, total;
};

Layout layout_of(int64_t T, int32_t E, int32_t k, int64_t H, int64_t I) {
  auto up = [](int64_t b) { return (b + 255) & ~(int64_t)255; };
  Layout l;
  const int64_t P = T * k;
  l.logits = 0;
  l.hhi = up(T * E * 4);
  l.hlo = l.hhi + up(P * I * 2);
  l.y = l.hlo + up(P * I * 2);
  l.counters = l.y + up(P * H * 4);
  l.total = l.counters + up((kCounters + H / 16) * 4);
  return l;
}

template <Fmt F, int NPL>
cudaError_t launch_t(const LayerArgs& a, int num_sms, cudaStream_t s) {
  constexpr auto k = moe_experts<F, NPL>;
  cudaError_t e = opt_in_smem<k>(Smem::end);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.p.E, (unsigned)((a.p.T + kRouterTokens - 1) / kRouterTokens));
  cfg.blockDim = dim3((unsigned)std::min<int64_t>(kRouterThreads, (a.p.H / 8 + 31) / 32 * 32));
  cfg.stream = s;
  e = cudaLaunchKernelEx(&cfg, moe_router, a);
  if (e != cudaSuccess) return e;
  // Whole tiles of H per CTA in phase B spare the counting of a tile's experts
  // across CTAs (about 1.5 us) but leave the last round of tiles uneven: taken
  // when that costs at most kAlignChunks chunks of 2 KB per CTA (about 46 ns
  // each at the measured HBM rate).
  constexpr int64_t kAlignChunks = 32;
  const int64_t tiles = a.p.H / 16, A = std::min<int64_t>(a.p.E, a.p.T * a.p.k);
  const int64_t whole = (tiles + num_sms - 1) / num_sms * A;
  const int64_t even = (tiles * A + num_sms - 1) / num_sms;
  const int aligned = (whole - even) * ((a.p.I + 255) / 256) <= kAlignChunks;
  return launch_kernel<k>(num_sms, kThreads, Smem::end, s, true, a, aligned);
}

template <Fmt F>
cudaError_t launch_f(const LayerArgs& a, int num_sms, cudaStream_t s) {
  return a.p.E <= 128 ? launch_t<F, 4>(a, num_sms, s) : launch_t<F, kMaxE / 32>(a, num_sms, s);
}

}  // namespace

int64_t layer_workspace(int64_t T, int32_t E, int32_t k, int64_t H, int64_t I) {
  return layout_of(T, E, k, H, I).total;
}

cudaError_t launch_layer(Fmt f, const LayerProblem& p, void* workspace, int num_sms,
                         cudaStream_t s) {
  if (p.T == 0) return cudaSuccess;
  const Layout l = layout_of(p.T, p.E, p.k, p.H, p.I);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  const LayerArgs a{p,
                    reinterpret_cast<float*>(w + l.logits),
                    reinterpret_cast<uint16_t*>(w + l.hhi),
                    reinterpret_cast<uint16_t*>(w + l.hlo),
                    reinterpret_cast<float*>(w + l.y),
                    reinterpret_cast<int*>(w + l.counters)};
  return f == Fmt::NF4 ? launch_f<Fmt::NF4>(a, num_sms, s) : launch_f<Fmt::MXFP4>(a, num_sms, s);
}

}  // namespace gbw
