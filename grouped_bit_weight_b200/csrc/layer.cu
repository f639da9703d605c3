// layer.cu -- a whole mixture-of-experts layer for a few tokens (T <= 32) on NF4
// or MXFP4 expert weights.
//
//   l[t, e] = sum_k x[t, k] Wr[e, k] (+ b[e]); ids, w = the k largest and their
//   softmax weights (route.cuh); per slot (t, s) with e = ids[t, s]:
//     h = silu(x Wg_e^T) * (x Wu_e^T),  y = h Wd_e^T;   out[t] = sum_s w y
//
// Bound: the active experts' packed bytes from HBM.  Two ways:
//
// (1) NF4, and MXFP4 on few weights (takes_pieces): two launches.  Kernel 1
// (moe_router): the router logits, one CTA per expert and 8 tokens, fp32; it also
// zeroes kernel 2's counters.  Kernel 2 (moe_experts), one CTA per SM, launched
// early behind kernel 1 (programmatic dependent launch: its codebook table is
// built meanwhile):
//   every CTA chooses the experts itself from the logits (no third kernel) and
//   cuts each expert's rows into groups of at most 8;
//   phase A  gate_up + SwiGLU in units of (group, 16 gate rows + the matching
//            16 up rows), h written as bf16 high and low parts;
//   phase B  down in units of (32 rows, group), y in fp32; the CTA that
//            finishes a tile's last group combines the tile's slots in slot
//            order (no sum depends on the order of arrival).
//   Between the phases a CTA waits until all of phase A is done.  Shares of
//   both phases are claimed from counters, and a CTA waits only once no share
//   of phase A is unclaimed, so every share waited for is held by a running
//   CTA: the wait ends whether or not all CTAs are resident at a time, also
//   with other kernels on the device.
// A loading warp fills a ring of two 4 KB stages (32 weight rows x 256 k, one TMA
// box) for each of 11 multiplying warps -- across the wait between the phases
// too: the next phase's weights do not depend on it.  A packed byte becomes two
// bf16 values by one conflict-free table lookup and goes straight into mma.sync
// m16n8k16 as the A operand (weights are M, tokens N; from a register operand a
// decoded weight needs no way through shared memory), one scale block at a time;
// block sums are scaled in fp32.  The low part of h keeps the down projection's
// input at 16 bits of mantissa, at one more column and no conversion.  A unit's K
// is split over several warps (joined through shared memory in a fixed order)
// when a CTA has fewer units than warps.
// What bounds it is the latency of lookups and x loads at 11 warps an SM (168
// registers a thread; 15 warps spill and took 58 instead of 55 us for 8 tokens): over the
// whole NF4 8-token kernel the shared-memory pipe is 44 % busy, issue 37 %, DRAM
// 31 %.  With the lookups left out the MXFP4 32-token case fell from 165 to 137
// us, with the loads of x 127, with the weight loads hardly.  Hidden 2880, 32
// experts, MXFP4, 1 token: 35 us (1.5 TB/s); hidden 2048, 128 experts, 8 chosen,
// NF4, 1 / 8 / 32 tokens: 22 / 54 / 104 us (0.97 / 2.5 / 2.9 TB/s).
//
// (2) MXFP4 on more weights: no lookups and no mma.sync, the
// packed weights go to tcgen05 as they are.  x and h become rows of sixteen 4-bit
// pieces (a4.cu: 32 bits of each 32-block's maximum) and the block-scaled 4-bit
// product sums a row's pieces in fp32: logits, routing, pieces of x, gate_up,
// SwiGLU + pieces of h, down, combine, seven launches behind one another.  32
// tokens: 99 us (4.2 TB/s) against 154 of (1).
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "launch.cuh"
#include "route.cuh"
#include "swiglu.cuh"

namespace gbw {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn get_encode_fn();

namespace {

constexpr int kWarps = 11;                 // that multiply; one more loads
constexpr int kConsumers = 32 * kWarps;
constexpr int kThreads = kConsumers + 32;
constexpr int kMaxE = 1024;
constexpr int kMaxP = 512;
constexpr int kRows = 8;           // most rows of a group: rows of one expert that share a decode
constexpr int CKB = 128;           // bytes per weight row and stage: 256 k
constexpr int D = 2;               // stages per warp (3: 58 instead of 57 us for NF4, 8 tokens)
constexpr int kStage = 32 * CKB;   // 4 KB: 32 weight rows

// Shared memory by address in the shared window (dynamic shared memory starts
// at 1 KB).  The table lies at 64 KB: entry b of lane l at 65536 + b * 256 +
// l * 4, so that one byte permute of a packed word gives the whole address.
// The other half of each 256 bytes holds partial sums (kParts rows of 32
// floats).  The warps' rings lie on both sides of it.
constexpr int kParts = 256;
constexpr int kLowWarps = 7;
struct Smem {
  static constexpr int base = 1024;
  static constexpr int ids = base;               // [kMaxP] int
  static constexpr int wts = ids + 4 * kMaxP;    // [kMaxP] float
  static constexpr int rows = wts + 4 * kMaxP;   // [kMaxP] uint16 slot of sorted row
  static constexpr int active = rows + 2 * kMaxP;  // [kMaxP] uint16 expert
  static constexpr int misc = active + 2 * kMaxP;  // 16 ints
  static constexpr int shares = misc + 64;         // [4] Share, 32 bytes apart
  static constexpr int bars = shares + 128;        // full and empty [kWarps][2][D], published [2]
  static constexpr int low_end = bars + 8 * (2 * kWarps * D + 2);
  static constexpr int table = 65536;
  static constexpr int ring_low = table - kLowWarps * D * kStage;
  static constexpr int count = ring_low;  // [kMaxE] int: token bits, then first row (before the ring is used)
  static constexpr int ring_high = 2 * table;
  static constexpr int first = ring_high + (kWarps - kLowWarps) * D * kStage;  // [kMaxP + 4] int first sorted row
  static constexpr int e8m0 = first + 4 * (kMaxP + 4);  // [256] float (MXFP4)
  static constexpr int part = e8m0 + 1024;              // [kWarps + 1] scan parts
  static constexpr int end = part + 64;
  static constexpr int bytes = end - base;  // dynamic
};
static_assert(Smem::low_end <= Smem::ring_low, "the small arrays fit below the rings");
static_assert(Smem::ring_low + 4 * kMaxE <= Smem::table, "the expert counts fit the rings below");
static_assert(Smem::bytes <= 232448, "shared memory exceeds the 227 KB a CTA can have");

struct LayerArgs {
  LayerProblem p;
  float* logits;      // [T, E]
  uint16_t* hhi;      // [P, I] bf16
  uint16_t* hlo;      // [P, I] bf16
  float* y;           // [P, H]
  int* counters;      // claimA, claimB, doneA, then one per 16 columns of H; or null
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
  if (a.counters && blockIdx.x == 0 && blockIdx.y == 0)
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
    // all loads before the first use
    uint4 xv[kRouterTokens];
#pragma unroll
    for (int j = 0; j < kRouterTokens; ++j)
      xv[j] = __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)(t0 + min(j, n - 1)) * p.H) + u);
#pragma unroll
    for (int j = 0; j < kRouterTokens; ++j) {
      const uint32_t xx[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[j] = fmaf(__uint_as_float(wx[i] << 16), __uint_as_float(xx[i] << 16), acc[j]);
        acc[j] = fmaf(__uint_as_float(wx[i] & 0xFFFF0000u), __uint_as_float(xx[i] & 0xFFFF0000u),
                      acc[j]);
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

// The NF4 levels enter the table times this, rounded to bf16, and the sums are
// divided by it: of the factors in [1, 2) it is the one whose products with the 16
// levels round with the least error, 6.3e-4 of their root mean square (1.1e-3
// without it, as in the other NF4 calls, which round the level or the decoded
// weight to bf16).  Levels 9 and 11 are rounded down instead, which makes 7.5e-4 of
// it but takes the levels' mean error from 2.6e-4 to 9e-6: a mean error meets the
// sum of a row's x, so that with x = 1 + N(0, 1) the output was off by 1.5e-2 of its
// norm (now 1.8e-3).  With x = N(0, 1) it is off by 2.1e-3, 1.65e-3 of that its own
// rounding to bf16.  Levels of full precision leave 1.65e-3 and cost time:
// 2048 x 768, 1 / 8 / 32 tokens take 22 / 54 / 104 us as it is, 27 / 71 / 142 with
// levels of a high and a low bf16 part (twice the lookups' bytes and mmas), 24 / 57
// / 113 with fp16 levels (x and h scaled into fp16's range by powers of two, more
// registers than there are).
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
  const bool down = F == Fmt::NF4 && (q == 9 || q == 11);
  return __bfloat16_as_ushort(down ? __float2bfloat16_rd(v) : __float2bfloat16_rn(v));
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

// Whether the phase with `parity` has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
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
__device__ __forceinline__ int ld_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// 32 rows x 128 bytes of a packed matrix to shared address dst, 128B swizzle
// (16-byte unit u of row r at u ^ (r & 7)), counted in bytes on barrier `bar`.
// One box per stage: issuing a box takes about 130 cycles whatever its size (two
// boxes of 1 KB per stage bound the whole kernel).
__device__ __forceinline__ void tma_box3(uint32_t dst, const CUtensorMap* m, int x, int y, int z,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// A share of one phase: units [u0, u0 + n) of nc chunks (256 k) each.  Warp w
// takes whole units w, w + kWarps, .. of the first `whole` (a multiple of kWarps)
// and parts of the others, which are cut into 1 << lgS parts each and joined
// through shared memory.
struct Share {
  int phase;  // 0: gate_up, 1: down, 2: no more
  int u0, n, nc, whole, lgS;
  // Item `i` of warp w: chunks [c, c1) of unit u; false past the last.
  __device__ __forceinline__ bool item(int w, int i, int& u, int& c, int& c1) const {
    u = w + i * kWarps;
    c = 0;
    c1 = nc;
    if (u < whole) return true;
    const int l = lgS, j = u - whole, sp = j & ((1 << l) - 1);
    u = whole + (j >> l);
    c = (sp * nc) >> l;
    c1 = ((sp + 1) * nc) >> l;
    return u < n;
  }
};

// Barrier of the multiplying warps.
__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
}
// The same; whether any of them says `v` (they leave together after a wait that
// ran out).
__device__ __forceinline__ bool consumer_any(bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n bar.red.or.pred q, 1, %1, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "n"(kConsumers), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

template <Fmt F, int NPL>
__global__ void __launch_bounds__(kThreads, 1) moe_experts(const LayerArgs a, const int aligned,
                                                            const __grid_constant__ CUtensorMap map_gu,
                                                            const __grid_constant__ CUtensorMap map_dn) {
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
  if (smem_u32(smem_raw) != Smem::base) {  // (the layout above takes 1 KB as given)
    raise_error(p.err, GBW_DEVERR_TIMEOUT);
    return;
  }
  // misc: 0 claim A, 1 claim B, 2 shares begun, 3 abort, 4 groups, 5 last of a
  // tile, 6 rows of the largest expert
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Smem::bars);
  uint64_t* published = bars + 2 * kWarps * D;  // [2] share 0, 2, .. and 1, 3, .. is known

  {
    // a warp writes the 16 bytes of one high nibble: lane l holds level l & 15
    const uint32_t level = code_bf16<F>(lane & 15);
#pragma unroll 1
    for (int h = warp; h < 16; h += kWarps + 1) {
      const uint32_t top = __shfl_sync(0xffffffffu, level, h);
#pragma unroll
      for (int l = 0; l < 16; ++l) {
        const uint32_t low = __shfl_sync(0xffffffffu, level, l);
        sts32(Smem::table + (h * 16 + l) * 256 + lane * 4,
              F == Fmt::NF4 ? top | (low << 16) : low | (top << 16));
      }
    }
    if (F == Fmt::MXFP4)
      for (int i = threadIdx.x; i < 256; i += kThreads)
        sts32(Smem::e8m0 + 4 * i, i == 0 ? 0x00400000u : i == 255 ? 0x7FC00000u : (uint32_t)i << 23);
  }
  for (int e = threadIdx.x; e < E; e += kThreads) count[e] = 0;
  if (threadIdx.x == 0) {
    misc[2] = misc[3] = misc[6] = 0;
    tma_prefetch_desc(&map_gu);
    tma_prefetch_desc(&map_dn);
  }
  for (int i = threadIdx.x; i < 2 * kWarps * D + 2; i += kThreads) mbar_init(bars + i, 1);
  fence_barrier_init();
  __syncthreads();
  grid_dependency_wait();
  if (threadIdx.x >= kThreads - 2) {  // (a warp without a token, usually)
    const int i = threadIdx.x - (kThreads - 2);
    misc[i] = atomicAdd(&a.counters[i], 1);
  }

  // ---- the choice of experts, the same in every CTA
  for (int t = warp; t < T; t += kWarps + 1) {
    int id = 0;
    float w = 0.0f;
    choose<float, NPL, true>(a.logits + (int64_t)t * E, E, k, p.renorm, lane, id, w);
    if (lane < k) {
      ids[t * k + lane] = id;
      wts[t * k + lane] = w;
      atomicOr(&count[id], (int)(1u << t));
    }
  }
  __syncthreads();
  // rows sorted by expert and cut into groups of at most kRows rows of one
  // expert: a packed scan (rows below, groups below) over three experts per
  // thread.  count[e] holds the tokens of expert e as bits (T <= 32), so a
  // slot's place among its expert's rows is the number of lower bits: the same
  // in every CTA, as it must be for the groups to hold the same rows everywhere.
  {
    constexpr int kPer = 3;
    static_assert(kPer * kThreads >= kMaxE && 2 * kThreads >= kMaxP, "one round each");
    const int e0 = threadIdx.x * kPer;
    int c[kPer], sum = 0, top = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      c[j] = e0 + j < E ? __popc(count[e0 + j]) : 0;
      sum += c[j] | (((c[j] + kRows - 1) / kRows) << 16);
      top = max(top, c[j]);
    }
    int at[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int slot = threadIdx.x + j * kThreads;
      at[j] = slot < P ? __popc((unsigned)count[ids[slot]] & ((1u << (slot / k)) - 1u)) : 0;
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int s = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += s;
    }
    if (lane == 31) part[warp] = incl;
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) atomicMax(const_cast<int*>(&misc[6]), top);
    __syncthreads();
    int below = incl - sum;
    for (int i = 0; i < warp; ++i) below += part[i];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int r = below & 0xFFFF, n = (c[j] + kRows - 1) / kRows;
      for (int i = 0; i < n; ++i) {
        active[(below >> 16) + i] = (uint16_t)(e0 + j);
        first[(below >> 16) + i] = r + i * kRows;
      }
      if (e0 + j < E) count[e0 + j] = r;
      below += c[j] | (n << 16);
    }
    if (threadIdx.x == kThreads - 1) {
      misc[4] = below >> 16;
      first[below >> 16] = P;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int slot = threadIdx.x + j * kThreads;
      if (slot < P) rows[count[ids[slot]] + at[j]] = (uint16_t)slot;
    }
  }
  __syncthreads();
  const int A = misc[4];  // groups
  const int G = gridDim.x;
  const int tiles_a = I / 16, tiles_b = H / 32;

  // Column tiles of 8: phase A, up to 8 rows of a group are one tile; phase B,
  // 4 rows a tile, the high parts of h in columns 0..3, the low ones in 4..7.
  const bool two_tiles = misc[6] > 4;  // some group has more than 4 rows
  // The CTA's shares in order, in shared memory, four at a time.
  auto share = [&](int i) __attribute__((always_inline)) -> Share* {
    return reinterpret_cast<Share*>(smem + Smem::shares + (i & 3) * 32);
  };
  // (group, output tile) of unit u
  auto unit_of = [&](int phase, int u, int& ai, int& tile) __attribute__((always_inline)) {
    const int d = phase ? A : tiles_a, q = u / d, r = u - q * d;
    ai = phase ? r : q;
    tile = phase ? q : r;
  };
  // A unit has 32 weight rows.  gate_up: 16 gate rows, then the 16 up rows of the
  // same columns, I further; down: 32 rows in order.
  auto first_row = [&](int phase, int ai, int tile) __attribute__((always_inline)) -> int {
    const int e = active[ai];
    return phase ? e * H + tile * 32 : e * 2 * I + tile * 16;
  };

  if (warp == kWarps) {
    // ---------------- loads: lane l feeds warp l's ring ----------------
    const uint32_t ring = lane < kLowWarps ? Smem::ring_low + lane * (D * kStage)
                                           : Smem::ring_high + (lane - kLowWarps) * (D * kStage);
    uint64_t* full = bars + 2 * D * min(lane, kWarps - 1);
    uint64_t* empty = full + D;
    int known = 0;         // shares published
    int kind = -1;         // phase of the last one; 2: no more
    bool ended = lane >= kWarps;
    int mine = -1;         // share this lane is at, its item and chunk
    int item = 0, c = 0, c1 = 0;
    int y = 0, z = 0;      // its box: row, and matrix (gate_up: [2 E] of I rows; down: one)
    const CUtensorMap* map = nullptr;
    bool busy = false;     // a chunk is waiting to be loaded
    uint32_t q = 0, slot = 0, ph = 1;  // chunks loaded, next slot, its empty phase
    uint32_t idle = 0;
    uint64_t since = 0;
    auto open = [&]() __attribute__((always_inline)) {
      const Share& s = *share(mine);
      int u, ai, tile;
      busy = s.item(lane, item, u, c, c1);
      if (busy) {
        unit_of(s.phase, s.u0 + u, ai, tile);
        const int e = active[ai];
        y = s.phase ? e * H + tile * 32 : tile * 16;
        z = s.phase ? 0 : 2 * e;
        map = s.phase ? &map_dn : &map_gu;
      }
    };
    for (;;) {
      // a lane has loaded its last share, and the others have begun that one:
      // claim the next (all of phase A before any of phase B).  Every lane votes,
      // whatever it reads of the others' progress.
      const bool next_due = misc[2] >= known && !ended && !busy && mine + 1 == known;
      if (kind != 2 && __any_sync(0xffffffffu, next_due)) {
        int idx = 0;
        if (kind < 0) {
          kind = 0;
          idx = misc[0];
        } else if (kind == 0) {
          if (lane == 0) idx = atomicAdd(&a.counters[0], 1);
          idx = __shfl_sync(0xffffffffu, idx, 0);
        } else {
          if (lane == 0) idx = atomicAdd(&a.counters[1], 1);
          idx = __shfl_sync(0xffffffffu, idx, 0);
        }
        if (kind == 0 && idx >= G) {
          kind = 1;
          idx = misc[1];
        }
        if (idx >= G) kind = 2;
        if (lane == 0) {
          Share* s = share(known);
          s->phase = kind;
          s->n = 0;
          if (kind < 2) {
            const int tiles = kind ? tiles_b : tiles_a;
            // phase B, aligned: whole tiles, so that no tile is shared between CTAs
            const int per = kind && aligned ? A : 1;
            const unsigned total = (unsigned)(per > 1 ? tiles : tiles * A);
            const unsigned each = total / (unsigned)G, r = total - each * (unsigned)G;
            const int n = (int)(each + (idx < (int)r)) * per, nc = ((kind ? I : H) + 255) >> 8;
            // the split of the last units with the least work for the busiest
            // warp, as far as the partial sums fit (8 rows for each column tile)
            const int whole = n - n % kWarps;
            const int rest = n - whole, rows4 = kind && two_tiles ? 16 : 8;
            int lgS = 0, best = rest ? 8 : 0;  // eighths of a unit
            for (int l = 1; l <= 3; ++l) {
              if ((1 << l) <= nc && (rest << l) * rows4 <= kParts) {
                const int cost = (((rest << l) + kWarps - 1) / kWarps) << (3 - l);
                if (cost < best) { best = cost; lgS = l; }
              }
            }
            s->u0 = (int)(each * idx + min((unsigned)idx, r)) * per;
            s->n = n;
            s->nc = nc;
            s->whole = whole;
            s->lgS = lgS;
          }
          mbar_arrive(&published[known & 1]);
        }
        ++known;
        __syncwarp();
      }
      if (!ended && !busy && mine + 1 < known) {
        ++mine;
        item = 0;
        if (share(mine)->phase == 2) ended = true;
        else open();
      }
      if (__all_sync(0xffffffffu, ended)) break;
      bool went = false;
      if (busy) {
        if (mbar_test(&empty[slot], ph)) {
          mbar_arrive_expect_tx(&full[slot], kStage);
          tma_box3(ring + slot * kStage, map, c * CKB, y, z, smem_u32(&full[slot]));
          ++q;
          if (++slot == D) { slot = 0; ph ^= 1u; }
          went = true;
          if (++c == c1) {
            ++item;
            open();
          }
        }
      }
      if (__any_sync(0xffffffffu, went)) {
        idle = 0;
        since = 0;
      } else if ((++idle & 1023u) == 0) {
        if (misc[3]) break;
        if (!since) since = globaltimer_ns();
        if (globaltimer_ns() - since > kWaitLimitNs) {
          misc[3] = 1;
          raise_error(p.err, GBW_DEVERR_TIMEOUT);
          break;
        }
      }
    }
    if (misc[3] && lane < kWarps)  // let the loads in flight land
      for (uint32_t i = q > D ? q - D : 0; i < q; ++i) mbar_drain(&full[i % D], (i / D) & 1u);
    return;
  }

  // ---------------- the multiplying warps ----------------
  const int g = lane >> 2, t4 = lane & 3;
  const uint32_t lut = Smem::table | (uint32_t)lane * 4u;
  const uint32_t ring = warp < kLowWarps ? Smem::ring_low + warp * (D * kStage)
                                         : Smem::ring_high + (warp - kLowWarps) * (D * kStage);
  uint64_t* full = bars + 2 * D * warp;
  uint64_t* empty = full + D;
  uint32_t slot = 0, ph = 0;  // of the next chunk to multiply

  constexpr int kSecond = F == Fmt::NF4 ? 8 : 32;        // distance of a lane's second 8 k
  constexpr int kScChunk = F == Fmt::NF4 ? 16 : 8;       // scale bytes of a row and chunk

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
  // Weight fragments of block b of one of a stage's two halves of 16 rows: the
  // lane's 16 weights of mma rows g and g + 8.  gate_up: gate rows 8 m + pg with
  // the up rows of the same columns 16 rows further; down: rows 16 m + pg and 8
  // further.  NF4, one scale block: bytes 8 t4 .. of its 32; MXFP4, two blocks of
  // 16 bytes: 4 bytes of each, so that every mma stays inside a scale block.
  // `st` is this lane's address in block 0; the blocks differ in address bits 5
  // and 6 alone.  Mma row g is row pg of eight: with that order the swizzle
  // spreads every access over all banks.
  const int pg = F == Fmt::NF4 ? (g & 3) * 2 + (g >> 2) : g;
  const uint32_t get_w = ring + pg * CKB + (F == Fmt::NF4 ? ((t4 >> 1) ^ pg) * 16 + (t4 & 1) * 8
                                                          : pg * 16 + t4 * 4);
  auto decode = [&](uint32_t st, int b, int far, uint32_t (&fa)[8], uint32_t (&fb)[8]) __attribute__((always_inline)) {
    uint2 wa, wb;
    const uint8_t* at = smem + (st ^ (b * 32));
    if (F == Fmt::NF4) {
      wa = *reinterpret_cast<const uint2*>(at);
      wb = *reinterpret_cast<const uint2*>(at + far);
    } else {
      const uint8_t* au = smem + (st ^ (b * 32 + 16));
      wa.x = *reinterpret_cast<const uint32_t*>(at);
      wa.y = *reinterpret_cast<const uint32_t*>(au);
      wb.x = *reinterpret_cast<const uint32_t*>(at + far);
      wb.y = *reinterpret_cast<const uint32_t*>(au + far);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // byte i & 3 to address bits 8 .. 15, the table's base and the lane around
      const uint32_t sel = 0x7604u | ((uint32_t)(i & 3) << 4);
      fa[i] = lds_table(prmt(i < 4 ? wa.x : wa.y, lut, sel));
      fb[i] = lds_table(prmt(i < 4 ? wb.x : wb.y, lut, sel));
    }
  };
  // Scales of a chunk: lane t4 of a row holds those of block t4 (of its four mma
  // rows), loaded a chunk ahead; the others get them by shuffle.
  using Raw = uint32_t[4];  // [half m][row g, g + 8]; NF4: fp32 bits; MXFP4: two e8m0 bytes
  auto scale_ptr = [&](int phase, int ai, int tile, int c) __attribute__((always_inline)) -> const uint8_t* {
    const int64_t sr = F == Fmt::NF4 ? (phase ? I : H) / 16 : (phase ? I : H) / 32;
    return static_cast<const uint8_t*>(phase ? p.dn_scale : p.gu_scale) +
           (first_row(phase, ai, tile) + pg) * sr + c * kScChunk + t4 * (kScChunk / 4);
  };
  // `next`, `far`: from row pg to the second half's, and to row g + 8's, in bytes
  auto load_scales = [&](const uint8_t* sp, int next, int64_t far, bool on, Raw& v) __attribute__((always_inline)) {
    if (on) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint8_t* at = sp + (m ? next : 0);
        if (F == Fmt::NF4) {
          v[2 * m] = __ldg(reinterpret_cast<const uint32_t*>(at));
          v[2 * m + 1] = __ldg(reinterpret_cast<const uint32_t*>(at + far));
        } else {
          v[2 * m] = __ldg(reinterpret_cast<const uint16_t*>(at));
          v[2 * m + 1] = __ldg(reinterpret_cast<const uint16_t*>(at + far));
        }
      }
    }
  };
  struct Scales {
    float g0, g1, h0, h1;  // mma rows g, g + 8; MXFP4: the two halves of the block
  };
  auto scales_of = [&](uint32_t v0, uint32_t v1) __attribute__((always_inline)) -> Scales {
    if (F == Fmt::NF4) return {__uint_as_float(v0), 0.0f, __uint_as_float(v1), 0.0f};
    auto f = [&](uint32_t b) { return *reinterpret_cast<const float*>(smem + Smem::e8m0 + b * 4); };
    return {f(v0 & 255u), f((v0 >> 8) & 255u), f(v1 & 255u), f((v1 >> 8) & 255u)};
  };
  // acc += block b times the lane's x
  auto mma_block = [&](float (&acc)[4], const uint32_t (&fa)[8], const uint32_t (&fb)[8],
                       const uint4& x0, const uint4& x1, const Scales& v, int b) __attribute__((always_inline)) {
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
      const int from = (lane & 28) | b;
      const float fg = __shfl_sync(0xffffffffu, m0 ? v.g1 : v.g0, from);
      const float fh = __shfl_sync(0xffffffffu, m0 ? v.h1 : v.h0, from);
      acc[0] = fmaf(d[0], fg, acc[0]);
      acc[1] = fmaf(d[1], fg, acc[1]);
      acc[2] = fmaf(d[2], fh, acc[2]);
      acc[3] = fmaf(d[3], fh, acc[3]);
    }
  };

  // Waits for the chunk to multiply; this lane's address in its stage.
  auto wait_stage = [&]() __attribute__((always_inline)) -> uint32_t {
    mbar_wait(&full[slot], ph, &misc[3], p.err);
    return get_w + slot * kStage;
  };
  // The stage may be loaded again: what was read of it has been used (the sums
  // wait for it), by every lane.
  auto used = [&](float (&acc)[4]) __attribute__((always_inline)) {
    asm volatile("" : "+f"(acc[0]), "+f"(acc[1]), "+f"(acc[2]), "+f"(acc[3]) : : "memory");
  };
  auto release = [&]() __attribute__((always_inline)) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[slot]);
    if (++slot == D) { slot = 0; ph ^= 1u; }
  };
  // One column tile, the `nb` blocks of one chunk: x holds the columns of its
  // first two blocks, raw its scales; at the end those of the chunk after it,
  // whose columns are at nsrc and scales at nsp.
  auto step_one = [&](int phase, uint4 (&x)[2][2], Raw& raw, const uint16_t* src, int nb,
                      const uint16_t* nsrc, const uint8_t* nsp, int next, int64_t far, int nnb,
                      float (&acc)[2][4]) __attribute__((always_inline)) {
    uint4 y[2][2];
    auto load_cols = [&](uint4 (&v)[2][2], const uint16_t* from, int n) __attribute__((always_inline)) {
      if (n > 0) load_x(from, v[0][0], v[0][1]);
      if (n > 1) load_x(from + 64, v[1][0], v[1][1]);
    };
    load_cols(y, src + 128, nb - 2);
    const Scales sc[2] = {scales_of(raw[0], raw[1]), scales_of(raw[2], raw[3])};
    load_scales(nsp, next, far, t4 < nnb, raw);
    const uint32_t st = wait_stage();
    const int half = phase ? 16 * CKB : 8 * CKB, other = phase ? 8 * CKB : 16 * CKB;
    auto block = [&](int b, const uint4 (&v)[2]) __attribute__((always_inline)) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t fa[8], fb[8];
        decode(st + (m ? half : 0), b, other, fa, fb);
        mma_block(acc[m], fa, fb, v[0], v[1], sc[m], b);
      }
    };
    if (nb >= 4) {
      block(0, x[0]);
      block(1, x[1]);
      load_cols(x, nsrc, nnb);
      block(2, y[0]);
      block(3, y[1]);
    } else {
      block(0, x[0]);
      if (nb > 1) block(1, x[1]);
      load_cols(x, nsrc, nnb);
      if (nb > 2) block(2, y[0]);
    }
    used(acc[0]);
    used(acc[1]);
    release();
  };
  // Phase B, two column tiles: the columns are loaded a block ahead.
  auto step_two = [&](uint4 (&x)[2][2][2], Raw& raw, const uint16_t* s0, const uint16_t* s1, int left,
                      const uint8_t* nsp, int next, int64_t far, int nnb,
                      float (&acc)[2][2][4]) __attribute__((always_inline)) {
    const Scales sc[2] = {scales_of(raw[0], raw[1]), scales_of(raw[2], raw[3])};
    load_scales(nsp, next, far, t4 < nnb, raw);
    const uint32_t st = wait_stage();
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (b < left) {
        if (b + 1 < left) {
          load_x(s0 + b * 64 + 64, x[(b + 1) & 1][0][0], x[(b + 1) & 1][0][1]);
          load_x(s1 + b * 64 + 64, x[(b + 1) & 1][1][0], x[(b + 1) & 1][1][1]);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint32_t fa[8], fb[8];
          decode(st + m * 16 * CKB, b, 8 * CKB, fa, fb);
          mma_block(acc[0][m], fa, fb, x[b & 1][0][0], x[b & 1][0][1], sc[m], b);
          mma_block(acc[1][m], fa, fb, x[b & 1][1][0], x[b & 1][1][1], sc[m], b);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      used(acc[0][m]);
      used(acc[1][m]);
    }
    release();
  };

  constexpr float kUnscale = F == Fmt::NF4 ? 1.0f / kLevelScale : 1.0f;
  // Writes half m of one column tile of a finished unit: h (phase A) or y (B).
  auto finish = [&](int phase, const float (&d)[4], int cnt, int r0, int tile, int nt, int m) __attribute__((always_inline)) {
    if (phase == 0) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = nt * 8 + 2 * t4 + j;
        if (c < cnt) {
          const int slot = rows[r0 + c];
          const float gate = d[j] * kUnscale, up = d[2 + j] * kUnscale;
          const float h = swiglu(gate, up);
          const __nv_bfloat16 hi = __float2bfloat16_rn(h);
          // an infinite high part keeps a zero low part (inf - inf is NaN)
          const float low = h - __bfloat162float(hi);
          const __nv_bfloat16 lo = __float2bfloat16_rn(isfinite(low) ? low : 0.0f);
          a.hhi[(int64_t)slot * I + tile * 16 + m * 8 + pg] = __bfloat16_as_ushort(hi);
          a.hlo[(int64_t)slot * I + tile * 16 + m * 8 + pg] = __bfloat16_as_ushort(lo);
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
          float* y = a.y + (int64_t)rows[r0 + c] * H + tile * 32 + m * 16 + pg;
          y[0] = v[j] * kUnscale;
          y[8] = v[2 + j] * kUnscale;
        }
      }
    }
  };

  float* parts = reinterpret_cast<float*>(smem + Smem::table + 128);  // row i at i * 64
  // A share: this warp's items, then the units cut into parts, joined.
  auto run_share = [&](const Share& s) __attribute__((always_inline)) {
    const int phase = s.phase;
    const int nbk = (phase ? I : H) >> 6;  // blocks of a unit
    const int64_t sr = F == Fmt::NF4 ? (phase ? I : H) / 16 : (phase ? I : H) / 32;
    const int64_t far = (phase ? 8 : I) * sr;
    const int next = (int)((phase ? 16 : 8) * sr);
    const bool wide = phase && two_tiles;
    const int rows4 = wide ? 16 : 8;       // part rows of an item
    int item = 0, u, c, c1;
    if (s.item(warp, 0, u, c, c1)) {
      uint4 x[2][2];
      Raw raw = {0, 0, 0, 0};
      const uint16_t* src = nullptr;
      const uint8_t* sp = nullptr;
      bool ready = false;  // x holds the first columns of the item
#pragma unroll 1
      for (;;) {
        int ai, tile;
        unit_of(phase, s.u0 + u, ai, tile);
        const int r0 = first[ai], cnt = first[ai + 1] - r0;
        // the columns and scales of the item after this one, loaded with its
        // last chunk
        int nu, nc0, nc1, nai, ntile;
        const bool more = s.item(warp, item + 1, nu, nc0, nc1);
        unit_of(phase, s.u0 + (more ? nu : u), nai, ntile);
        const uint16_t* nsrc = column(phase, first[nai], first[nai + 1] - first[nai], 0) + nc0 * 256;
        const uint8_t* nsp = scale_ptr(phase, nai, ntile, nc0);
        const int nnb = more ? nbk - nc0 * 4 : 0;
        if (item == 0) {
          src = column(phase, r0, cnt, 0) + c * 256;
          sp = scale_ptr(phase, ai, tile, c);
          load_scales(sp, next, far, t4 < nbk - c * 4, raw);
        }
        const bool two = phase && cnt > 4;
        if (!two && !ready) {
          load_x(src, x[0][0], x[0][1]);
          if (nbk - c * 4 > 1) load_x(src + 64, x[1][0], x[1][1]);
        }
        ready = !two;
        float acc[2][2][4];  // [column tile][half]
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[0][0][j] = acc[0][1][j] = acc[1][0][j] = acc[1][1][j] = 0.0f;
        if (!two) {
#pragma unroll 1
          for (; c < c1; ++c, src += 256, sp += kScChunk) {
            const bool last = c + 1 == c1;
            step_one(phase, x, raw, src, nbk - c * 4, last ? nsrc : src + 256,
                     last ? nsp : sp + kScChunk, next, far, last ? nnb : nbk - c * 4 - 4, acc[0]);
          }
        } else {
          const uint16_t* src1 = column(1, r0, cnt, 1) + c * 256;
          uint4 y[2][2][2];
          load_x(src, y[0][0][0], y[0][0][1]);
          load_x(src1, y[0][1][0], y[0][1][1]);
#pragma unroll 1
          for (; c < c1; ++c, src += 256, src1 += 256, sp += kScChunk) {
            const bool last = c + 1 == c1;
            step_two(y, raw, src, src1, last ? min(4, nbk - c * 4) : nbk - c * 4,
                     last ? nsp : sp + kScChunk, next, far, last ? nnb : nbk - c * 4 - 4, acc);
          }
        }
        if (u < s.whole || s.lgS == 0) {
          finish(phase, acc[0][0], cnt, r0, tile, 0, 0);
          finish(phase, acc[0][1], cnt, r0, tile, 0, 1);
          if (two) {
            finish(1, acc[1][0], cnt, r0, tile, 1, 0);
            finish(1, acc[1][1], cnt, r0, tile, 1, 1);
          }
        } else {
          // the part's place among the parts of the split units
          float* to = parts + (warp + item * kWarps - s.whole) * rows4 * 64 + lane;
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) to[(m * 4 + j) * 64] = acc[0][m][j];
          if (two)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int j = 0; j < 4; ++j) to[(8 + m * 4 + j) * 64] = acc[1][m][j];
        }
        if (!more) break;
        ++item;
        u = nu;
        c = nc0;
        c1 = nc1;
        src = nsrc;
        sp = nsp;
      }
    }
    if (s.lgS) {
      consumer_sync();
      // fewer than kWarps units are split: a piece is half a column tile of one
      const int rest = s.n - s.whole, pieces = wide ? 4 : 2;
#pragma unroll 1
      for (int w = warp; w < rest * pieces; w += kWarps) {
        const int uj = w / pieces, i = w - uj * pieces;
        int ai, tile;
        unit_of(phase, s.u0 + s.whole + uj, ai, tile);
        const int r0 = first[ai], cnt = first[ai + 1] - r0;
        if (i < 2 || cnt > 4) {
          const float* from = parts + ((uj << s.lgS) * rows4 + i * 4) * 64 + lane;
          float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
          for (int part_i = 0; part_i < (1 << s.lgS); ++part_i)
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j] += from[(part_i * rows4 + j) * 64];
          finish(phase, d, cnt, r0, tile, i >> 1, i & 1);
        }
      }
    }
  };

  // Waits until every share of phase A is done; false after a wait that ran out.
  auto wait_a = [&]() __attribute__((always_inline)) -> bool {
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
    return !consumer_any(misc[3] != 0);
  };
  // Combines the slots of output tile `tile` in slot order.
  auto combine = [&](int tile) __attribute__((always_inline)) {
    for (int i = threadIdx.x; i < T * 32; i += kConsumers) {
      const int t = i >> 5, n = tile * 32 + (i & 31);
      float v = 0.0f;
      for (int s = 0; s < k; ++s) {
        const float w = wts[t * k + s];
        if (w != 0.0f) v = fmaf(w, __ldcg(a.y + (int64_t)(t * k + s) * H + n), v);
      }
      p.out[(int64_t)t * H + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
  };

  bool waited = false;
#pragma unroll 1
  for (int i = 0;; ++i) {
    mbar_wait(&published[i & 1], (i >> 1) & 1, &misc[3], p.err);
    if (consumer_any(misc[3] != 0)) break;
    const Share& s = *share(i);
    if (threadIdx.x == 0) misc[2] = i + 1;
    if (s.phase == 2) break;
    if (s.phase == 1 && !waited) {
      waited = true;
      if (!wait_a()) break;
    }
    run_share(s);
    if (s.phase == 0 || !aligned) __threadfence();
    consumer_sync();
    if (s.phase == 0) {
      if (threadIdx.x == 0) atomicAdd(&a.counters[2], 1);
    } else if (s.n > 0) {
      // tiles that this share touches: an aligned share holds all of a tile's
      // experts; else the CTA that brings the tile's count to A combines it
      const int ub = s.u0, ue = ub + s.n, last_tile = (ue - 1) / A;
      for (int tile = ub / A; tile <= last_tile; ++tile) {
        if (aligned) {
          combine(tile);
        } else {
          if (threadIdx.x == 0) {
            const int part_n = min(ue, (tile + 1) * A) - max(ub, tile * A);
            misc[5] = atomicAdd(&a.counters[kCounters + tile], part_n) + part_n == A;
            __threadfence();
          }
          consumer_sync();
          if (misc[5]) combine(tile);
          consumer_sync();
        }
      }
    }
  }
}

// z matrices of y rows of x bytes, boxes of 128 bytes x by rows x bz.
cudaError_t make_map_3d(CUtensorMap* m, const void* base, uint64_t x, uint64_t y, uint64_t z,
                        uint32_t by, uint32_t bz) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {x, y, z}, strides[2] = {x, x * y};
  const cuuint32_t box[3] = {(cuuint32_t)CKB, by, bz}, es[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides,
                         box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
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

cudaError_t launch_router(const LayerArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.p.E, (unsigned)((a.p.T + kRouterTokens - 1) / kRouterTokens));
  const int threads = (int)std::min<int64_t>(kRouterThreads, (a.p.H / 8 + 31) / 32 * 32);
  return launch_kernel<moe_router>(grid, threads, 0, s, false, a);
}

template <Fmt F, int NPL>
cudaError_t launch_t(const LayerArgs& a, int num_sms, cudaStream_t s) {
  constexpr auto k = moe_experts<F, NPL>;
  cudaError_t e = opt_in_smem<k>(Smem::bytes);
  if (e != cudaSuccess) return e;
  e = launch_router(a, s);
  if (e != cudaSuccess) return e;
  // Whole tiles of H per CTA in phase B spare the counting of a tile's experts
  // across CTAs (about 1.5 us) but leave the last round of tiles uneven: taken
  // when that costs at most kAlignChunks chunks of 4 KB per CTA (about 92 ns
  // each at the measured HBM rate).
  constexpr int64_t kAlignChunks = 16;
  const int64_t tiles = a.p.H / 32, A = std::min<int64_t>(a.p.E, a.p.T * a.p.k);
  const int64_t whole = (tiles + num_sms - 1) / num_sms * A;
  const int64_t even = (tiles * A + num_sms - 1) / num_sms;
  const int aligned = (whole - even) * ((a.p.I + 255) / 256) <= kAlignChunks;
  CUtensorMap gu, dn;  // boxes of 16 gate and 16 up rows, and of 32 down rows
  const uint64_t kb = (uint64_t)a.p.H / 2, ib = (uint64_t)a.p.I / 2;
  e = make_map_3d(&gu, a.p.gu, kb, (uint64_t)a.p.I, (uint64_t)a.p.E * 2, 16, 2);
  if (e != cudaSuccess) return e;
  e = make_map_3d(&dn, a.p.dn, ib, (uint64_t)a.p.E * (uint64_t)a.p.H, 1, 32, 1);
  if (e != cudaSuccess) return e;
  return launch_kernel<k>(num_sms, kThreads, Smem::bytes, s, true, a, aligned, gu, dn);
}

template <Fmt F>
cudaError_t launch_f(const LayerArgs& a, int num_sms, cudaStream_t s) {
  return a.p.E <= 128 ? launch_t<F, 4>(a, num_sms, s) : launch_t<F, kMaxE / 32>(a, num_sms, s);
}

// ----------------------------------------------------------------------
// MXFP4, more weights: the layer in seven launches on the tensor cores' 4-bit path
// ----------------------------------------------------------------------

struct PiecesLayout {
  int64_t logits, ids, weights, offsets, r2t, ros, sor, xq, xs, gu, hq, hs, y, total;
};

PiecesLayout pieces_layout(int64_t T, int32_t E, int32_t k, int64_t H, int64_t I) {
  const int64_t P = T * k;
  PiecesLayout l = {};
  auto put = [&](int64_t& at, int64_t bytes) {
    at = l.total;
    l.total += (bytes + 255) & ~(int64_t)255;
  };
  put(l.logits, T * E * 4);
  put(l.ids, P * 4);
  put(l.weights, P * 4);
  put(l.offsets, (E + 1) * 4);
  put(l.r2t, P * 4);
  put(l.ros, P * 4);
  put(l.sor, P * 4);
  put(l.xq, P * kPieces * (H / 2));
  put(l.xs, P * kPieces * ((H + 127) / 128) * 4);
  put(l.gu, P * 2 * I * 4);
  put(l.hq, P * kPieces * (I / 2));
  put(l.hs, P * kPieces * ((I + 127) / 128) * 4);
  put(l.y, P * H * 4);
  return l;
}

cudaError_t launch_pieces(const LayerProblem& p, uint8_t* w, int num_sms, cudaStream_t s) {
  const PiecesLayout l = pieces_layout(p.T, p.E, p.k, p.H, p.I);
  const int64_t P = p.T * p.k;
  auto ints = [&](int64_t at) { return reinterpret_cast<int32_t*>(w + at); };
  auto floats = [&](int64_t at) { return reinterpret_cast<float*>(w + at); };
  auto words = [&](int64_t at) { return reinterpret_cast<uint32_t*>(w + at); };
  const LayerArgs a{p, floats(l.logits), nullptr, nullptr, nullptr, nullptr};
  RouteProblem r = {};
  r.logits = floats(l.logits);
  r.fp32 = 1;
  r.T = p.T;
  r.E = p.E;
  r.k = p.k;
  r.renorm = p.renorm;
  r.ids = ints(l.ids);
  r.weights = floats(l.weights);
  r.offsets = ints(l.offsets);
  r.row_to_token = ints(l.r2t);
  r.row_of_slot = ints(l.ros);
  r.slot_of_row = ints(l.sor);
  r.nan_rows = true;
  cudaError_t e = launch_router(a, s);
  if (e != cudaSuccess) return e;
  e = launch_route(r, num_sms, true, s);
  if (e != cudaSuccess) return e;
  e = launch_quantize_pieces(p.x, p.T, p.H, r.row_to_token, P, false, w + l.xq, words(l.xs), p.err, s);
  if (e != cudaSuccess) return e;
  e = launch_gemm_pieces(w + l.xq, words(l.xs), P, p.H, p.gu, static_cast<const uint8_t*>(p.gu_scale),
                         p.E, 2 * p.I, r.offsets, floats(l.gu), p.err, num_sms, s);
  if (e != cudaSuccess) return e;
  e = launch_quantize_pieces(floats(l.gu), P, p.I, nullptr, P, true, w + l.hq, words(l.hs), p.err, s);
  if (e != cudaSuccess) return e;
  e = launch_gemm_pieces(w + l.hq, words(l.hs), P, p.I, p.dn, static_cast<const uint8_t*>(p.dn_scale),
                         p.E, p.H, r.offsets, floats(l.y), p.err, num_sms, s);
  if (e != cudaSuccess) return e;
  return launch_combine_f32(floats(l.y), P, p.H, r.row_of_slot, r.weights, p.T, p.k, p.out, p.err,
                            num_sms, s);
}

// Whether MXFP4 takes that way: its five launches more cost 1 to 4 us, its
// products take the weights nearer to the memory rate, so it pays from some
// number of bytes on: 40 to 110 MB of codes, fewer where an expert has more of the
// tokens; from 100 MB it never measured slower.  T tokens that choose independently
// are expected to need E (1 - (1 - k / E)^T) experts.  us, (1) / (2), and those
// experts' codes:
//   hidden 2880, 4 of 32 experts   1 token 34 / 35 (50 MB), 2: 47 / 46 (93),
//     3: 61 / 50 (131), 4: 70 / 58 (165), 8: 99 / 76 (261), 32: 154 / 99 (393)
//   hidden 2048, intermediate 768, 8 of 128   6: 50 / 51 (97), 8: 56 / 56 (122),
//     12: 66 / 64 (163), 16: 80 / 73 (194), 32: 109 / 92 (264)
//   hidden 4096, intermediate 2048, 2 of 8   1: 23 / 27 (25), 4: 47 / 39 (69),
//     8: 51 / 41 (91), 32: 69 / 45 (101)
bool takes_pieces(const LayerProblem& p) {
  const double experts = p.E * (1.0 - std::pow(1.0 - (double)p.k / p.E, (double)p.T));
  constexpr int64_t most = (int64_t)65535 * 256;  // a launch's grid of 256-value pieces
  return p.H <= most && p.I <= most && experts * 1.5 * (double)p.H * (double)p.I >= 1e8;
}

}  // namespace

int64_t layer_workspace(int64_t T, int32_t E, int32_t k, int64_t H, int64_t I) {
  return std::max(layout_of(T, E, k, H, I).total, pieces_layout(T, E, k, H, I).total);
}

cudaError_t launch_layer(Fmt f, const LayerProblem& p, void* workspace, int num_sms,
                         cudaStream_t s) {
  if (p.T == 0) return cudaSuccess;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  if (f == Fmt::MXFP4 && takes_pieces(p)) return launch_pieces(p, w, num_sms, s);
  const Layout l = layout_of(p.T, p.E, p.k, p.H, p.I);
  const LayerArgs a{p,
                    reinterpret_cast<float*>(w + l.logits),
                    reinterpret_cast<uint16_t*>(w + l.hhi),
                    reinterpret_cast<uint16_t*>(w + l.hlo),
                    reinterpret_cast<float*>(w + l.y),
                    reinterpret_cast<int*>(w + l.counters)};
  return f == Fmt::NF4 ? launch_f<Fmt::NF4>(a, num_sms, s) : launch_f<Fmt::MXFP4>(a, num_sms, s);
}

}  // namespace gbw
