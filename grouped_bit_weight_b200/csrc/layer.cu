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
constexpr int kMaxT = 32;
constexpr int kMaxP = 512;
constexpr int NT = kMaxT / 4;      // most column tiles (MMA N = 8) of one expert
constexpr int CKB = 128;           // bytes per weight row and stage: 256 k
constexpr int D = 4;               // stages per warp
constexpr int kStage = 16 * CKB;   // 2 KB
constexpr int kScStage = 256;      // scales of a stage

// Shared memory.  Table entry b of lane l at b * 256 + l * 4; the other half
// of each 256 bytes holds partial sums (kParts rows of 32 floats).
constexpr int kParts = 256;
struct Smem {
  static constexpr int table = 0;
  static constexpr int ring = 65536;
  static constexpr int scales = ring + kWarps * D * kStage;
  static constexpr int ids = scales + kWarps * D * kScStage;  // [kMaxP] int
  static constexpr int wts = ids + 4 * kMaxP;                 // [kMaxP] float
  static constexpr int rows = wts + 4 * kMaxP;                // [kMaxP] uint16 slot of sorted row
  static constexpr int active = rows + 2 * kMaxP;             // [kMaxP] uint16 expert
  static constexpr int first = active + 2 * kMaxP;            // [kMaxP + 1] int first sorted row
  static constexpr int misc = first + 4 * (kMaxP + 4);        // 32 ints
  static constexpr int part = misc + 128;                     // [kWarps] scan parts
  static constexpr int count = part + 4 * kWarps;             // [kMaxE] int
  static constexpr int total = count + 4 * kMaxE;
};
static_assert(Smem::total <= 232448, "shared memory exceeds the 227 KB a CTA can have");

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

constexpr int kRouterThreads = 256;
constexpr int kRouterTokens = 8;

__global__ void __launch_bounds__(kRouterThreads) moe_router(const LayerArgs a) {
  const LayerProblem& p = a.p;
  __shared__ float part[kRouterThreads / 32][kRouterTokens];
  grid_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < kCounters + (int)(p.H / 16); i += kRouterThreads) a.counters[i] = 0;
  const int e = blockIdx.x, t0 = blockIdx.y * kRouterTokens;
  const int n = min(kRouterTokens, (int)p.T - t0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int U = (int)(p.H / 8);
  const uint4* w = reinterpret_cast<const uint4*>(p.rw + (int64_t)e * p.H);
  float acc[kRouterTokens] = {};
  for (int u = threadIdx.x; u < U; u += kRouterThreads) {
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
#pragma unroll
    for (int i = 0; i < kRouterThreads / 32; ++i) v += part[i][threadIdx.x];
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

// D += A (16 x 16, row) * B (16 x 8, col), bf16 in, fp32 out.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// 16-byte unit u of row r of a stage is stored at u ^ swizzle(r): the rows'
// lanes then read different banks (NF4: 8 bytes a lane, 4 rows a wavefront;
// MXFP4: 4 bytes a lane, 8 rows).
template <Fmt F>
__device__ __forceinline__ uint32_t swizzle(int r) {
  return F == Fmt::NF4 ? 2u * (r & 3) : (uint32_t)(r & 7);
}

// One phase's share of this CTA: units [u0, u0 + n) of nc chunks (256 k)
// each, every unit split into 1 << lgS parts.
struct Share {
  int phase;  // 0: gate_up, 1: down
  int u0, n, lgS;
  int nc;
  __device__ __forceinline__ int items() const { return n << lgS; }
  // first chunk of part sp
  __device__ __forceinline__ int chunk0(int sp) const { return (sp * nc) >> lgS; }
};

// A warp's place in its stream of (item, chunk) over both shares.
struct Cursor {
  int phase, item, c, c1;   // chunk c of [.., c1) of the item
  const uint8_t* w;         // codes of row 0 of the unit (chunk 0)
  const uint8_t* sc;        // scales of row 0 of the unit
};

// Column tiles of an expert with cnt rows.  Phase A: 8 rows a tile.  Phase B:
// 4 rows, the high parts of h in columns 0..3 and the low parts in 4..7.
__device__ __forceinline__ int col_tiles(int phase, int cnt) {
  return phase ? (cnt + 3) >> 2 : (cnt + 7) >> 3;
}

template <Fmt F, int NPL, bool kFew>
__global__ void __launch_bounds__(kThreads, 1) moe_experts(const LayerArgs a, const int aligned) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const LayerProblem& p = a.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int T = (int)p.T, E = p.E, k = p.k, P = T * k;
  const int H = (int)p.H, I = (int)p.I;
  const uint32_t sbase = smem_u32(smem);
  int* ids = reinterpret_cast<int*>(smem + Smem::ids);
  float* wts = reinterpret_cast<float*>(smem + Smem::wts);
  uint16_t* rows = reinterpret_cast<uint16_t*>(smem + Smem::rows);
  uint16_t* active = reinterpret_cast<uint16_t*>(smem + Smem::active);
  int* first = reinterpret_cast<int*>(smem + Smem::first);
  volatile int* misc = reinterpret_cast<volatile int*>(smem + Smem::misc);
  int* part = reinterpret_cast<int*>(smem + Smem::part);
  int* count = reinterpret_cast<int*>(smem + Smem::count);
  // misc: 0 claim A, 1 claim B, 2 next claim, 3 abort, 4 active experts, 5 last of a tile,
  // 6 rows of the largest expert

  {
    // warp w writes the 16 bytes of high nibble w: lane l holds level l & 15
    const uint32_t level = code_bf16<F>(lane & 15), top = code_bf16<F>(warp);
#pragma unroll
    for (int l = 0; l < 16; ++l) {
      const uint32_t low = __shfl_sync(0xffffffffu, level, l);
      sts32(sbase + Smem::table + (warp * 16 + l) * 256 + lane * 4,
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
    choose<LogitL2, NPL>(reinterpret_cast<const LogitL2*>(a.logits) + (int64_t)t * E, E, k, p.renorm, lane, id, w);
    if (lane < k) {
      ids[t * k + lane] = id;
      wts[t * k + lane] = w;
      atomicAdd(&count[id], 1);
    }
  }
  __syncthreads();
  // rows sorted by expert and the list of active experts: two packed scans
  // (rows below, active experts below), two experts per thread
  {
    const int e0 = threadIdx.x * 2;
    const int c0 = e0 < E ? count[e0] : 0, c1 = e0 + 1 < E ? count[e0 + 1] : 0;
    const int v = (c0 + c1) | (((c0 > 0) + (c1 > 0)) << 16);
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
    if (c0) { active[a0] = (uint16_t)e0; first[a0] = r0; }
    if (c1) { active[a0 + (c0 > 0)] = (uint16_t)(e0 + 1); first[a0 + (c0 > 0)] = r0 + c0; }
    if (threadIdx.x == kThreads - 1) {
      misc[4] = (below + v) >> 16;
      first[(below + v) >> 16] = P;
    }
    __syncthreads();
    if (e0 < E) count[e0] = r0;
    if (e0 + 1 < E) count[e0 + 1] = r0 + c0;
    __syncthreads();
    // the order of an expert's rows does not enter any sum
    for (int s = threadIdx.x; s < P; s += kThreads) rows[atomicAdd(&count[ids[s]], 1)] = (uint16_t)s;
  }
  __syncthreads();
  const int A = misc[4];
  const int G = gridDim.x;
  int next_a = misc[0], next_b = misc[1];
  const int tiles_a = I / 8, tiles_b = H / 16;

  const int largest = misc[6];  // rows of the largest expert
  auto make_share = [&](int phase, int idx) -> Share {
    Share s;
    s.phase = phase;
    const int tiles = phase ? tiles_b : tiles_a;
    // phase B, aligned: whole tiles, so that no tile is shared between CTAs
    const int per = phase && aligned ? A : 1;
    const unsigned total = (unsigned)(tiles * (A / per));
    const unsigned q = total / (unsigned)G, r = total - q * (unsigned)G;
    s.u0 = (int)(q * idx + min((unsigned)idx, r)) * per;
    s.n = idx < G ? (int)(q + (idx < (int)r)) * per : 0;
    s.nc = ((phase ? I : H) + 255) >> 8;
    // the split with the least work for the busiest warp, as far as the
    // partial sums (4 rows of 32 for each column tile) fit
    const int rows4 = 4 * col_tiles(phase, largest);
    s.lgS = 0;
    int best = ((s.n + kWarps - 1) / kWarps) * 8;  // eighths of a unit
#pragma unroll
    for (int l = 1; l <= 3; ++l) {
      if ((1 << l) <= s.nc && (s.n << l) * rows4 <= kParts) {
        const int cost = (((s.n << l) + kWarps - 1) / kWarps) << (3 - l);
        if (cost < best) { best = cost; s.lgS = l; }
      }
    }
    return s;
  };

  // (expert index, tile) of unit u
  auto unit_of = [&](int phase, int u, int& ai, int& tile) {
    if (phase == 0) {
      ai = u / tiles_a;
      tile = u - ai * tiles_a;
    } else {
      tile = u / A;
      ai = u - tile * A;
    }
  };

  const int64_t kb_a = H / 2, kb_b = I / 2;                       // bytes of codes per row
  const int64_t sr_a = F == Fmt::NF4 ? H / 16 : H / 32;           // scale bytes per row
  const int64_t sr_b = F == Fmt::NF4 ? I / 16 : I / 32;

  // Points cur at the first chunk of `item` of share s (item < s.n * s.S).
  auto seek = [&](Cursor& cur, const Share& s, int item) {
    cur.phase = s.phase;
    cur.item = item;
    const int u = item >> s.lgS, sp = item - (u << s.lgS);
    cur.c = s.chunk0(sp);
    cur.c1 = s.chunk0(sp + 1);
    int ai, tile;
    unit_of(s.phase, s.u0 + u, ai, tile);
    const int64_t e = active[ai];
    if (s.phase == 0) {
      const int64_t r = e * 2 * I + tile * 8;
      cur.w = p.gu + r * kb_a;
      cur.sc = static_cast<const uint8_t*>(p.gu_scale) + r * sr_a;
    } else {
      const int64_t r = e * H + tile * 16;
      cur.w = p.dn + r * kb_b;
      cur.sc = static_cast<const uint8_t*>(p.dn_scale) + r * sr_b;
    }
  };

  const uint32_t ring = sbase + Smem::ring + warp * D * kStage;
  const uint32_t scr = sbase + Smem::scales + warp * D * kScStage;
  // row r of a unit lies r rows below row 0, or (up rows) I - 8 further
  const int my_row = lane >> 3, my_unit = lane & 7;  // cp.async: rows my_row + 4 j
  const int sc_row = lane >> 1, sc_half = lane & 1;
  uint32_t sv0 = 0, sv1 = 0;       // scales loaded for the stage before
  uint32_t sv_to = 0xffffffffu;    // where they go, or nothing pending

  auto put_scales = [&]() {
    if (sv_to != 0xffffffffu) {
      if (F == Fmt::NF4) {
        sts32(sv_to, __float_as_uint(__uint_as_float(sv0) * (1.0f / kLevelScale)));
        sts32(sv_to + 4, __float_as_uint(__uint_as_float(sv1) * (1.0f / kLevelScale)));
      } else {
        // e8m0 byte s -> bf16 bits of 2^(s - 127)
        auto f = [](uint32_t s) -> uint32_t { return s == 0u ? 0x40u : s == 255u ? 0x7FC0u : s << 7; };
        sts32(sv_to, f(sv0 & 255u) | (f((sv0 >> 8) & 255u) << 16));
        sts32(sv_to + 4, f(sv1 & 255u) | (f((sv1 >> 8) & 255u) << 16));
      }
      sv_to = 0xffffffffu;
    }
  };
  // Issues the loads of one chunk into ring slot q & (D - 1).
  auto fetch = [&](const Cursor& cur, uint32_t q) {
    put_scales();
    const uint32_t slot = q & (D - 1);
    const int64_t kb = cur.phase ? kb_b : kb_a, sr = cur.phase ? sr_b : sr_a;
    const int valid = min(8, (int)((kb - (int64_t)cur.c * CKB) >> 4));  // 16-byte units per row
    const int64_t skip = cur.phase ? 0 : I - 8;
    if (my_unit < valid) {
      const uint8_t* src = cur.w + (int64_t)cur.c * CKB + my_unit * 16;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = my_row + 4 * j;
        cp_async_16(ring + slot * kStage + r * CKB + ((my_unit ^ swizzle<F>(r)) << 4),
                    src + (r + (j >= 2 ? skip : 0)) * kb);
      }
    }
    const int nb = valid >> 1;  // 64-k blocks
    const uint8_t* sp = cur.sc + (sc_row + (sc_row >= 8 ? skip : 0)) * sr;
    sv0 = sv1 = 0;
    if (F == Fmt::NF4) {
      const uint32_t* f = reinterpret_cast<const uint32_t*>(sp) + cur.c * 4 + sc_half * 2;
      if (sc_half * 2 < nb) sv0 = __ldg(f);
      if (sc_half * 2 + 1 < nb) sv1 = __ldg(f + 1);
    } else {
      const uint16_t* f = reinterpret_cast<const uint16_t*>(sp + cur.c * 8) + sc_half * 2;
      if (sc_half * 2 < nb) sv0 = __ldg(f);
      if (sc_half * 2 + 1 < nb) sv1 = __ldg(f + 1);
    }
    sv_to = scr + slot * kScStage + sc_row * 16 + sc_half * 8;
  };

  // ---- the warp's stream of chunks: share A, then share B
  Share sa = make_share(0, next_a), sb = make_share(1, next_b);
  uint32_t q_in = 0, q_out = 0;  // chunks issued and consumed
  Cursor pc{};                   // next chunk to issue
  bool more;                     // whether there is one
  auto start = [&]() {  // the stream from share sa's first item
    more = true;
    if (warp < sa.items()) seek(pc, sa, warp);
    else if (warp < sb.items()) seek(pc, sb, warp);
    else more = false;
  };
  auto advance = [&]() {
    if (++pc.c < pc.c1) return;
    const Share& s = pc.phase ? sb : sa;
    const int item = pc.item + kWarps;
    if (item < s.items()) seek(pc, s, item);
    else if (pc.phase == 0 && warp < sb.items()) seek(pc, sb, warp);
    else more = false;
  };
  auto issue = [&]() {
    if (more) {
      fetch(pc, q_in);
      ++q_in;
      advance();
    } else {
      put_scales();
    }
    cp_async_commit();
  };

  const int g = lane >> 2, t4 = lane & 3;
  const uint32_t lut = (uint32_t)lane * 4u;

  constexpr int kSecond = F == Fmt::NF4 ? 8 : 32;  // distance of a lane's second 8 k

  // This lane's column in column tile i of an expert's rows, at its first k of
  // a stage, or null.
  auto column = [&](int phase, int i, int r0, int cnt) -> const uint16_t* {
    const int row = phase ? i * 4 + (g & 3) : i * 8 + g;
    if (row >= cnt) return nullptr;
    const int slot = rows[r0 + row], k0 = t4 * (F == Fmt::NF4 ? 16 : 8);
    if (phase == 0) return p.x + (int64_t)(slot / k) * H + k0;
    return (g < 4 ? a.hhi : a.hlo) + (int64_t)slot * I + k0;
  };
  // plain loads: h was written by other CTAs of this launch, before the wait
  auto load_x = [&](const uint16_t* src, int c, int b, uint4& x0, uint4& x1) {
    x0 = x1 = make_uint4(0, 0, 0, 0);
    if (src) {
      const uint16_t* xp = src + c * 256 + b * 64;
      x0 = *reinterpret_cast<const uint4*>(xp);
      x1 = *reinterpret_cast<const uint4*>(xp + kSecond);
    }
  };
  // Weight fragments of block b of a stage: the lane's 16 weights of rows g and
  // g + 8 (same swizzle).  NF4, one scale block: bytes 8 t4 .. of its 32;
  // MXFP4, two blocks of 16 bytes: 4 bytes of each, so that every mma stays
  // inside a scale block.
  auto decode = [&](const uint8_t* st, int b, uint32_t (&fa)[8], uint32_t (&fb)[8]) {
    uint2 wa, wb;
    if (F == Fmt::NF4) {
      const uint32_t at = ((uint32_t)(2 * b + (t4 >> 1)) ^ swizzle<F>(g)) * 16 + (t4 & 1) * 8;
      wa = *reinterpret_cast<const uint2*>(st + at);
      wb = *reinterpret_cast<const uint2*>(st + 8 * CKB + at);
    } else {
      const uint32_t a0 = ((uint32_t)(2 * b) ^ swizzle<F>(g)) * 16 + t4 * 4;
      const uint32_t a1 = ((uint32_t)(2 * b + 1) ^ swizzle<F>(g)) * 16 + t4 * 4;
      auto word = [&](uint32_t at) { return *reinterpret_cast<const uint32_t*>(st + at); };
      wa = make_uint2(word(a0), word(a1));
      wb = make_uint2(word(8 * CKB + a0), word(8 * CKB + a1));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t sel = 0x7704u | ((uint32_t)(i & 3) << 4);  // byte i & 3 to bits 8..15
      fa[i] = lds_table(sbase + Smem::table + prmt(i < 4 ? wa.x : wa.y, lut, sel));
      fb[i] = lds_table(sbase + Smem::table + prmt(i < 4 ? wb.x : wb.y, lut, sel));
    }
  };
  // acc += block b (scale words sg, sh of rows g, g + 8) times the lane's x
  auto mma_block = [&](float (&acc)[4], const uint32_t (&fa)[8], const uint32_t (&fb)[8],
                       const uint4& x0, const uint4& x1, uint32_t sg, uint32_t sh) {
    const uint32_t xb[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
    constexpr int kPer = F == Fmt::NF4 ? 4 : 2;  // mma of one scale block
#pragma unroll
    for (int m0 = 0; m0 < 4; m0 += kPer) {
      float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int m = m0; m < m0 + kPer; ++m) {
        const uint32_t fr[4] = {fa[2 * m], fb[2 * m], fa[2 * m + 1], fb[2 * m + 1]};
        mma16816(d, fr, xb[2 * m], xb[2 * m + 1]);
      }
      const uint32_t wg = F == Fmt::NF4 ? sg : m0 ? sg & 0xFFFF0000u : sg << 16;
      const uint32_t wh = F == Fmt::NF4 ? sh : m0 ? sh & 0xFFFF0000u : sh << 16;
      acc[0] = fmaf(d[0], __uint_as_float(wg), acc[0]);
      acc[1] = fmaf(d[1], __uint_as_float(wg), acc[1]);
      acc[2] = fmaf(d[2], __uint_as_float(wh), acc[2]);
      acc[3] = fmaf(d[3], __uint_as_float(wh), acc[3]);
    }
  };

  // Chunks [c0, c1) of one unit against N column tiles.  One tile (the usual
  // case): the columns of the next chunk are loaded while this one is
  // multiplied.
  auto run_one = [&](int phase, int c0, int c1, int r0, int cnt, float (&acc)[4]) {
    const int K = phase ? I : H;
    const uint16_t* src = column(phase, 0, r0, cnt);
    uint4 x[4][2];
#pragma unroll
    for (int b = 0; b < 4; ++b) load_x(c0 * 256 + b * 64 < K ? src : nullptr, c0, b, x[b][0], x[b][1]);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = 0.0f;
    for (int c = c0; c < c1; ++c, ++q_out) {
      issue();
      uint4 y[4][2];
#pragma unroll
      for (int b = 0; b < 4; ++b)
        load_x(c + 1 < c1 && (c + 1) * 256 + b * 64 < K ? src : nullptr, c + 1, b, y[b][0], y[b][1]);
      cp_async_wait_group<D - 1>();
      __syncwarp();
      const uint32_t slot = q_out & (D - 1);
      const uint8_t* st = smem + Smem::ring + (warp * D + slot) * kStage + g * CKB;
      const uint8_t* ss = smem + Smem::scales + (warp * D + slot) * kScStage + g * 16;
      const uint4 s0 = *reinterpret_cast<const uint4*>(ss);
      const uint4 s1 = *reinterpret_cast<const uint4*>(ss + 8 * 16);
      const uint32_t sx[4] = {s0.x, s0.y, s0.z, s0.w}, sy[4] = {s1.x, s1.y, s1.z, s1.w};
      const int nb = (K - c * 256) >> 6;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (b < nb) {
          uint32_t fa[8], fb[8];
          decode(st, b, fa, fb);
          mma_block(acc, fa, fb, x[b][0], x[b][1], sx[b], sy[b]);
        }
      }
      __syncwarp();
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        x[b][0] = y[b][0];
        x[b][1] = y[b][1];
      }
    }
  };
  auto run_many = [&](int phase, int c0, int c1, int r0, int cnt, int nt, auto& acc) {
    constexpr int N = sizeof(acc) / sizeof(acc[0]);
    const int K = phase ? I : H;
    const uint16_t* src[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      src[i] = i < nt ? column(phase, i, r0, cnt) : nullptr;
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    }
    for (int c = c0; c < c1; ++c, ++q_out) {
      issue();
      cp_async_wait_group<D - 1>();
      __syncwarp();
      const uint32_t slot = q_out & (D - 1);
      const uint8_t* st = smem + Smem::ring + (warp * D + slot) * kStage + g * CKB;
      const uint8_t* ss = smem + Smem::scales + (warp * D + slot) * kScStage + g * 16;
      const int nb = min(4, (K - c * 256) >> 6);
      for (int b = 0; b < nb; ++b) {
        uint4 x0[2], x1[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) load_x(src[i], c, b, x0[i], x1[i]);
        const uint32_t sg = *reinterpret_cast<const uint32_t*>(ss + b * 4);
        const uint32_t sh = *reinterpret_cast<const uint32_t*>(ss + 8 * 16 + b * 4);
        uint32_t fa[8], fb[8];
        decode(st, b, fa, fb);
        mma_block(acc[0], fa, fb, x0[0], x1[0], sg, sh);
        mma_block(acc[1], fa, fb, x0[1], x1[1], sg, sh);
#pragma unroll
        for (int i = 2; i < N; ++i) {
          if (i < nt) {
            load_x(src[i], c, b, x0[0], x1[0]);
            mma_block(acc[i], fa, fb, x0[0], x1[0], sg, sh);
          }
        }
      }
      __syncwarp();
    }
  };

  // Writes one column tile of a finished unit: h (phase A) or y (phase B).
  auto finish = [&](int phase, const float (&d)[4], int cnt, int r0, int tile, int nt) {
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

  float* parts = reinterpret_cast<float*>(smem + Smem::table + 128);  // row i at i * 64 floats
  // All items of a share, their partial sums joined, results written.
  auto run_share = [&](const Share& s) {
    const int items = s.items();
    const int per = items ? kParts / items : 0;  // part rows of an item: [tile][4] of 32 floats
    for (int item = warp; item < items; item += kWarps) {
      const int u = item >> s.lgS, sp = item - (u << s.lgS);
      int ai, tile;
      unit_of(s.phase, s.u0 + u, ai, tile);
      const int r0 = first[ai], cnt = first[ai + 1] - r0;
      const int c0 = s.chunk0(sp), c1 = s.chunk0(sp + 1), nt = col_tiles(s.phase, cnt);
      auto store = [&](const float (&d)[4], int i) {
        if (s.lgS == 0) {
          finish(s.phase, d, cnt, r0, tile, i);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) parts[(item * per + i * 4 + j) * 64 + lane] = d[j];
        }
      };
      if (nt == 1) {
        float acc[4];
        run_one(s.phase, c0, c1, r0, cnt, acc);
        store(acc, 0);
      } else if (kFew || nt == 2) {
        float acc[2][4];
        run_many(s.phase, c0, c1, r0, cnt, nt, acc);
        store(acc[0], 0);
        store(acc[1], 1);
      } else {
        float acc[NT][4];
        run_many(s.phase, c0, c1, r0, cnt, nt, acc);
#pragma unroll
        for (int i = 0; i < NT; ++i)
          if (i < nt) store(acc[i], i);
      }
    }
    if (s.lgS > 0) {
      __syncthreads();
      for (int u = 0; u < s.n; ++u) {
        int ai, tile;
        unit_of(s.phase, s.u0 + u, ai, tile);
        const int r0 = first[ai], cnt = first[ai + 1] - r0, nt = col_tiles(s.phase, cnt);
        for (int i = (warp - u * nt) & (kWarps - 1); i < nt; i += kWarps) {
          float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          for (int sp = 0; sp < (1 << s.lgS); ++sp)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              d[j] += parts[(((u << s.lgS) + sp) * per + i * 4 + j) * 64 + lane];
          finish(s.phase, d, cnt, r0, tile, i);
        }
      }
    }
  };

  start();
#pragma unroll
  for (int i = 0; i < D - 1; ++i) issue();

  // ---- phase A
  while (next_a < G) {
    run_share(sa);
    if (threadIdx.x == 0) misc[2] = atomicAdd(&a.counters[0], 1);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) atomicAdd(&a.counters[2], 1);
    next_a = misc[2];
    if (next_a < G) {
      // another share is unclaimed (some CTAs have not started): what is in
      // flight belongs to share B; drop it and start the stream again
      cp_async_wait_group<0>();
      __syncthreads();
      sa = make_share(0, next_a);
      sv_to = 0xffffffffu;
      q_in = q_out = 0;
      start();
#pragma unroll
      for (int i = 0; i < D - 1; ++i) issue();
    }
  }
  // ---- all of phase A done?
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
  // ---- phase B
  while (next_b < G && !misc[3]) {
    run_share(sb);
    if (threadIdx.x == 0) misc[2] = atomicAdd(&a.counters[1], 1);
    if (!aligned) __threadfence();
    __syncthreads();
    // Tiles that this share touches: an aligned share holds all of a tile's
    // experts; else the CTA that brings the tile's count to A combines it.
    if (sb.n > 0) {
      const int first_tile = sb.u0 / A, last_tile = (sb.u0 + sb.n - 1) / A;
      for (int tile = first_tile; tile <= last_tile; ++tile) {
        bool whole = true;
        if (!aligned) {
          if (threadIdx.x == 0) {
            const int mine = min(sb.u0 + sb.n, (tile + 1) * A) - max(sb.u0, tile * A);
            misc[5] = atomicAdd(&a.counters[kCounters + tile], mine) + mine == A;
            __threadfence();
          }
          __syncthreads();
          whole = misc[5];
        }
        if (whole) {
          for (int i = threadIdx.x; i < T * 16; i += kThreads) {
            const int t = i >> 4, n = tile * 16 + (i & 15);
            float v = 0.0f;
            for (int s = 0; s < k; ++s) {
              const float w = wts[t * k + s];
              if (w != 0.0f) v = fmaf(w, __ldcg(a.y + (int64_t)(t * k + s) * H + n), v);
            }
            p.out[(int64_t)t * H + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
          }
        }
        if (!aligned) __syncthreads();
      }
    }
    next_b = misc[2];
    if (next_b < G) {
      cp_async_wait_group<0>();
      __syncthreads();  // before misc[2] and the part rows are written again
      sa.n = 0;
      sb = make_share(1, next_b);
      sv_to = 0xffffffffu;
      q_in = q_out = 0;
      start();
#pragma unroll
      for (int i = 0; i < D - 1; ++i) issue();
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

template <Fmt F, int NPL, bool kFew>
cudaError_t launch_t(const LayerArgs& a, int num_sms, cudaStream_t s) {
  constexpr auto k = moe_experts<F, NPL, kFew>;
  cudaError_t e = opt_in_smem<k>(Smem::total);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.p.E, (unsigned)((a.p.T + kRouterTokens - 1) / kRouterTokens));
  cfg.blockDim = dim3(kRouterThreads);
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
  return launch_kernel<k>(num_sms, kThreads, Smem::total, s, true, a, aligned);
}

template <Fmt F>
cudaError_t launch_f(const LayerArgs& a, int num_sms, cudaStream_t s) {
  const bool few = a.p.T <= 8;  // at most 8 rows per expert: two column tiles
  if (a.p.E <= 128) return few ? launch_t<F, 4, true>(a, num_sms, s) : launch_t<F, 4, false>(a, num_sms, s);
  return launch_t<F, 32, false>(a, num_sms, s);
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
