// a4.cu -- microscaled 4-bit activations: rows of bf16 to MXFP4, and the
// grouped product of MXFP4 rows with MXFP4 expert weights on the tensor
// cores' block-scaled 4-bit path.
//
//   quantise  per 32 consecutive values: X = floor(log2 max|v|) - 2 clamped to
//             [-127, 127], scale byte X + 127, codes = v / 2^X to the nearest
//             e2m1 (ties to the even code, saturating); v is a row of x, or
//             silu(gate) * up of a gate_up row, in fp32
//   product   out[p, n] = sum_k xq[p, k] wq[n, k], both e2m1 * 2^(scale - 127);
//             the products of 32-blocks and their two scales are exact in the
//             tensor core, the sum is fp32, one rounding to bf16
//
// Quantise is bound by the instructions of its conversion.
//
// Product, one persistent CTA per SM, 20 warps ("swap AB": MMA M is 128
// weight rows, MMA N the routed rows of one expert, so few rows give a narrow
// N instead of a padded M):
//   warp 0      TMA: packed weights [128 x 128 bytes = 256 k] and the rows'
//               codes (boxes of 64 rows) into a 4-stage ring, 128B swizzle --
//               the packed bytes are the MMA's operands as they are
//   warps 4-11  the scale bytes of 128 weight rows and up to 256 routed rows,
//               loaded two stages ahead and written to TMEM (a set per stage)
//   warp 1      tcgen05.mma.kind::mxf4.block_scale, 64 k each
//   warps 12-19 epilogue: tcgen05.ld -> bf16 -> 64-byte row segments
// A tile holds up to 256 routed rows.  Tiles of up to 192 alternate between two
// accumulator halves, so that an epilogue overlaps the next tile's MMAs; larger
// ones take both.
// Tiles (expert, weight tile, row tile) run with row tiles innermost: an
// expert's weights come from HBM once.
// What bounds it: no one part.  Of 109 us for 8192 ragged rows of 32 experts,
// 5760 x 2880 (2.5 PFLOP/s; 3.6 TB/s of weights, rows and output), the MMAs alone
// are 27 (twice as many took that much longer), the bytes 60.  When it took 134,
// leaving out the stores, the scale loads or the row loads won 8, 10 and 1 % each.
// The rest is waiting along the chain from an empty stage to a full one (scale bytes to
// registers, shared memory, TMEM) and, for tiles over 192 rows, for the
// epilogue.  4004 rows, 2880 x 2880: 41 us (1.6 PFLOP/s); 16 rows each of
// 8 experts, 256 x 512: 4.4 us, latency.
//
// Rows in pieces (quantize_pieces_kernel, gemm_a4_kernel<kPieces>) are for the
// layer of a few tokens: a bf16 or fp32 row becomes sixteen MXFP4 rows that sum to
// it within 2^-32 of each 32-block's maximum, so that weights meet rows of full
// precision on the same path.
#include "common.cuh"
#include "launch.cuh"
#include "swiglu.cuh"

namespace gbw {

cudaError_t make_map_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base,
                        uint64_t d0, uint64_t d1, uint64_t pitch, uint32_t b0,
                        uint32_t b1, CUtensorMapSwizzle sw);

namespace {

// ----------------------------------------------------------------------
// quantise
// ----------------------------------------------------------------------

// Two values to one byte of e2m1 codes, `lo` in the low nibble.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t d;
  asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n cvt.u32.u8 %0, t;\n}\n"
      : "=r"(d)
      : "f"(hi), "f"(lo));
  return d;
}

// Eight values to a word of codes, the first in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t d;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(d)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return d;
}

// The two values of a byte of codes.
__device__ __forceinline__ float2 e2m1_values(uint32_t byte) {
  uint32_t h;
  asm("{\n .reg .b8 t;\n cvt.u8.u32 t, %1;\n cvt.rn.f16x2.e2m1x2 %0, t;\n}\n" : "=r"(h) : "r"(byte));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ void unpack8(uint4 q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// A warp quantises kUnits * 256 values of a row, 8 a lane and unit; the 4 lanes
// of a 32-block share its maximum.  The scale bytes of 128 k are one word, word
// (k / 128) * P + p; a block's warps take neighbouring rows, whose words share a
// sector.  8192 rows of 2880, gathered from 2048 tokens, take 11.4 us (5 TB/s in and
// out, most of it L2: 2.1 TB/s of distinct bytes), 4004 SwiGLU rows 12.6 (4 TB/s),
// bound by about 60 and 140 instructions per unit.  (When they took
// 12.8 and 13.1: rows by whole warps 12.1 and 14.3, one unit a warp 16.8 and 14.3,
// six 12.3 and 13.1, but 2.7 instead of 2.3 us for a few rows.)
constexpr int kQRows = 4;  // warps, and rows, of a block
template <bool kGLU>
constexpr int kUnits = kGLU ? 2 : 4;  // loaded before the first is used
template <bool kGLU>
__global__ void __launch_bounds__(32 * kQRows) quantize_rows_kernel(
    const uint16_t* __restrict__ x, int64_t T, int K, const int32_t* __restrict__ r2t, int64_t P,
    uint8_t* __restrict__ codes, uint32_t* __restrict__ scales, int* err) {
  constexpr int NB = kUnits<kGLU>;
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, U = K / 8, KA = (K + 127) / 128;
  const int64_t p = (int64_t)blockIdx.x * kQRows + (threadIdx.x >> 5);
  if (p >= P) return;
  const int64_t t = token_of_row(r2t, (int32_t)p, T, lane == 0 ? err : nullptr);
  const uint4* row = reinterpret_cast<const uint4*>(x + t * K * (kGLU ? 2 : 1));
  uint32_t* out = reinterpret_cast<uint32_t*>(codes) + p * U;
  const int c0 = blockIdx.y * (32 * NB) + lane;
  uint4 g[NB], u[kGLU ? NB : 1];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int c = c0 + 32 * i;
    g[i] = make_uint4(0, 0, 0, 0);
    if (kGLU) u[i] = make_uint4(0, 0, 0, 0);
    if (c < U) {
      g[i] = __ldg(row + c);
      if (kGLU) u[i] = __ldg(row + U + c);
    }
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int c = c0 + 32 * i;
    float v[8];
    unpack8(g[i], v);
    uint32_t m = 0;  // magnitudes order as their bits do, NaN and inf on top
    if (kGLU) {
      float w[8];
      unpack8(u[i], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = swiglu(v[j], w[j]);
        m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
      }
    } else {  // two at a time
      const uint32_t k2 = 0x7FFF7FFFu;
      m = __vmaxu2(__vmaxu2(g[i].x & k2, g[i].y & k2), __vmaxu2(g[i].z & k2, g[i].w & k2));
      m = max(m & 0xFFFF0000u, m << 16);
    }
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t ex = m >> 23;
    uint32_t byte = ex > 2u ? ex - 2u : 0u;
    uint32_t q = 0;
    if (ex == 255u) {
      byte = 255u;  // a value that is not finite: the block is NaN
    } else if (m) {
      const float inv = __uint_as_float((254u - byte) << 23);  // 2^-X
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= inv;
      q = e2m1x8(v);
    }
    if (c < U) out[c] = q;
    if (c >= U) byte = 127u;  // blocks of a word past the row: 2^0
    // the four blocks of 16 lanes make a word
    uint32_t w = byte << (8 * ((lane >> 2) & 3));
    w |= __shfl_xor_sync(0xffffffffu, w, 4);
    w |= __shfl_xor_sync(0xffffffffu, w, 8);
    if ((lane & 15) == 0 && c < KA * 16) scales[(int64_t)(c >> 4) * P + p] = w;
  }
}

// A row in four-bit pieces (kPieces = 16), each an MXFP4 row of its own.  Piece j
// quantises what pieces 0 .. j - 1 left, exactly known in fp32, with a quarter of
// the scale before: what is below 8 scales leaves less than 2 (1 below 6, else
// saturated), so sixteen leave 2^-32 of the block's maximum: less than fp32 sums of
// the block drop, and nothing of a bf16 value down to 2^-24 of the maximum.  With
// eight (2^-16) nothing was left of a value beside fp32 ones 2^17 times as large:
// the whole result, where the weights of the large ones are zero.  (Scales from each
// remainder's own maximum: 103 instead of 99 us for the layer of 32 tokens of 2880.)

// A warp takes 256 values of a row, as above.  kGLU: fp32 rows [2K], silu(gate)
// * up; else bf16 rows gathered through r2t.  Codes [P * kPieces, K / 2] and
// scale words [ceil(K / 128)][P * kPieces]: row p's pieces are rows p * kPieces ..
template <bool kGLU>
__global__ void __launch_bounds__(32 * kQRows) quantize_pieces_kernel(
    const void* __restrict__ x, int64_t T, int K, const int32_t* __restrict__ r2t, int64_t P,
    uint8_t* __restrict__ codes, uint32_t* __restrict__ scales, int* err) {
  // the product's CTAs fill the SMs: not before this kernel has its own going
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, U = K / 8;
  const int64_t p = (int64_t)blockIdx.x * kQRows + (threadIdx.x >> 5);
  if (p >= P) return;
  const int c = blockIdx.y * 32 + lane;
  float v[8] = {};
  if (kGLU) {
    if (c < U) {
      const float4* g = reinterpret_cast<const float4*>(static_cast<const float*>(x) + p * 2 * K) + 2 * c;
      const float4 a = __ldcg(g), b = __ldcg(g + 1), d = __ldcg(g + K / 4), e = __ldcg(g + K / 4 + 1);
      const float gate[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      const float up[8] = {d.x, d.y, d.z, d.w, e.x, e.y, e.z, e.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = swiglu(gate[j], up[j]);
    }
  } else {
    const int64_t t = token_of_row(r2t, (int32_t)p, T, lane == 0 ? err : nullptr);
    if (c < U) unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + t * K) + c), v);
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const uint32_t ex = m >> 23;
  uint32_t byte = ex > 2u ? ex - 2u : 0u;
  // the four blocks of 16 lanes make a word; a block with a value that is not finite
  // is NaN by its first piece
  uint32_t w = (c >= U ? 127u : ex == 255u ? 255u : byte) << (8 * ((lane >> 2) & 3));
  w |= __shfl_xor_sync(0xffffffffu, w, 4);
  w |= __shfl_xor_sync(0xffffffffu, w, 8);
  // each of them writes a piece's
  static_assert(kPieces == 16, "a lane per piece");
  if ((c >> 4) < (K + 127) / 128)
    scales[(int64_t)(c >> 4) * (P * kPieces) + p * kPieces + (lane & 15)] =
        __vsubus4(w, 0x02020202u * (lane & 15));
  if (c >= U) return;
  if (ex == 255u)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  uint32_t* out = reinterpret_cast<uint32_t*>(codes) + p * kPieces * U + c;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const float inv = __uint_as_float((254u - byte) << 23);
    const float back = byte ? __uint_as_float(byte << 23) : __uint_as_float(0x00400000u);
    uint32_t q = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t two = e2m1x2(v[2 * j] * inv, v[2 * j + 1] * inv);
      const float2 was = e2m1_values(two);
      v[2 * j] = fmaf(-was.x, back, v[2 * j]);
      v[2 * j + 1] = fmaf(-was.y, back, v[2 * j + 1]);
      q |= two << (8 * j);
    }
    out[i * U] = q;
    byte = byte > 2u ? byte - 2u : 0u;
  }
}

// ----------------------------------------------------------------------
// product
// ----------------------------------------------------------------------

constexpr int BM = 128;       // weight rows per tile (MMA M)
constexpr int BH = 192;       // TMEM columns of an accumulator half
constexpr int BT = 256;       // routed rows per tile (MMA N)
constexpr int BKB = 128;      // bytes of codes per row and stage: 256 k
constexpr int BOX = 64;       // routed rows per TMA box, and twice that
constexpr int ST = 4;         // ring stages
constexpr int kThreads = 640;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSfCol = 2 * BH;  // scale columns: a set per ring stage
constexpr uint32_t kSfSet = 8 + 16;
static_assert(kSfCol + ST * kSfSet <= kTmemCols, "accumulators and scales fit TMEM");

constexpr int kABytes = BM * BKB;                 // 16 KB
constexpr int kBBytes = BT * BKB;                 // 32 KB
constexpr int kSfBytes = 8 * (BM + BT);           // 3 KB: 8 scale bytes a row
constexpr int kStageBytes = kABytes + kBBytes + kSfBytes;
static_assert(kStageBytes % 1024 == 0, "swizzle atoms stay aligned");
static_assert(BH <= BT && BT % BOX == 0, "the boxes of a tile fit its stage");
constexpr int kEpiWarps = 8;

struct Smem {
  static constexpr int bars = ST * kStageBytes;
  static constexpr int nbars = 2 * ST + 4 + 1;
  static constexpr int misc = bars + nbars * 8;
  static constexpr int tables = misc + 16;
};
static_assert(1024 + Smem::tables + 8 * (1024 + 1) <= 232448,
              "shared memory for 1024 experts exceeds the 227 KB a CTA can have");

struct A4Problem {
  const uint32_t* xs;      // [ceil(K/128), P] words of four e8m0
  const uint8_t* ws;       // [E, N, K/32] e8m0
  int64_t P, K, N;
  int32_t E;
  const int32_t* offsets;  // [E + 1]
  void* out;               // [P, N] bf16; of rows in pieces [P / 8, N] fp32
  int* err;
};

struct Tile {
  int32_t e, n0, p0, nv;  // expert, first weight row, first routed row, routed rows
};

// Up to BT rows are one tile; more are cut so that the tiles alternate halves.
__device__ __forceinline__ int32_t row_tiles(int32_t cnt) {
  return cnt <= BT ? (cnt + BT - 1) / BT : (cnt + BH - 1) / BH;
}

// ts[e] = tiles of the experts below e, ts[E] = all: per_tile_n times the row tiles
// of each.  Warp 0 scans 32 experts at a time; the block must sync afterwards.
__device__ __forceinline__ void tiles_below(const int32_t* off_s, int32_t E, int32_t per_tile_n,
                                            int32_t* ts) {
  if (threadIdx.x >= 32) return;
  const int lane = threadIdx.x;
  int32_t carry = 0;
  for (int32_t base = 0; base < E; base += 32) {
    const int32_t e = base + lane;
    const int32_t v = e < E ? per_tile_n * row_tiles(off_s[e + 1] - off_s[e]) : 0;
    int32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    if (e < E) ts[e] = carry + incl - v;
    carry += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) ts[E] = carry;
}

// Tile t, for a caller whose tiles only grow: e is the expert of its last one
// (0 at first).  The next is usually a few experts on.
__device__ __forceinline__ Tile tile_info(int64_t t, const int32_t* off, const int32_t* ts,
                                          int32_t E, int32_t& e) {
  int tries = 0;
  while (ts[e + 1] <= t && ++tries < 8) ++e;
  if (ts[e + 1] <= t) {
    int32_t lo = e, hi = E - 1;
    while (lo < hi) {
      const int32_t mid = (lo + hi + 1) >> 1;
      if (ts[mid] <= t) lo = mid; else hi = mid - 1;
    }
    e = lo;
  }
  const int32_t cnt = off[e + 1] - off[e];
  const int32_t rt = row_tiles(cnt);
  int32_t nt = (int32_t)(t - ts[e]), r = 0, per = cnt;
  if (rt > 1) {
    const int32_t u = nt;
    nt = u / rt;
    r = u - nt * rt;
    // rows dealt evenly over the expert's row tiles, in sixteens
    per = ((cnt + rt - 1) / rt + 15) & ~15;
  }
  Tile d;
  d.e = e;
  d.n0 = nt * BM;
  d.p0 = off[e] + r * per;
  d.nv = min(per, cnt - r * per);
  return d;
}

// Which accumulator half a tile of up to BH rows uses: they alternate, so that
// an epilogue overlaps the next tile's MMAs; a larger tile takes both.  The MMA
// thread and the epilogue step identical copies.
struct AccSched {
  uint32_t h = 0;
  uint32_t use0 = 0, use1 = 0;
  __device__ __forceinline__ uint32_t phase(uint32_t k) const { return (k ? use1 : use0) & 1u; }
  __device__ __forceinline__ void next(bool both) {
    if (both) {
      ++use0;
      ++use1;
    } else {
      if (h) ++use1; else ++use0;
      h ^= 1u;
    }
  }
};

// Instruction descriptor, kind::mxf4: A and B e2m1 (K-major), e8m0 scales,
// fp32 D; sf: which 16-bit half of a scale word (two 32-blocks) is used.
__device__ __forceinline__ uint32_t idesc_mxf4(uint32_t N, uint32_t sf) {
  return (sf << 4)              // B scale id
         | (1u << 7)            // A format: e2m1
         | (1u << 10)           // B format: e2m1
         | ((N >> 3) << 17)     // N / 8
         | (1u << 23)           // scale format: e8m0
         | ((uint32_t)(BM >> 4) << 24)  // M / 16
         | (sf << 29);          // A scale id
}

// D[tmem] (+)= (A * 2^sfa)[smem] * (B * 2^sfb)[smem]^T over 64 k.
__device__ __forceinline__ void tc_mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                            uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// 8 or 16 columns of this warp's 32 TMEM lanes from registers; the registers
// belong to the store until the wait, so that sits in the same statement.
__device__ __forceinline__ void tmem_store_8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void tmem_store_16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};\n"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// One lane of the warp, the same for every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t v;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(v));
  return v != 0;
}

// Barrier of the four warps of a scale group; whether all of them say `ok` (so
// that after a wait that ran out they leave together).
__device__ __forceinline__ bool group_sync(int group, bool ok) {
  uint32_t v;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n bar.red.and.pred q, %1, 128, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(v)
      : "r"(1 + group), "r"((uint32_t)ok)
      : "memory");
  return v != 0;
}

// Eight scale bytes of a weight row, of which the first `valid` exist: rows have
// any pitch, so these are the one or two aligned 8-byte words around them (bytes,
// where a word reaches past the matrix [base, end)).  get() shifts them into
// place when they are needed: done at once, it would wait for the loads.
struct RowScales {
  uint64_t lo, hi;
  int shift, valid;
  __device__ __forceinline__ void load(const uint8_t* p, int n, const uint8_t* base,
                                       const uint8_t* end) {
    const int o = (int)(reinterpret_cast<uintptr_t>(p) & 7u);
    const uint8_t* q = p - o;
    const bool two = o + min(n, 8) > 8;
    valid = n;
    shift = 8 * o;
    if (q >= base && q + (two ? 16 : 8) <= end) {
      lo = __ldg(reinterpret_cast<const uint64_t*>(q));
      if (two) hi = __ldg(reinterpret_cast<const uint64_t*>(q) + 1);
    } else {
      shift = 0;
      lo = 0;
      for (int i = 0; i < min(n, 8); ++i) lo |= (uint64_t)__ldg(p + i) << (8 * i);
    }
  }
  // Bytes that do not exist read as 127 (2^0: their codes are zeros).
  __device__ __forceinline__ uint2 get() const {
    uint64_t v = lo;
    if (shift) v = (lo >> shift) | (hi << (64 - shift));
    if (valid < 8) {
      const uint64_t m = valid > 0 ? ~0ull << (8 * valid) : ~0ull;
      v = (v & ~m) | (0x7F7F7F7F7F7F7F7Full & m);
    }
    return make_uint2((uint32_t)v, (uint32_t)(v >> 32));
  }
};

// The experts' first rows, checked: 0 at first, never falling, at most P.  The
// last may be below P (rows past it belong to no expert and are not written).
// Anything else is clamped to a running maximum and recorded.
__device__ __forceinline__ void load_offsets(const int32_t* offsets, int32_t E, int64_t P,
                                             int32_t* off_s, int* err) {
  int bad = 0;
  for (int32_t e = threadIdx.x; e <= E; e += kThreads) {
    const int32_t v = __ldg(offsets + e);
    off_s[e] = v;
    bad |= v < 0 || v > P || (e == 0 && v != 0) || (e < E && __ldg(offsets + e + 1) < v);
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) {
      int32_t last = 0;
      for (int32_t e = 0; e <= E; ++e) {
        if (e > 0) last = max(last, (int32_t)min((int64_t)off_s[e], P));
        off_s[e] = last;
      }
      raise_error(err, GBW_DEVERR_OFFSETS);
    }
    __syncthreads();
  }
}

// R: rows of x that make one of the output, 1 or kPieces.
template <int R>
__global__ void __launch_bounds__(kThreads, 1)
gemm_a4_kernel(const A4Problem pb, const __grid_constant__ CUtensorMap tmw,
               const __grid_constant__ CUtensorMap tmx, const __grid_constant__ CUtensorMap tmx2) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Smem::bars);
  uint64_t* full = bars;
  uint64_t* empty = full + ST;
  uint64_t* acc_full = empty + ST;     // [2]
  uint64_t* acc_empty = acc_full + 2;  // [2]
  uint64_t* mma_done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Smem::misc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + Smem::misc + 4);
  int32_t* off_s = reinterpret_cast<int32_t*>(smem + Smem::tables);
  int32_t* ts_s = off_s + (pb.E + 1);

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int32_t E = pb.E;
  const int64_t N = pb.N;
  const int32_t KB = (int32_t)(pb.K / 2);         // bytes of codes per row
  const int32_t KS = (int32_t)(pb.K / 32);        // scale bytes per row
  const int NS = (KB + BKB - 1) / BKB;            // stages per tile
  const int32_t ntn = (int32_t)((N + BM - 1) / BM);

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) { mbar_init(&full[i], 1 + 4); mbar_init(&empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&acc_full[i], 1); mbar_init(&acc_empty[i], kEpiWarps); }
    mbar_init(mma_done, 1);
    *abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmw);
    tma_prefetch_desc(&tmx);
    tma_prefetch_desc(&tmx2);
  }
  // Rows in pieces: the kernel before this one lets it launch only after the one
  // that wrote the offsets is complete, so only what reads the pieces or writes
  // the output waits; the first weights are on their way by then.
  if (R == 1) grid_dependency_wait();
  load_offsets(pb.offsets, E, pb.P / R, off_s, pb.err);
  if (R > 1) {
    for (int i = threadIdx.x; i <= E; i += kThreads) off_s[i] *= R;
    __syncthreads();
  }
  tiles_below(off_s, E, ntn, ts_s);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int64_t ntiles = ts_s[E];
  int32_t at_e = 0;  // tile_info's place

  if (warp == 0) {
    // ---------------- codes: weights and routed rows ----------------
    {
      const bool leader = elect_one();
      uint32_t g = 0, s = 0, ph = 1;
      bool ok = true;
      // stages whose weights are loaded ahead of the wait
      const uint32_t ahead = R > 1 && blockIdx.x < ntiles ? (uint32_t)min(NS, ST) : 0;
      if (R > 1) {
        if (ahead && leader) {
          int32_t e = 0;
          const Tile d = tile_info(blockIdx.x, off_s, ts_s, E, e);
          for (uint32_t i = 0; i < ahead; ++i) {
            mbar_arrive_expect_tx(&full[i], kABytes + (uint32_t)((d.nv + BOX - 1) / BOX) * (BOX * BKB));
            tma_load_2d(smem + i * kStageBytes, &tmw, (int)i * BKB, (int32_t)((int64_t)d.e * N + d.n0), &full[i]);
          }
        }
        __syncwarp();
        grid_dependency_wait();
      }
      for (int64_t t = blockIdx.x; t < ntiles && ok; t += gridDim.x) {
        Tile d = tile_info(t, off_s, ts_s, E, at_e);
        d.nv = __shfl_sync(0xffffffffu, d.nv, 0);
        d.p0 = __shfl_sync(0xffffffffu, d.p0, 0);
        const int32_t wrow = __shfl_sync(0xffffffffu, (int32_t)((int64_t)d.e * N + d.n0), 0);
        const int boxes = (d.nv + BOX - 1) / BOX;
        const uint32_t bytes = kABytes + (uint32_t)boxes * (BOX * BKB);
        for (int ks = 0; ks < NS; ++ks, ++g) {
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], ph, abort, pb.err));
          if (!ok) break;
          if (leader) {
            uint8_t* st = smem + s * kStageBytes;
            if (g >= ahead) {
              mbar_arrive_expect_tx(&full[s], bytes);
              tma_load_2d(st, &tmw, ks * BKB, wrow, &full[s]);
            }
            uint8_t* dst = st + kABytes;
            int p0 = d.p0, n = boxes;
            for (; n >= 2; n -= 2, dst += 2 * BOX * BKB, p0 += 2 * BOX)
              tma_load_2d(dst, &tmx2, ks * BKB, p0, &full[s]);
            if (n) tma_load_2d(dst, &tmx, ks * BKB, p0, &full[s]);
          }
          if (++s == ST) { s = 0; ph ^= 1u; }
        }
      }
      grid_launch_dependents();  // the next kernel's launch overlaps the last tiles
      if (leader && *abort)
        for (uint32_t i = (g > ST ? g - ST : 0); i < max(g, ahead); ++i) mbar_drain(&full[i % ST], (i / ST) & 1u);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    // One thread issues everything, so its instructions count: descriptors are
    // built once and advance by constants, a whole stage is unrolled.
    {
      const bool leader = elect_one();
      uint32_t s = 0, ph = 0;
      bool ok = true;
      AccSched acc;
      auto all = [](bool v) { return __all_sync(0xffffffffu, v) != 0; };
      const uint64_t adesc0 = make_sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t bdesc0 = make_sdesc_sw128(smem_u32(smem + kABytes), 16, 1024);
      for (int64_t t = blockIdx.x; t < ntiles && ok; t += gridDim.x) {
        Tile d = tile_info(t, off_s, ts_s, E, at_e);
        d.nv = __shfl_sync(0xffffffffu, d.nv, 0);
        const bool both = d.nv > BH;
        const uint32_t h0 = both ? 0u : acc.h;
        const uint32_t id = idesc_mxf4((uint32_t)(d.nv + 15) & ~15u, 0);
        constexpr uint32_t kUpper = (2u << 4) | (2u << 29);  // the scale words' upper halves
        const uint32_t d0 = tmem + h0 * BH;
        if (!(ok = all(mbar_wait(&acc_empty[h0], acc.phase(h0) ^ 1u, abort, pb.err)))) break;
        if (both && !(ok = all(mbar_wait(&acc_empty[1], acc.phase(1) ^ 1u, abort, pb.err)))) break;
        for (int ks = 0; ks < NS; ++ks) {
          if (!(ok = all(mbar_wait(&full[s], ph, abort, pb.err)))) break;
          tc_fence_after();
          const uint64_t so = (uint64_t)((s * kStageBytes) >> 4);
          const uint64_t ad = adesc0 + so, bd = bdesc0 + so;
          const uint32_t sf = tmem + kSfCol + s * kSfSet;
          // the two 64-k steps of 128-k scale atom a
          auto atom = [&](int a, bool second) __attribute__((always_inline)) {
            tc_mma_mxf4(d0, ad + 4 * a, bd + 4 * a, id, sf + a * 4, sf + 8 + a * 8, a > 0 || ks > 0);
            if (second)
              tc_mma_mxf4(d0, ad + 4 * a + 2, bd + 4 * a + 2, id | kUpper, sf + a * 4, sf + 8 + a * 8, 1u);
          };
          const int nk = (KB - ks * BKB + 31) / 32;  // 64-k steps left
          if (leader) {
            if (nk >= 4) {
              atom(0, true);
              atom(1, true);
            } else {
              atom(0, nk > 1);
              if (nk > 2) atom(1, false);
            }
            tc_commit(&empty[s]);
          }
          if (++s == ST) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        if (leader) {
          tc_commit(&acc_full[h0]);
          if (both) tc_commit(&acc_full[1]);
        }
        acc.next(both);
      }
      if (leader) {
        tc_commit(mma_done);
        mbar_drain(mma_done, 0);
      }
      __syncwarp();
    }
  } else if (warp >= 4 && warp < 12) {
    // ---------------- scales ----------------
    // two groups of four warps take alternate stages: what bounds them is the
    // instructions of one stage.  Thread i of a group loads the scales of weight
    // row i and routed rows i, i + 128 of the tile, two stages ahead;
    // through shared memory every warp gets them all, since TMEM wants row r in
    // lane r % 32, column r / 32 of each of the four 32-lane quarters, and a warp
    // writes its own quarter.  (tcgen05.cp does the same from shared memory, but
    // held up the MMAs behind it: 45 of 220 us at 8192 rows x 5760 x 2880.)
    const int group = (warp - 4) >> 2, i = ((warp - 4) & 3) * 32 + lane;
    const uint2 ones = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    const uint8_t* wend = pb.ws + (int64_t)E * N * KS;
    const uint8_t* wp = nullptr;                    // the weight row's scales, or null
    const uint32_t* xp[2] = {nullptr, nullptr};     // the routed rows' first words, or null
    const int KA = (KS + 3) / 4;                    // words of a routed row
    int64_t t = blockIdx.x;                         // stage to load: tile and step
    int ks = 0;
    auto open = [&]() __attribute__((always_inline)) {
      const Tile d = tile_info(t, off_s, ts_s, E, at_e);
      wp = d.n0 + i < N ? pb.ws + ((int64_t)d.e * N + d.n0 + i) * KS : nullptr;
#pragma unroll
      for (int q = 0; q < 2; ++q) xp[q] = i + 128 * q < d.nv ? pb.xs + d.p0 + i + 128 * q : nullptr;
    };
    // the scales of the group's next stage
    RowScales w = {0, 0, 0, 0};
    uint2 x[2] = {ones, ones};
    bool on = false;
    auto step = [&]() __attribute__((always_inline)) {  // to the next stage
      if (++ks == NS) {
        ks = 0;
        t += gridDim.x;
        if (t < ntiles) open();
      }
    };
    auto load = [&]() __attribute__((always_inline)) {
      on = t < ntiles;
      if (!on) return;
      if (wp) w.load(wp + 8 * ks, KS - 8 * ks, pb.ws, wend);
      else w.valid = 0;
      const int64_t off = (int64_t)(2 * ks) * pb.P;
      const bool second = 2 * ks + 1 < KA;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        x[q] = ones;
        if (xp[q]) {
          x[q].x = __ldg(xp[q] + off);
          if (second) x[q].y = __ldg(xp[q] + off + pb.P);
        }
      }
      step();
      step();
    };
    uint32_t s = (uint32_t)group, ph = 0;
    if (R > 1) grid_dependency_wait();
    if (t < ntiles) open();
    if (group) step();
    load();
    while (on) {
      const bool ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], ph ^ 1u, abort, pb.err));
      tc_fence_after();
      // 8 bytes a row: 128 weight rows, then the routed rows
      uint2* sf = reinterpret_cast<uint2*>(smem + s * kStageBytes + kABytes + kBBytes);
      uint2* sb = sf + BM;
      sf[i] = w.get();
#pragma unroll
      for (int q = 0; q < 2; ++q) sb[i + 128 * q] = x[q];
      load();
      if (!group_sync(group, ok)) break;
      const uint32_t sc = tmem + (((uint32_t)warp & 3u) << 21) + kSfCol + s * kSfSet;
      {
        uint32_t r[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint2 u = sf[c * 32 + lane];
          r[c] = u.x;
          r[4 + c] = u.y;
        }
        tmem_store_8(sc, r);
      }
      {
        uint32_t r[16];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint2 u = sb[c * 32 + lane];
          r[c] = u.x;
          r[8 + c] = u.y;
        }
        tmem_store_16(sc + 8, r);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[s]);
      s += 2;
      if (s >= ST) { s -= ST; ph ^= 1u; }
    }
  } else if (warp >= 12) {
    // ---------------- epilogue ----------------
    // warp quarter q reads weight rows 32 q .. of the tile (TMEM lanes); the two
    // warps of a quarter take alternate 32-row pieces of the routed rows.  Lanes
    // 2 i and 2 i + 1 trade halves, so that each stores words of two weight rows:
    // the even lane those of the even routed rows, 64 bytes a row and warp.
    const uint32_t q = (uint32_t)warp & 3u;
    const int mine = (warp - 12) >> 2, odd = lane & 1;
    const uint32_t keep_sel = odd ? 0x7632u : 0x5410u, send_sel = odd ? 0x5410u : 0x7632u;
    const uint32_t lo_sel = odd ? 0x1054u : 0x5410u, hi_sel = odd ? 0x3276u : 0x7632u;
    AccSched acc;
    bool ok = true;
    if (R > 1) grid_dependency_wait();
    for (int64_t t = blockIdx.x; t < ntiles && ok; t += gridDim.x) {
      const Tile d = tile_info(t, off_s, ts_s, E, at_e);
      const bool both = d.nv > BH;
      const uint32_t h = both ? 0u : acc.h;
      ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[h], acc.phase(h), abort, pb.err));
      if (ok && both)
        ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[1], acc.phase(1), abort, pb.err));
      if (!ok) break;
      tc_fence_after();
      const int64_t n = d.n0 + (int64_t)(q * 32 + (R > 1 ? lane : lane & 30));
      uint16_t* dst = static_cast<uint16_t*>(pb.out) + (int64_t)(d.p0 + odd) * N + n;
      float* sums = static_cast<float*>(pb.out) + (int64_t)(d.p0 / R) * N + n;
      const uint32_t taddr = tmem + ((q * 32u) << 16) + h * BH;
#pragma unroll 1
      for (int c = mine * 32; c < d.nv; c += 64) {
        uint32_t r[32];
        tmem_load_32x32b_x32(taddr + c, r);
        if (R > 1) {  // a row's pieces, the smallest first
#pragma unroll
          for (int j = 0; j < 32; j += R) {
            float v = __uint_as_float(r[j + R - 1]);
#pragma unroll
            for (int i = R - 2; i >= 0; --i) v += __uint_as_float(r[j + i]);
            if (n < N && c + j < d.nv) sums[(int64_t)((c + j) / R) * N] = v;
          }
          continue;
        }
        uint16_t* to = dst + (int64_t)c * N;
        const int left = n < N ? d.nv - c - odd : 0;
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const uint32_t a = pack_bf16x2(__uint_as_float(r[j]), __uint_as_float(r[j + 1]));
          const uint32_t b = pack_bf16x2(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3]));
          const uint32_t keep = prmt(a, b, keep_sel);
          const uint32_t got = __shfl_xor_sync(0xffffffffu, prmt(a, b, send_sel), 1);
          if (j < left) *reinterpret_cast<uint32_t*>(to + j * N) = prmt(keep, got, lo_sel);
          if (j + 2 < left) *reinterpret_cast<uint32_t*>(to + (j + 2) * N) = prmt(keep, got, hi_sel);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&acc_empty[h]);
        if (both) mbar_arrive(&acc_empty[1]);
      }
      acc.next(both);
    }
  }

  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

cudaError_t launch_quantize_rows(const uint16_t* x, int64_t T, int64_t K, const int32_t* r2t,
                                 int64_t P, bool glu, uint8_t* codes, uint8_t* scales, int* err,
                                 cudaStream_t s) {
  if (P == 0) return cudaSuccess;
  uint32_t* words = reinterpret_cast<uint32_t*>(scales);
  auto grid = [&](int64_t units) {
    return dim3((unsigned)((P + kQRows - 1) / kQRows), (unsigned)((K + 256 * units - 1) / (256 * units)));
  };
  return glu ? launch_kernel<quantize_rows_kernel<true>>(grid(kUnits<true>), 32 * kQRows, 0, s, false, x,
                                                         T, (int)K, r2t, P, codes, words, err)
             : launch_kernel<quantize_rows_kernel<false>>(grid(kUnits<false>), 32 * kQRows, 0, s, false, x,
                                                          T, (int)K, r2t, P, codes, words, err);
}

cudaError_t launch_quantize_pieces(const void* x, int64_t T, int64_t K, const int32_t* r2t, int64_t P,
                                   bool glu, uint8_t* codes, uint32_t* scales, int* err,
                                   cudaStream_t s) {
  const dim3 grid((unsigned)((P + kQRows - 1) / kQRows), (unsigned)((K + 255) / 256));
  // The rows of x start behind a router that has a CTA on most SMs: left to
  // itself, the scheduler packs these CTAs onto the others (9 instead of 4 us for
  // 128 rows of 2880).  Shared memory that nothing uses allows four an SM.
  constexpr size_t kSpread = 48 * 1024;
  return glu ? launch_kernel<quantize_pieces_kernel<true>>(grid, 32 * kQRows, 0, s, true, x, T, (int)K,
                                                           r2t, P, codes, scales, err)
             : launch_kernel<quantize_pieces_kernel<false>>(grid, 32 * kQRows, kSpread, s, true, x, T, (int)K,
                                                            r2t, P, codes, scales, err);
}

namespace {

template <int R>
cudaError_t launch_gemm_t(const uint8_t* xq, const uint8_t* xs, int64_t P, int64_t K,
                           const uint8_t* w, const uint8_t* ws, int32_t E, int64_t N,
                           const int32_t* offsets, void* out, int* err, int num_sms,
                           cudaStream_t s) {
  if (P == 0) return cudaSuccess;
  CUtensorMap tmw, tmx;
  cudaError_t e = make_map_2d(&tmw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, (uint64_t)K / 2,
                              (uint64_t)E * (uint64_t)N, (uint64_t)K / 2, BKB, BM,
                              CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  e = make_map_2d(&tmx, CU_TENSOR_MAP_DATA_TYPE_UINT8, xq, (uint64_t)K / 2, (uint64_t)P,
                  (uint64_t)K / 2, BKB, BOX, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  CUtensorMap tmx2;
  e = make_map_2d(&tmx2, CU_TENSOR_MAP_DATA_TYPE_UINT8, xq, (uint64_t)K / 2, (uint64_t)P,
                  (uint64_t)K / 2, BKB, 2 * BOX, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  const A4Problem pb{reinterpret_cast<const uint32_t*>(xs), ws, P, K, N, E, offsets, out, err};
  constexpr size_t most = 1024 + Smem::tables + 8 * (1024 + 1);
  e = opt_in_smem<gemm_a4_kernel<R>>(most);
  if (e != cudaSuccess) return e;
  const size_t smem = 1024 + Smem::tables + 8 * (size_t)(E + 1);
  return launch_kernel<gemm_a4_kernel<R>>(num_sms, kThreads, smem, s, true, pb, tmw, tmx, tmx2);
}

}  // namespace

cudaError_t launch_gemm_a4(const uint8_t* xq, const uint8_t* xs, int64_t P, int64_t K,
                           const uint8_t* w, const uint8_t* ws, int32_t E, int64_t N,
                           const int32_t* offsets, uint16_t* out, int* err, int num_sms,
                           cudaStream_t s) {
  return launch_gemm_t<1>(xq, xs, P, K, w, ws, E, N, offsets, out, err, num_sms, s);
}

cudaError_t launch_gemm_pieces(const uint8_t* xq, const uint32_t* xs, int64_t P, int64_t K,
                               const uint8_t* w, const uint8_t* ws, int32_t E, int64_t N,
                               const int32_t* offsets, float* out, int* err, int num_sms,
                               cudaStream_t s) {
  return launch_gemm_t<kPieces>(xq, reinterpret_cast<const uint8_t*>(xs), P * kPieces, K, w, ws, E, N,
                                offsets, out, err, num_sms, s);
}

}  // namespace gbw
