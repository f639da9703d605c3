// route.cu -- what stands between a router and the grouped expert calls:
// the choice of k experts per token with its softmax weights, the stable
// expert-sorted plan that the grouped kernels read, and the weighted combine
// of the routed rows back into tokens; each with its gradient.
//
//   l = logits[t, :], NaN counted as -inf; ids = the k largest (ties: lowest
//   index); m = max l; p_e = exp(l_e - m) (1 where l_e == m, so infinite
//   maxima share); w_s = p_ids[s] / sum of p over the chosen (renormalised)
//   or over all experts; a row without any logit above -inf has w = 0.
//   Sorting the slots (t, s) by expert, stably, gives expert_offsets,
//   row_to_token, row_of_slot and slot_of_row.
//   Gradient: dl_e = [e = ids[s]] w_s dw_s - q_e * sum_s w_s dw_s, where q is w
//   on the chosen experts (renormalised) or p / sum p on all.
//
// Bound: these are a few hundred bytes per token; launches and the latency
// of dependent steps count, not bandwidth.  One warp holds a token's logits
// in registers (E / 32 each) and takes the maxima with two warp reductions
// per choice; up to kSingleTokens tokens are routed and sorted by one CTA in
// one launch, more by two kernels (choose + count, then place), the second
// launched early behind the first (a plain launch: 1 us more).  8 of 128 experts
// for 4 tokens: 4.3 us on the device; for 4096: 8.4; 4 of 32 for 16411 tokens
// with the gradient: 17.8.  On the host a call takes 7 to 15 us, what bounds the
// small ones.
#include <type_traits>

#include "common.cuh"
#include "launch.cuh"
#include "route.cuh"

namespace gbw {
namespace {

constexpr int kWarps = 32;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxE = 1024;
constexpr int64_t kSingleTokens = 128;

__device__ __forceinline__ void store_logit(uint16_t* p, float v) {
  *p = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }

// Exclusive scan of v over the block's threads (kThreads of them); `part` has
// kWarps entries.  Returns the sum over lower threads.
__device__ __forceinline__ int block_exclusive(int v, int* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, lane < warp ? part[lane] : 0) + incl - v;
}

// The slots [slot0, slot0 + n) of a CTA: each warp owns a contiguous run
// [i0, i1) of them and walks it 32 at a time, so equal experts keep their slot
// order.  whist[w * E + e] counts warp w's slots of expert e, then is the row of
// its next one.
struct Slots {
  int64_t slot0;
  int nw, i0, i1;
  __device__ __forceinline__ Slots(int64_t s, int n) : slot0(s) {
    const int warp = threadIdx.x >> 5;
    nw = min(kWarps, (n + 31) / 32);
    const int seg = nw ? (n + nw - 1) / nw : 0;
    i0 = min(n, warp * seg);
    i1 = warp < nw ? min(n, i0 + seg) : i0;
  }
  // `id`: expert of slot i0 + lane (the only one of most lanes)
  __device__ __forceinline__ void count(const RouteProblem& p, int id, int* whist) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = i0 + lane; i < i1; i += 32) {
      atomicAdd(&whist[warp * p.E + id], 1);
      if (i + 32 < i1) id = p.ids[slot0 + i + 32];
    }
  }
  // Thread e: the rows of expert e from `run` on, warp after warp.
  __device__ __forceinline__ void scan(int E, int run, int* whist) const {
    for (int w0 = 0; w0 < nw; w0 += 8) {
      int c[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = w0 + j < nw ? whist[(w0 + j) * E + threadIdx.x] : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (w0 + j < nw) whist[(w0 + j) * E + threadIdx.x] = run;
        run += c[j];
      }
    }
  }
  __device__ __forceinline__ void place(const RouteProblem& p, int id, int* whist) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = p.E;
    for (int i = i0; i < i1; i += 32) {
      const bool on = i + lane < i1;
      const int64_t slot = slot0 + i + lane;
      const unsigned same = __match_any_sync(0xffffffffu, on ? id : -1 - lane);
      const int rank = __popc(same & ((1u << lane) - 1u));
      const int at = on ? whist[warp * E + id] + rank : 0;
      __syncwarp();
      if (on) {
        if (rank == 0) whist[warp * E + id] += __popc(same);
        p.row_of_slot[slot] = at;
        p.row_to_token[at] = (int32_t)((uint32_t)slot / (uint32_t)p.k);
        p.slot_of_row[at] = (int32_t)slot;
        if (i + 32 + lane < i1) id = p.ids[slot + 32];
      }
      __syncwarp();
    }
  }
};

// Chooses the experts of tokens [b * per, (b + 1) * per) and counts them;
// kSingle (one CTA): sorts and places them too.
template <typename TL, int NPL, bool kSingle, bool kNanRows = false>
__global__ void __launch_bounds__(kThreads) route_choose(const RouteProblem p, const int per) {
  extern __shared__ int sm[];
  // kSingle: part [kWarps], whist [kWarps][E]; else count [E]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = p.E, k = p.k;
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t t0 = (int64_t)blockIdx.x * per;
  const int n = (int)max((int64_t)0, min((int64_t)per, p.T - t0));
  int* const hist = kSingle ? sm + kWarps : sm;
  const Slots slots(t0 * k, n * k);
  for (int i = threadIdx.x; i < (kSingle ? slots.nw * E : E); i += kThreads) hist[i] = 0;
  if (!kSingle) __syncthreads();
  for (int i = warp; i < n; i += kWarps) {
    const int64_t t = t0 + i;
    int id = 0;
    float w = 0.0f;
    choose<TL, NPL, kNanRows>(reinterpret_cast<const TL*>(p.logits) + t * E, E, k, p.renorm, lane, id, w);
    if (lane < k) {
      p.ids[t * k + lane] = id;
      p.weights[t * k + lane] = w;
      if (!kSingle) atomicAdd(&hist[id], 1);
    }
  }
  __syncthreads();
  const int e = threadIdx.x;  // E <= kThreads
  if (kSingle) {
    const int id = slots.i0 + lane < slots.i1 ? p.ids[slots.slot0 + slots.i0 + lane] : 0;
    slots.count(p, id, hist);
    __syncthreads();
    int c = 0;
    if (e < E)
      for (int w = 0; w < slots.nw; ++w) c += hist[w * E + e];
    const int at = block_exclusive(c, sm);
    if (e < E) {
      p.offsets[e] = at;
      if (e == E - 1) p.offsets[E] = at + c;
      slots.scan(E, at, hist);
    }
    __syncthreads();
    slots.place(p, id, hist);
  } else if (e < E) {
    p.hist[(int64_t)blockIdx.x * E + e] = hist[e];
  }
}

// Second kernel: rows of this CTA's slots from all CTAs' counts.
__global__ void __launch_bounds__(kThreads) route_place(const RouteProblem p, const int per) {
  extern __shared__ int sm[];
  int* part = sm;                // [kWarps]
  int* red = part + kWarps;      // [2][kThreads]
  int* whist = red + 2 * kThreads;
  const int E = p.E, lane = threadIdx.x & 31;
  int lg = 5;  // threads of one part: a power of two >= E
  while ((1 << lg) < E) ++lg;
  const int parts = kThreads >> lg, me = threadIdx.x >> lg, e = threadIdx.x & ((1 << lg) - 1);
  const int64_t t0 = (int64_t)blockIdx.x * per;
  const int n = (int)max((int64_t)0, min((int64_t)per, p.T - t0));
  const Slots slots(t0 * p.k, n * p.k);
  for (int i = threadIdx.x; i < slots.nw * E; i += kThreads) whist[i] = 0;
  grid_dependency_wait();
  const int id = slots.i0 + lane < slots.i1 ? p.ids[slots.slot0 + slots.i0 + lane] : 0;
  int total = 0, before = 0;
  if (e < E) {
#pragma unroll 8
    for (int b = me; b < (int)gridDim.x; b += parts) {
      const int c = p.hist[(int64_t)b * E + e];
      total += c;
      before += b < (int)blockIdx.x ? c : 0;
    }
  }
  red[threadIdx.x] = total;
  red[kThreads + threadIdx.x] = before;
  __syncthreads();
  slots.count(p, id, whist);
  total = before = 0;
  if (threadIdx.x < (unsigned)E) {
#pragma unroll 8
    for (int i = 0; i < parts; ++i) {
      total += red[(i << lg) + threadIdx.x];
      before += red[kThreads + (i << lg) + threadIdx.x];
    }
  }
  const int at = block_exclusive(total, part);  // its barrier completes whist
  if (threadIdx.x < (unsigned)E) {
    if (blockIdx.x == 0) {
      p.offsets[threadIdx.x] = at;
      if ((int)threadIdx.x == E - 1) p.offsets[E] = at + total;
    }
    slots.scan(E, at + before, whist);
  }
  __syncthreads();
  slots.place(p, id, whist);
}

// One warp per token: dlogits row built in shared memory, written once.
template <typename TL>
__global__ void __launch_bounds__(256) route_bwd_kernel(
    const TL* __restrict__ logits, int64_t T, int E, int k, int renorm,
    const int32_t* __restrict__ ids, const float* __restrict__ weights,
    const float* __restrict__ dweights, TL* __restrict__ dlogits, int* err) {
  extern __shared__ float rows[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = rows + warp * E;
  const int64_t nw = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp; t < T; t += nw) {
    float w = 0.0f, dw = 0.0f;
    int id = -1;
    if (lane < k) {
      w = __ldg(weights + t * k + lane);
      dw = __ldg(dweights + t * k + lane);
      id = __ldg(ids + t * k + lane);
      if (id < 0 || id >= E) {
        raise_error(err, GBW_DEVERR_ROUTE);
        id = -1;
      }
    }
    // a weight of zero passes nothing on, whatever dw holds, nor does a bad id
    const float wdw = w == 0.0f || id < 0 ? 0.0f : w * dw;
    const float sum = warp_sum(wdw);
    if (renorm) {
      for (int e = lane; e < E; e += 32) row[e] = 0.0f;
    } else {
      float m = __int_as_float(0xFF800000);
      for (int e = lane; e < E; e += 32) {
        const float v = no_nan(load_logit(logits + t * E + e));
        row[e] = v;
        m = fmaxf(m, v);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      float all = 0.0f;
      for (int e = lane; e < E; e += 32) {
        const float q = m == __int_as_float(0xFF800000) ? 0.0f : share(row[e], m);
        row[e] = q;
        all += q;
      }
      all = warp_sum(all);
      const float f = all > 0.0f ? -sum / all : 0.0f;
      for (int e = lane; e < E; e += 32) row[e] *= f;
    }
    __syncwarp();
    if (id >= 0) atomicAdd(&row[id], renorm ? wdw - w * sum : wdw);
    __syncwarp();
    for (int e = lane; e < E; e += 32) store_logit(dlogits + t * E + e, row[e]);
    __syncwarp();
  }
}

// Row of one slot, or -1 (contributes nothing) when it is out of range.
__device__ __forceinline__ int32_t slot_row(const int32_t* row_of_slot, int64_t slot, int64_t P,
                                            int* err) {
  const int32_t r = __ldg(row_of_slot + slot);
  if (r >= 0 && r < P) return r;
  raise_error(err, GBW_DEVERR_ROUTE);
  return -1;
}

// Eight columns of a row, bf16 or fp32, read past L1.
template <typename TY>
struct Unit;
template <>
struct Unit<uint16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void add_to(float (&a)[8], float w) const {
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[2 * i] = fmaf(w, __uint_as_float(x[i] << 16), a[2 * i]);
      a[2 * i + 1] = fmaf(w, __uint_as_float(x[i] & 0xFFFF0000u), a[2 * i + 1]);
    }
  }
};
template <>
struct Unit<float> {
  float4 v[2];
  __device__ __forceinline__ void load(const float* p) {
    v[0] = __ldcg(reinterpret_cast<const float4*>(p));
    v[1] = __ldcg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void add_to(float (&a)[8], float w) const {
    const float x[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = fmaf(w, x[i], a[i]);
  }
};

// out[t, :] = sum_s w[t, s] * y[row(t, s), :], summed in slot order in fp32.
// A thread owns 8 columns of one token; up to four rows' loads are in flight.
// Each row is read once, so past L1.  A slot of weight 0 adds nothing, whatever
// its row holds: the row is not read.  Bound by memory: 2048 tokens, 4 rows of
// 2880 each: 12.5 us, 4.7 TB/s.
template <typename TY>
__global__ void __launch_bounds__(256) combine_kernel(
    const TY* __restrict__ y, int64_t P, uint32_t units, const int32_t* __restrict__ rows,
    const float* __restrict__ weights, int64_t n, int k, uint16_t* __restrict__ out, int* err) {
  const int64_t H = (int64_t)units * 8;
  grid_dependency_wait();
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = i / units;
    const int64_t c = (i - t * units) * 8;
    float a[8] = {};
    for (int s0 = 0; s0 < k; s0 += 4) {
      Unit<TY> v[4];
      float w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = {};
        w[j] = 0.0f;
        if (s0 + j < k) {
          const int32_t r = slot_row(rows, t * k + s0 + j, P, err);
          if (r >= 0) {
            w[j] = weights ? __ldg(weights + t * k + s0 + j) : 1.0f;
            if (w[j] != 0.0f) v[j].load(y + r * H + c);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j].add_to(a, w[j]);
    }
    uint4 o;
    o.x = pack_bf16x2(a[0], a[1]);
    o.y = pack_bf16x2(a[2], a[3]);
    o.z = pack_bf16x2(a[4], a[5]);
    o.w = pack_bf16x2(a[6], a[7]);
    __stcs(reinterpret_cast<uint4*>(out + t * H + c), o);
  }
}

// One warp per slot: dy[row] = w * dout[t], dw = <y[row], dout[t]>.  Only the
// slot that slot_of_row names writes a row.  Bound by memory: with the combine,
// 4096 tokens, 8 rows of 2048 each: 81 us, 5.4 TB/s (streaming hints or four
// units of a row ahead: 86).
__global__ void __launch_bounds__(256) combine_bwd_kernel(
    const uint16_t* __restrict__ dout, const uint16_t* __restrict__ y, int64_t P, int32_t units,
    const int32_t* __restrict__ rows, const int32_t* __restrict__ slots,
    const float* __restrict__ weights, int64_t n, int k, uint16_t* __restrict__ dy,
    float* __restrict__ dweights, int* err) {
  const int lane = threadIdx.x & 31;
  const int64_t nw = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t slot = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); slot < n;
       slot += nw) {
    const int64_t t = slot / k;
    int32_t r = slot_row(rows, slot, P, lane == 0 ? err : nullptr);
    if (r >= 0 && __ldg(slots + r) != slot) {
      if (lane == 0) raise_error(err, GBW_DEVERR_ROUTE);
      r = -1;
    }
    float dot = 0.0f;
    if (r >= 0) {
      const float w = __ldg(weights + slot);
      const uint4* d = reinterpret_cast<const uint4*>(dout) + t * units;
      const uint4* a = reinterpret_cast<const uint4*>(y) + (int64_t)r * units;
      uint4* o = reinterpret_cast<uint4*>(dy) + (int64_t)r * units;
      for (int u = lane; u < units; u += 32) {
        const uint4 dv = __ldg(d + u), yv = __ldg(a + u);
        const uint32_t dx[4] = {dv.x, dv.y, dv.z, dv.w}, yx[4] = {yv.x, yv.y, yv.z, yv.w};
        uint32_t ox[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float d0 = __uint_as_float(dx[i] << 16), d1 = __uint_as_float(dx[i] & 0xFFFF0000u);
          dot = fmaf(d0, __uint_as_float(yx[i] << 16), dot);
          dot = fmaf(d1, __uint_as_float(yx[i] & 0xFFFF0000u), dot);
          ox[i] = w == 0.0f ? 0u : pack_bf16x2(w * d0, w * d1);
        }
        o[u] = make_uint4(ox[0], ox[1], ox[2], ox[3]);
      }
    }
    dot = warp_sum(dot);
    if (lane == 0) dweights[slot] = dot;
  }
}

size_t choose_smem(int E, bool single) {
  return 4 * (single ? kWarps + (size_t)kWarps * E : (size_t)E);
}
size_t place_smem(int E) { return 4 * (kWarps + 2 * kThreads + (size_t)kWarps * E); }

template <auto Fn>
cudaError_t single_t(const RouteProblem& p, int per, bool dependent, cudaStream_t s) {
  cudaError_t e = opt_in_smem<Fn>(choose_smem(kMaxE, true));
  if (e != cudaSuccess) return e;
  return launch_kernel<Fn>(1, kThreads, choose_smem(p.E, true), s, dependent, p, per);
}

template <typename TL, int NPL>
cudaError_t route_t(const RouteProblem& p, int num_sms, bool dependent, cudaStream_t s) {
  const int ctas = route_ctas(p.T, num_sms);
  const int per = (int)((p.T + ctas - 1) / ctas);
  if (ctas == 1) {
    if (std::is_same<TL, float>::value && p.nan_rows)
      return single_t<route_choose<float, NPL, true, true>>(p, per, dependent, s);
    return single_t<route_choose<TL, NPL, true>>(p, per, dependent, s);
  }
  cudaError_t e = opt_in_smem<route_place>(place_smem(kMaxE));
  if (e != cudaSuccess) return e;
  constexpr auto k = route_choose<TL, NPL, false>;
  e = launch_kernel<k>(ctas, kThreads, choose_smem(p.E, false), s, dependent, p, per);
  if (e != cudaSuccess) return e;
  return launch_kernel<route_place>(ctas, kThreads, place_smem(p.E), s, true, p, per);
}

template <typename TL>
cudaError_t route_l(const RouteProblem& p, int num_sms, bool d, cudaStream_t s) {
  const int npl = (p.E + 31) / 32;
  if (npl <= 1) return route_t<TL, 1>(p, num_sms, d, s);
  if (npl <= 2) return route_t<TL, 2>(p, num_sms, d, s);
  if (npl <= 4) return route_t<TL, 4>(p, num_sms, d, s);
  if (npl <= 8) return route_t<TL, 8>(p, num_sms, d, s);
  if (npl <= 16) return route_t<TL, 16>(p, num_sms, d, s);
  return route_t<TL, 32>(p, num_sms, d, s);
}

}  // namespace

int route_ctas(int64_t T, int num_sms) {
  if (T <= kSingleTokens) return 1;
  const int64_t n = (T + kWarps - 1) / kWarps;
  const int64_t most = num_sms < kMaxRouteCtas ? num_sms : kMaxRouteCtas;
  return (int)(n < most ? n : most);
}

cudaError_t launch_route(const RouteProblem& p, int num_sms, bool dependent, cudaStream_t s) {
  return p.fp32 ? route_l<float>(p, num_sms, dependent, s) : route_l<uint16_t>(p, num_sms, dependent, s);
}

cudaError_t launch_route_bwd(const void* logits, int32_t fp32, int64_t T, int32_t E, int32_t k,
                             int32_t renorm, const int32_t* ids, const float* weights,
                             const float* dweights, void* dlogits, int* err, int num_sms,
                             cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  const int64_t need = (T + 7) / 8;
  const int grid = (int)(need < 8 * (int64_t)num_sms ? need : 8 * (int64_t)num_sms);
  const size_t smem = 8 * 4 * (size_t)E;
  if (fp32)
    return launch_kernel<route_bwd_kernel<float>>(
        grid, 256, smem, s, false, static_cast<const float*>(logits), T, E, k, renorm, ids, weights,
        dweights, static_cast<float*>(dlogits), err);
  return launch_kernel<route_bwd_kernel<uint16_t>>(
      grid, 256, smem, s, false, static_cast<const uint16_t*>(logits), T, E, k, renorm, ids, weights,
      dweights, static_cast<uint16_t*>(dlogits), err);
}

namespace {
template <typename TY>
cudaError_t combine_t(const TY* y, int64_t P, int64_t H, const int32_t* row_of_slot,
                      const float* weights, int64_t T, int32_t k, uint16_t* out, int* err,
                      int num_sms, bool dependent, cudaStream_t s) {
  const int64_t n = T * (H / 8);
  if (n == 0) return cudaSuccess;
  const int64_t need = (n + 255) / 256, most = 64 * (int64_t)num_sms;
  return launch_kernel<combine_kernel<TY>>((int)(need < most ? need : most), 256, 0, s, dependent, y, P,
                                           (uint32_t)(H / 8), row_of_slot, weights, n, (int)k, out, err);
}
}  // namespace

cudaError_t launch_combine(const uint16_t* y, int64_t P, int64_t H, const int32_t* row_of_slot,
                           const float* weights, int64_t T, int32_t k, uint16_t* out, int* err,
                           int num_sms, cudaStream_t s) {
  return combine_t(y, P, H, row_of_slot, weights, T, k, out, err, num_sms, false, s);
}

cudaError_t launch_combine_f32(const float* y, int64_t P, int64_t H, const int32_t* row_of_slot,
                               const float* weights, int64_t T, int32_t k, uint16_t* out, int* err,
                               int num_sms, cudaStream_t s) {
  return combine_t(y, P, H, row_of_slot, weights, T, k, out, err, num_sms, true, s);
}

cudaError_t launch_combine_bwd(const uint16_t* dout, const uint16_t* y, int64_t P, int64_t H,
                               const int32_t* row_of_slot, const int32_t* slot_of_row,
                               const float* weights, int64_t T, int32_t k, uint16_t* dy,
                               float* dweights, int* err, int num_sms, cudaStream_t s) {
  const int64_t n = T * k;
  if (n == 0) return cudaSuccess;
  const int64_t need = (n + 7) / 8, most = 64 * (int64_t)num_sms;
  return launch_kernel<combine_bwd_kernel>((int)(need < most ? need : most), 256, 0, s, false, dout,
                                           y, P, (int32_t)(H / 8), row_of_slot, slot_of_row, weights,
                                           n, (int)k, dy, dweights, err);
}

}  // namespace gbw
