// launch.cuh -- host-side launch helpers shared by the mixture-of-experts
// kernels (routing, combine, whole layer, MXFP4 x MXFP4 product).
#pragma once

#include <atomic>

#include "common.cuh"

namespace gbw {

// Opts kernel Fn in to `smem` bytes of dynamic shared memory, once per
// device.  Every call for one Fn passes the same size (its largest), so the
// first one settles it; host threads may race, the attribute is the same.
template <auto Fn>
cudaError_t opt_in_smem(size_t smem) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(reinterpret_cast<const void*>(Fn),
                           cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Launches Fn; with `dependent` it may start while the kernel before it on
// the stream finishes (programmatic dependent launch): Fn then calls
// grid_dependency_wait() before it touches what that kernel writes.
template <auto Fn, typename... Args>
cudaError_t launch_kernel(dim3 grid, int block, size_t smem, cudaStream_t s, bool dependent,
                          Args... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, Fn, args...);
}

// ----------------------------------------------------------------------
// launch arguments of the kernels that use these helpers
// ----------------------------------------------------------------------

struct RouteProblem {
  const void* logits;  // [T, E] bf16 or fp32
  int32_t fp32;        // logits' type
  int64_t T;
  int32_t E, k, renorm;
  int32_t* ids;        // [T, k]
  float* weights;      // [T, k]
  int32_t* offsets;    // [E + 1]
  int32_t* row_to_token;  // [P]
  int32_t* row_of_slot;   // [P]
  int32_t* slot_of_row;   // [P]
  int32_t* hist;       // workspace [CTAs, E]
  bool nan_rows = false;  // NaN weights for a token of NaN logits and no number
                          // (fp32 logits of at most 128 tokens)
};

// CTAs of the routing's first kernel (1: one kernel does it all), and so the
// rows of its histogram workspace: at most kMaxRouteCtas.
constexpr int kMaxRouteCtas = 160;
int route_ctas(int64_t T, int num_sms);
// dependent: started behind the kernel before it, for which it waits
cudaError_t launch_route(const RouteProblem& p, int num_sms, bool dependent, cudaStream_t s);
cudaError_t launch_route_bwd(const void* logits, int32_t fp32, int64_t T, int32_t E, int32_t k,
                             int32_t renorm, const int32_t* ids, const float* weights,
                             const float* dweights, void* dlogits, int* err, int num_sms,
                             cudaStream_t s);
cudaError_t launch_combine(const uint16_t* y, int64_t P, int64_t H, const int32_t* row_of_slot,
                           const float* weights, int64_t T, int32_t k, uint16_t* out, int* err,
                           int num_sms, cudaStream_t s);
// fp32 rows, started behind the kernel before it
cudaError_t launch_combine_f32(const float* y, int64_t P, int64_t H, const int32_t* row_of_slot,
                               const float* weights, int64_t T, int32_t k, uint16_t* out, int* err,
                               int num_sms, cudaStream_t s);
cudaError_t launch_combine_bwd(const uint16_t* dout, const uint16_t* y, int64_t P, int64_t H,
                               const int32_t* row_of_slot, const int32_t* slot_of_row,
                               const float* weights, int64_t T, int32_t k, uint16_t* dy,
                               float* dweights, int* err, int num_sms, cudaStream_t s);

// A whole layer for a few tokens: x [T, H], router [E, H] (+ bias [E]),
// packed gate_up [E, 2I, H/2] and down [E, H, I/2] with their scales.
struct LayerProblem {
  const uint16_t* x;
  int64_t T, H, I;
  int32_t E, k, renorm;
  const uint16_t* rw;
  const float* rb;      // or null
  const uint8_t* gu;
  const void* gu_scale;
  const uint8_t* dn;
  const void* dn_scale;
  uint16_t* out;        // [T, H]
  int* err;
};
int64_t layer_workspace(int64_t T, int32_t E, int32_t k, int64_t H, int64_t I);
cudaError_t launch_layer(Fmt f, const LayerProblem& p, void* workspace, int num_sms,
                         cudaStream_t s);

// bf16 rows (gathered through r2t unless it is null; glu: silu(gate) * up of
// rows [2K]) to MXFP4, and the grouped product of MXFP4 rows and weights.
cudaError_t launch_quantize_rows(const uint16_t* x, int64_t T, int64_t K, const int32_t* r2t,
                                 int64_t P, bool glu, uint8_t* codes, uint8_t* scales, int* err,
                                 cudaStream_t s);
cudaError_t launch_gemm_a4(const uint8_t* xq, const uint8_t* xs, int64_t P, int64_t K,
                           const uint8_t* w, const uint8_t* ws, int32_t E, int64_t N,
                           const int32_t* offsets, uint16_t* out, int* err, int num_sms,
                           cudaStream_t s);

// The same for rows in kPieces 4-bit pieces each (32 bits of a block's maximum):
// bf16 rows gathered through r2t, or silu(gate) * up of fp32 rows [2K], to codes
// [P * kPieces, K / 2] and scale words [ceil(K / 128)][P * kPieces]; their product
// with MXFP4 weights, summed over the pieces in fp32, [P, N].  Both start behind the kernel
// before them and wait for it.
constexpr int kPieces = 16;
cudaError_t launch_quantize_pieces(const void* x, int64_t T, int64_t K, const int32_t* r2t, int64_t P,
                                   bool glu, uint8_t* codes, uint32_t* scales, int* err,
                                   cudaStream_t s);
cudaError_t launch_gemm_pieces(const uint8_t* xq, const uint32_t* xs, int64_t P, int64_t K,
                               const uint8_t* w, const uint8_t* ws, int32_t E, int64_t N,
                               const int32_t* offsets, float* out, int* err, int num_sms,
                               cudaStream_t s);

}  // namespace gbw
