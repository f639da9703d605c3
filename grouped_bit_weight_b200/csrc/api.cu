// api.cu -- the extern "C" entry points declared in include/gbw.h: host-side
// argument checks, the sm_100 check, the per-device error word and the
// choice between the tensor-core GEMM and the bandwidth GEMV.
#include <stdio.h>
#include <string.h>

#include <mutex>

#include "common.cuh"
#include "launch.cuh"

namespace gbw {
namespace {

// GBW_DEVERR_* bits raised by the kernels of this library on this device,
// and the copy of it that gbw_device_status takes atomically.
__device__ int g_err_word;
__device__ int g_err_copy;

constexpr int kMaxDevices = 64;
// Experts per call: the kernels keep expert_offsets in shared memory.
constexpr int32_t kMaxExperts = 1024;

// Per-device state, set up once per device (std::call_once, so host threads
// that make their first calls at the same time see it complete).
struct DeviceState {
  int* err = nullptr;   // device address of g_err_word
  int* copy = nullptr;  // device address of g_err_copy
  int sms = 0;
  int arch_ok = 0;      // 1 sm_100, -1 other
  cudaError_t init = cudaSuccess;
};
DeviceState g_dev[kMaxDevices];
std::once_flag g_dev_once[kMaxDevices];

thread_local char g_msg[256] = "";

gbw_status launch_error(cudaError_t e) {
  snprintf(g_msg, sizeof(g_msg), "CUDA error: %s", cudaGetErrorString(e));
  return GBW_ERR_LAUNCH;
}

// Architecture check, SM count and the device addresses of the error word
// and its copy (resolved with the device current).
gbw_status device_state(int** err, int* sms, int** copy = nullptr) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return launch_error(e);
  if (dev < 0 || dev >= kMaxDevices) return GBW_ERR_ARCH;
  DeviceState& d = g_dev[dev];
  std::call_once(g_dev_once[dev], [&]() {
    int major = 0, minor = 0, n = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (major != 10 || minor != 0) {
      d.arch_ok = -1;
      return;
    }
    void* p = nullptr;
    void* c = nullptr;
    d.init = cudaGetSymbolAddress(&p, g_err_word);
    if (d.init == cudaSuccess) d.init = cudaGetSymbolAddress(&c, g_err_copy);
    if (d.init != cudaSuccess) return;
    d.err = static_cast<int*>(p);
    d.copy = static_cast<int*>(c);
    d.sms = n;
    d.arch_ok = 1;
  });
  if (d.init != cudaSuccess) return launch_error(d.init);
  if (d.arch_ok < 0) {
    snprintf(g_msg, sizeof(g_msg), "device %d is not sm_100 (B200)", dev);
    return GBW_ERR_ARCH;
  }
  *err = d.err;
  *sms = d.sms;
  if (copy) *copy = d.copy;
  return GBW_OK;
}

// Takes the error word in one atomic step (and clears it when asked), so a
// bit a kernel on another stream raises at the same time is either in the
// copy or still in the word, never lost.
__global__ void take_error_word(int* err, int* copy, int clear) {
  *copy = clear ? atomicExch(err, 0) : atomicOr(err, 0);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

gbw_status fail(gbw_status s, const char* what) {
  snprintf(g_msg, sizeof(g_msg), "%s", what);
  return s;
}

gbw_status grouped_forward(Fmt f, const uint16_t* x, int64_t T, int64_t K,
                           const uint8_t* w, const void* scale, int32_t E,
                           int64_t N, const int32_t* offsets,
                           const int32_t* row_to_token, int64_t P,
                           uint16_t* out, int32_t mode, void* stream) {
  if (T < 0 || K <= 0 || N <= 0 || E < 1 || P < 0)
    return fail(GBW_ERR_SHAPE, "need T >= 0, K > 0, N > 0, E >= 1, P >= 0");
  if (f == Fmt::NF4 && K % 64) return fail(GBW_ERR_SHAPE, "NF4 needs K % 64 == 0");
  if (f == Fmt::MXFP4 && K % 32) return fail(GBW_ERR_SHAPE, "MXFP4 needs K % 32 == 0");
  if (N % 8) return fail(GBW_ERR_SHAPE, "N must be a multiple of 8");
  if (K > (int64_t)1 << 30 || N > (int64_t)1 << 30 || P > INT32_MAX ||
      T > INT32_MAX || (int64_t)E * N > INT32_MAX)
    return fail(GBW_ERR_SHAPE, "sizes exceed the 32-bit row indices");
  const int32_t flags = mode & ~0xFF;
  mode &= 0xFF;
  if (mode < GBW_MODE_AUTO || mode > GBW_MODE_GEMV || (flags & ~GBW_FLAG_OVERLAP_PREV))
    return fail(GBW_ERR_SHAPE, "unknown mode or flag");
  if (E > kMaxExperts) return fail(GBW_ERR_SHAPE, "at most 1024 experts");
  if (!offsets || !w || !scale) return fail(GBW_ERR_NULL, "NULL weights or offsets");
  if (P > 0 && (!x || !out)) return fail(GBW_ERR_NULL, "NULL x or out");
  if (!row_to_token && T < P)
    return fail(GBW_ERR_SHAPE, "row_to_token == NULL needs T >= P");
  if (row_to_token && P > 0 && T < 1) return fail(GBW_ERR_SHAPE, "T must be >= 1");
  if (!aligned16(x) || !aligned16(w) || !aligned16(out))
    return fail(GBW_ERR_ALIGN, "x, packed weights and out must be 16-byte aligned");
  if (f == Fmt::NF4 && !aligned4(scale)) return fail(GBW_ERR_ALIGN, "absmax must be 4-byte aligned");
  if (f == Fmt::MXFP4 && (reinterpret_cast<uintptr_t>(scale) & 1u))
    return fail(GBW_ERR_ALIGN, "MXFP4 scales must be 2-byte aligned");
  if (!aligned4(offsets) || (row_to_token && !aligned4(row_to_token)))
    return fail(GBW_ERR_ALIGN, "offsets / row_to_token must be 4-byte aligned");
  int* err = nullptr;
  int sms = 0;
  gbw_status st = device_state(&err, &sms);
  if (st != GBW_OK) return st;
  if (P == 0) return GBW_OK;
  GroupedProblem pb{x, T, K, w, scale, E, N, offsets, row_to_token, P, out, err, flags};
  const bool fits = gemv_fits(f, pb, sms);
  if (mode == GBW_MODE_GEMV && !fits)
    return fail(GBW_ERR_SHAPE, "rows too long for the GEMV's shared-memory ring");
  // AUTO: the bandwidth GEMV while experts average at most four routed rows
  // (it streams each active expert's weights once and beats the tensor-core
  // GEMM there: measured on B200 at Qwen3-30B-A3B shapes, the GEMM wins from
  // about six rows per expert); the GEMM takes K % 64 == 32 (MXFP4) with a
  // half last stage
  const bool gemv = mode == GBW_MODE_GEMV ||
                    (mode == GBW_MODE_AUTO && fits && P <= 4 * (int64_t)E);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = gemv ? launch_gemv(f, pb, sms, s) : launch_gemm(f, pb, sms, s);
  return e == cudaSuccess ? GBW_OK : launch_error(e);
}

}  // namespace
}  // namespace gbw

using namespace gbw;

extern "C" {

gbw_status gnf4_grouped_gemm(const uint16_t* x, int64_t T, int64_t K,
                             const uint8_t* packed, const float* absmax,
                             int32_t E, int64_t N,
                             const int32_t* expert_offsets,
                             const int32_t* row_to_token, int64_t P,
                             uint16_t* out, int32_t mode, void* stream) {
  return grouped_forward(Fmt::NF4, x, T, K, packed, absmax, E, N,
                         expert_offsets, row_to_token, P, out, mode, stream);
}

gbw_status gmxfp4_grouped_gemm(const uint16_t* x, int64_t T, int64_t K,
                               const uint8_t* blocks, const uint8_t* scales,
                               int32_t E, int64_t N,
                               const int32_t* expert_offsets,
                               const int32_t* row_to_token, int64_t P,
                               uint16_t* out, int32_t mode, void* stream) {
  return grouped_forward(Fmt::MXFP4, x, T, K, blocks, scales, E, N,
                         expert_offsets, row_to_token, P, out, mode, stream);
}

static gbw_status grouped_dgrad(Fmt f, const uint16_t* dy, int64_t P, int64_t N,
                                const uint8_t* packed, const void* scale, int32_t E,
                                int64_t K, const int32_t* expert_offsets, uint16_t* dx,
                                void* stream) {
  if (P < 0 || N <= 0 || K <= 0 || E < 1)
    return fail(GBW_ERR_SHAPE, "need P >= 0, N > 0, K > 0, E >= 1");
  if (K % 64 || N % 64) return fail(GBW_ERR_SHAPE, "dgrad needs K % 64 == 0 and N % 64 == 0");
  if (E > kMaxExperts) return fail(GBW_ERR_SHAPE, "at most 1024 experts");
  if (K > (int64_t)1 << 30 || P > INT32_MAX || (int64_t)E * N > INT32_MAX)
    return fail(GBW_ERR_SHAPE, "sizes exceed the 32-bit row indices");
  if (!packed || !scale || !expert_offsets) return fail(GBW_ERR_NULL, "NULL weights or offsets");
  if (P > 0 && (!dy || !dx)) return fail(GBW_ERR_NULL, "NULL dy or dx");
  if (!aligned16(dy) || !aligned16(packed) || !aligned16(dx))
    return fail(GBW_ERR_ALIGN, "dy, packed and dx must be 16-byte aligned");
  if ((f == Fmt::NF4 ? !aligned4(scale) : (reinterpret_cast<uintptr_t>(scale) & 1u) != 0) ||
      !aligned4(expert_offsets))
    return fail(GBW_ERR_ALIGN, "absmax 4-byte, scales 2-byte, offsets 4-byte aligned");
  int* err = nullptr;
  int sms = 0;
  gbw_status st = device_state(&err, &sms);
  if (st != GBW_OK) return st;
  if (P == 0) return GBW_OK;
  GroupedProblem pb{dy, P, K, packed, scale, E, N, expert_offsets, nullptr, P, dx, err, 0};
  cudaError_t e = launch_dgrad(f, pb, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GBW_OK : launch_error(e);
}

gbw_status gnf4_grouped_dgrad(const uint16_t* dy, int64_t P, int64_t N,
                              const uint8_t* packed, const float* absmax,
                              int32_t E, int64_t K,
                              const int32_t* expert_offsets, uint16_t* dx,
                              void* stream) {
  return grouped_dgrad(Fmt::NF4, dy, P, N, packed, absmax, E, K, expert_offsets, dx, stream);
}

gbw_status gmxfp4_grouped_dgrad(const uint16_t* dy, int64_t P, int64_t N,
                                const uint8_t* blocks, const uint8_t* scales,
                                int32_t E, int64_t K,
                                const int32_t* expert_offsets, uint16_t* dx,
                                void* stream) {
  return grouped_dgrad(Fmt::MXFP4, dy, P, N, blocks, scales, E, K, expert_offsets, dx, stream);
}

static gbw_status expert_mlp(Fmt f, const uint16_t* x, int64_t T, int64_t H,
                             const uint8_t* gu, const void* gu_scale, const uint8_t* dn,
                             const void* dn_scale, int32_t E, int64_t I,
                             const int32_t* offsets, const int32_t* row_to_token, int64_t P,
                             uint16_t* h, uint16_t* out, int32_t mode, void* stream) {
  if (T < 0 || H <= 0 || I <= 0 || E < 1 || P < 0)
    return fail(GBW_ERR_SHAPE, "need T >= 0, H > 0, I > 0, E >= 1, P >= 0");
  if (H % 64 || I % 64)
    return fail(GBW_ERR_SHAPE, "the fused expert pass needs H % 64 == 0 and I % 64 == 0");
  if (H > (int64_t)1 << 30 || I > (int64_t)1 << 29 || P > INT32_MAX || T > INT32_MAX ||
      (int64_t)E * 2 * I > INT32_MAX || (int64_t)E * H > INT32_MAX)
    return fail(GBW_ERR_SHAPE, "sizes exceed the 32-bit row indices");
  if (mode < GBW_MODE_AUTO || mode > GBW_MODE_GEMV)
    return fail(GBW_ERR_SHAPE, "unknown mode (the fused pass takes no flags)");
  if (E > kMaxExperts) return fail(GBW_ERR_SHAPE, "at most 1024 experts");
  if (!offsets || !gu || !gu_scale || !dn || !dn_scale)
    return fail(GBW_ERR_NULL, "NULL weights or offsets");
  if (P > 0 && (!x || !h || !out)) return fail(GBW_ERR_NULL, "NULL x, h or out");
  if (!row_to_token && T < P) return fail(GBW_ERR_SHAPE, "row_to_token == NULL needs T >= P");
  if (row_to_token && P > 0 && T < 1) return fail(GBW_ERR_SHAPE, "T must be >= 1");
  if (!aligned16(x) || !aligned16(gu) || !aligned16(dn) || !aligned16(h) || !aligned16(out))
    return fail(GBW_ERR_ALIGN, "x, packed weights, h and out must be 16-byte aligned");
  if (f == Fmt::NF4 && (!aligned4(gu_scale) || !aligned4(dn_scale)))
    return fail(GBW_ERR_ALIGN, "absmax must be 4-byte aligned");
  if (f == Fmt::MXFP4 && ((reinterpret_cast<uintptr_t>(gu_scale) | reinterpret_cast<uintptr_t>(dn_scale)) & 1u))
    return fail(GBW_ERR_ALIGN, "MXFP4 scales must be 2-byte aligned");
  if (!aligned4(offsets) || (row_to_token && !aligned4(row_to_token)))
    return fail(GBW_ERR_ALIGN, "offsets / row_to_token must be 4-byte aligned");
  int* err = nullptr;
  int sms = 0;
  gbw_status st = device_state(&err, &sms);
  if (st != GBW_OK) return st;
  if (P == 0) return GBW_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // gate_up with SwiGLU fused into the output (h = silu(gate) * up), then
  // down over h (row p of h is routed row p); both on the bandwidth GEMV or
  // both on the tensor cores
  const bool gemv = mode == GBW_MODE_GEMV || (mode == GBW_MODE_AUTO && P <= 4 * (int64_t)E);
  GroupedProblem g{x, T, H, gu, gu_scale, E, 2 * I, offsets, row_to_token, P, h, err, 0};
  cudaError_t e = gemv ? launch_gemv(f, g, sms, s, true) : launch_gemm(f, g, sms, s, I);
  if (e != cudaSuccess) return launch_error(e);
  GroupedProblem d{h, P, I, dn, dn_scale, E, H, offsets, nullptr, P, out, err, 0};
  e = gemv ? launch_gemv(f, d, sms, s) : launch_gemm(f, d, sms, s);
  return e == cudaSuccess ? GBW_OK : launch_error(e);
}

gbw_status gnf4_grouped_expert_mlp(const uint16_t* x, int64_t T, int64_t H,
                                   const uint8_t* gu_packed, const float* gu_absmax,
                                   const uint8_t* dn_packed, const float* dn_absmax,
                                   int32_t E, int64_t I, const int32_t* expert_offsets,
                                   const int32_t* row_to_token, int64_t P, uint16_t* h,
                                   uint16_t* out, int32_t mode, void* stream) {
  return expert_mlp(Fmt::NF4, x, T, H, gu_packed, gu_absmax, dn_packed, dn_absmax, E, I,
                    expert_offsets, row_to_token, P, h, out, mode, stream);
}

gbw_status gmxfp4_grouped_expert_mlp(const uint16_t* x, int64_t T, int64_t H,
                                     const uint8_t* gu_blocks, const uint8_t* gu_scales,
                                     const uint8_t* dn_blocks, const uint8_t* dn_scales,
                                     int32_t E, int64_t I, const int32_t* expert_offsets,
                                     const int32_t* row_to_token, int64_t P, uint16_t* h,
                                     uint16_t* out, int32_t mode, void* stream) {
  return expert_mlp(Fmt::MXFP4, x, T, H, gu_blocks, gu_scales, dn_blocks, dn_scales, E, I,
                    expert_offsets, row_to_token, P, h, out, mode, stream);
}

// ---------------------------------------------------------------------------
// Fused expert pass without any device allocation.
//
// gnf4_grouped_expert_mlp asks the caller for the h workspace.  Some callers
// cannot provide one: a plugin inside an inference engine whose device memory
// is already handed out by the engine, or a serving loop that forbids device
// allocation after warm-up because cudaMalloc can synchronise the device and
// fragments memory a caching allocator holds.  For them the h rows live in a
// fixed array in this library's device image.  Every device that loads the
// library holds the array until the process exits, so it is kept small.
// ---------------------------------------------------------------------------

// h scratch of gnf4_grouped_expert_mlp_noalloc: P * I bf16 values at most.
constexpr int64_t kNoAllocHElems = (int64_t)1 << 21;  // 2,097,152 values, 4 MiB
static __device__ __align__(256) uint16_t g_noalloc_h[kNoAllocHElems];

// Device address of g_noalloc_h per device.  In host code the name
// g_noalloc_h is only a host-side stand-in, so the address is looked up once
// per device, with that device current, on the first call there.
static uint16_t* g_noalloc_ptr[kMaxDevices];
static cudaError_t g_noalloc_err[kMaxDevices];
static std::once_flag g_noalloc_once[kMaxDevices];

gbw_status gnf4_grouped_expert_mlp_noalloc(const uint16_t* x, int64_t T, int64_t H,
                                           const uint8_t* gu_packed, const float* gu_absmax,
                                           const uint8_t* dn_packed, const float* dn_absmax,
                                           int32_t E, int64_t I, const int32_t* expert_offsets,
                                           const int32_t* row_to_token, int64_t P,
                                           uint16_t* out, int32_t mode, void* stream) {
  if (P > 0 && I > 0 && P <= INT32_MAX && I <= ((int64_t)1 << 29) && P * I > kNoAllocHElems) {
    snprintf(g_msg, sizeof(g_msg),
             "P * I = %lld exceeds the %lld bf16 values of the no-allocation h scratch",
             (long long)(P * I), (long long)kNoAllocHElems);
    return GBW_ERR_SHAPE;
  }
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return launch_error(e);
  if (dev < 0 || dev >= kMaxDevices) return GBW_ERR_ARCH;
  std::call_once(g_noalloc_once[dev], [dev]() {
    void* p = nullptr;
    g_noalloc_err[dev] = cudaGetSymbolAddress(&p, g_noalloc_h);
    g_noalloc_ptr[dev] = static_cast<uint16_t*>(p);
  });
  if (g_noalloc_err[dev] != cudaSuccess) return launch_error(g_noalloc_err[dev]);
  // every h element the down projection reads is written by gate_up in the
  // same call, so the array's previous contents never matter
  return expert_mlp(Fmt::NF4, x, T, H, gu_packed, gu_absmax, dn_packed, dn_absmax, E, I,
                    expert_offsets, row_to_token, P, g_noalloc_ptr[dev], out, mode, stream);
}

// ---------------------------------------------------------------------------
// Routing and combine
// ---------------------------------------------------------------------------

static gbw_status route_shape(int32_t type, int64_t T, int32_t E, int32_t k) {
  if (type != GBW_LOGITS_BF16 && type != GBW_LOGITS_FP32)
    return fail(GBW_ERR_SHAPE, "unknown type of logits");
  if (T < 0 || E < 1 || k < 1) return fail(GBW_ERR_SHAPE, "need T >= 0, E >= 1, k >= 1");
  if (E > kMaxExperts) return fail(GBW_ERR_SHAPE, "at most 1024 experts");
  if (k > E || k > 32) return fail(GBW_ERR_SHAPE, "need k <= min(E, 32)");
  if (T > INT32_MAX || T * k > INT32_MAX) return fail(GBW_ERR_SHAPE, "T * k must be below 2^31");
  return GBW_OK;
}

int64_t gmoe_route_workspace(int64_t T, int32_t E) {
  if (T < 0 || E < 1) return 0;
  const int ctas = route_ctas(T, kMaxRouteCtas);
  return ctas > 1 ? (int64_t)ctas * E * 4 : 0;
}

gbw_status gmoe_route(const void* logits, int32_t logits_type, int64_t T, int32_t E, int32_t k,
                      int32_t renormalize, int32_t* topk_ids, float* topk_weights,
                      int32_t* expert_offsets, int32_t* row_to_token, int32_t* row_of_slot,
                      int32_t* slot_of_row, void* workspace, int64_t workspace_bytes,
                      void* stream) {
  gbw_status st = route_shape(logits_type, T, E, k);
  if (st != GBW_OK) return st;
  if (!expert_offsets) return fail(GBW_ERR_NULL, "NULL expert_offsets");
  if (T > 0 && (!logits || !topk_ids || !topk_weights || !row_to_token || !row_of_slot ||
                !slot_of_row))
    return fail(GBW_ERR_NULL, "NULL logits or output");
  const int64_t need = gmoe_route_workspace(T, E);
  if (need > 0 && !workspace) return fail(GBW_ERR_NULL, "NULL workspace");
  if (workspace_bytes < need) return fail(GBW_ERR_SHAPE, "workspace smaller than gmoe_route_workspace");
  if ((reinterpret_cast<uintptr_t>(logits) & (logits_type == GBW_LOGITS_FP32 ? 3u : 1u)) ||
      !aligned4(topk_ids) || !aligned4(topk_weights) || !aligned4(expert_offsets) ||
      !aligned4(row_to_token) || !aligned4(row_of_slot) || !aligned4(slot_of_row) ||
      !aligned4(workspace))
    return fail(GBW_ERR_ALIGN, "logits must be aligned to their type, the rest to 4 bytes");
  int* err = nullptr;
  int sms = 0;
  st = device_state(&err, &sms);
  if (st != GBW_OK) return st;
  const RouteProblem p{logits, logits_type == GBW_LOGITS_FP32, T, E, k, renormalize != 0, topk_ids,
                       topk_weights, expert_offsets, row_to_token, row_of_slot, slot_of_row,
                       static_cast<int32_t*>(workspace)};
  const cudaError_t e = launch_route(p, sms, false, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GBW_OK : launch_error(e);
}

gbw_status gmoe_route_bwd(const void* logits, int32_t logits_type, int64_t T, int32_t E, int32_t k,
                          int32_t renormalize, const int32_t* topk_ids, const float* topk_weights,
                          const float* dweights, void* dlogits, void* stream) {
  gbw_status st = route_shape(logits_type, T, E, k);
  if (st != GBW_OK) return st;
  if (T > 0 && (!topk_ids || !topk_weights || !dweights || !dlogits || (!renormalize && !logits)))
    return fail(GBW_ERR_NULL, "NULL argument");
  const uintptr_t mask = logits_type == GBW_LOGITS_FP32 ? 3u : 1u;
  if (((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(dlogits)) & mask) ||
      !aligned4(topk_ids) || !aligned4(topk_weights) || !aligned4(dweights))
    return fail(GBW_ERR_ALIGN, "logits must be aligned to their type, the rest to 4 bytes");
  int* err = nullptr;
  int sms = 0;
  st = device_state(&err, &sms);
  if (st != GBW_OK) return st;
  const cudaError_t e = launch_route_bwd(logits, logits_type == GBW_LOGITS_FP32, T, E, k,
                                         renormalize != 0, topk_ids, topk_weights, dweights,
                                         dlogits, err, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GBW_OK : launch_error(e);
}

static gbw_status combine_shape(int64_t P, int64_t H, int64_t T, int32_t k) {
  if (P < 0 || H <= 0 || T < 0 || k < 1 || k > 32)
    return fail(GBW_ERR_SHAPE, "need P >= 0, H > 0, T >= 0, 1 <= k <= 32");
  if (H % 8) return fail(GBW_ERR_SHAPE, "H must be a multiple of 8");
  if (H > (int64_t)1 << 30 || P > INT32_MAX || T > INT32_MAX || T * k > INT32_MAX)
    return fail(GBW_ERR_SHAPE, "sizes exceed the 32-bit row indices");
  return GBW_OK;
}

gbw_status gmoe_combine(const uint16_t* y, int64_t P, int64_t H, const int32_t* row_of_slot,
                        const float* weights, int64_t T, int32_t k, uint16_t* out, void* stream) {
  gbw_status st = combine_shape(P, H, T, k);
  if (st != GBW_OK) return st;
  if (T > 0 && ((P > 0 && !y) || !row_of_slot || !out)) return fail(GBW_ERR_NULL, "NULL argument");
  if (!aligned16(y) || !aligned16(out)) return fail(GBW_ERR_ALIGN, "y and out must be 16-byte aligned");
  if (!aligned4(row_of_slot) || !aligned4(weights))
    return fail(GBW_ERR_ALIGN, "row_of_slot and weights must be 4-byte aligned");
  int* err = nullptr;
  int sms = 0;
  st = device_state(&err, &sms);
  if (st != GBW_OK) return st;
  const cudaError_t e = launch_combine(y, P, H, row_of_slot, weights, T, k, out, err, sms,
                                       static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GBW_OK : launch_error(e);
}

gbw_status gmoe_combine_bwd(const uint16_t* dout, const uint16_t* y, int64_t P, int64_t H,
                            const int32_t* row_of_slot, const int32_t* slot_of_row,
                            const float* weights, int64_t T, int32_t k, uint16_t* dy,
                            float* dweights, void* stream) {
  gbw_status st = combine_shape(P, H, T, k);
  if (st != GBW_OK) return st;
  if (T > 0 && (!dout || !row_of_slot || !weights || !dweights ||
                (P > 0 && (!y || !dy || !slot_of_row))))
    return fail(GBW_ERR_NULL, "NULL argument");
  if (!aligned16(dout) || !aligned16(y) || !aligned16(dy))
    return fail(GBW_ERR_ALIGN, "dout, y and dy must be 16-byte aligned");
  if (!aligned4(row_of_slot) || !aligned4(slot_of_row) || !aligned4(weights) || !aligned4(dweights))
    return fail(GBW_ERR_ALIGN, "indices and weights must be 4-byte aligned");
  int* err = nullptr;
  int sms = 0;
  st = device_state(&err, &sms);
  if (st != GBW_OK) return st;
  const cudaError_t e = launch_combine_bwd(dout, y, P, H, row_of_slot, slot_of_row, weights, T, k,
                                           dy, dweights, err, sms,
                                           static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GBW_OK : launch_error(e);
}

// ---------------------------------------------------------------------------
// Whole layer for a few tokens
// ---------------------------------------------------------------------------

int64_t gmoe_layer_workspace(int64_t T, int32_t E, int32_t k, int64_t H, int64_t I) {
  if (T <= 0 || T > 32 || E < 1 || E > kMaxExperts || k < 1 || k > 16 || H <= 0 || I <= 0 ||
      H > (int64_t)1 << 30 || I > (int64_t)1 << 29)
    return 0;
  return layer_workspace(T, E, k, H, I);
}

static gbw_status moe_layer(Fmt f, const uint16_t* x, int64_t T, int64_t H, const uint16_t* router_w,
                            const float* router_bias, const uint8_t* gu, const void* gu_scale,
                            const uint8_t* dn, const void* dn_scale, int32_t E, int64_t I, int32_t k,
                            int32_t renormalize, uint16_t* out, void* workspace,
                            int64_t workspace_bytes, void* stream) {
  if (T < 0 || H <= 0 || I <= 0 || E < 1 || k < 1)
    return fail(GBW_ERR_SHAPE, "need T >= 0, H > 0, I > 0, E >= 1, k >= 1");
  if (T > 32)
    return fail(GBW_ERR_SHAPE, "the whole layer takes at most 32 tokens: use gmoe_route, the fused "
                               "expert pass and gmoe_combine");
  if (H % 64 || I % 64) return fail(GBW_ERR_SHAPE, "the layer needs H % 64 == 0 and I % 64 == 0");
  if (E > kMaxExperts) return fail(GBW_ERR_SHAPE, "at most 1024 experts");
  if (k > E || k > 16) return fail(GBW_ERR_SHAPE, "need k <= min(E, 16)");
  if (H > (int64_t)1 << 30 || I > (int64_t)1 << 29 || (int64_t)E * 2 * I > INT32_MAX ||
      (int64_t)E * H > INT32_MAX || H * I > (int64_t)1 << 33)
    return fail(GBW_ERR_SHAPE, "sizes exceed the 32-bit row indices");
  const int64_t need = gmoe_layer_workspace(T, E, k, H, I);
  if (T > 0 && (!x || !router_w || !gu || !gu_scale || !dn || !dn_scale || !out || !workspace))
    return fail(GBW_ERR_NULL, "NULL argument");
  if (workspace_bytes < need) return fail(GBW_ERR_SHAPE, "workspace smaller than gmoe_layer_workspace");
  if (!aligned16(x) || !aligned16(router_w) || !aligned16(gu) || !aligned16(dn) || !aligned16(out))
    return fail(GBW_ERR_ALIGN, "x, router_w, packed weights and out must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return fail(GBW_ERR_ALIGN, "the workspace must be 256-byte aligned");
  if (!aligned16(gu_scale) || !aligned16(dn_scale))
    return fail(GBW_ERR_ALIGN, "the layer's scales must be 16-byte aligned");
  if (!aligned4(router_bias)) return fail(GBW_ERR_ALIGN, "router_bias must be 4-byte aligned");
  int* err = nullptr;
  int sms = 0;
  gbw_status st = device_state(&err, &sms);
  if (st != GBW_OK) return st;
  const LayerProblem p{x, T, H, I, E, k, renormalize != 0, router_w, router_bias, gu, gu_scale, dn,
                       dn_scale, out, err};
  const cudaError_t e = launch_layer(f, p, workspace, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GBW_OK : launch_error(e);
}

gbw_status gnf4_moe_layer(const uint16_t* x, int64_t T, int64_t H, const uint16_t* router_w,
                          const float* router_bias, const uint8_t* gu_packed,
                          const float* gu_absmax, const uint8_t* dn_packed, const float* dn_absmax,
                          int32_t E, int64_t I, int32_t k, int32_t renormalize, uint16_t* out,
                          void* workspace, int64_t workspace_bytes, void* stream) {
  return moe_layer(Fmt::NF4, x, T, H, router_w, router_bias, gu_packed, gu_absmax, dn_packed,
                   dn_absmax, E, I, k, renormalize, out, workspace, workspace_bytes, stream);
}

gbw_status gmxfp4_moe_layer(const uint16_t* x, int64_t T, int64_t H, const uint16_t* router_w,
                            const float* router_bias, const uint8_t* gu_blocks,
                            const uint8_t* gu_scales, const uint8_t* dn_blocks,
                            const uint8_t* dn_scales, int32_t E, int64_t I, int32_t k,
                            int32_t renormalize, uint16_t* out, void* workspace,
                            int64_t workspace_bytes, void* stream) {
  return moe_layer(Fmt::MXFP4, x, T, H, router_w, router_bias, gu_blocks, gu_scales, dn_blocks,
                   dn_scales, E, I, k, renormalize, out, workspace, workspace_bytes, stream);
}

// ---------------------------------------------------------------------------
// MXFP4 activations
// ---------------------------------------------------------------------------

gbw_status gmxfp4_quantize_rows(const uint16_t* x, int64_t T, int64_t K,
                                const int32_t* row_to_token, int64_t P, int32_t swiglu,
                                uint8_t* codes, uint8_t* scales, void* stream) {
  if (T < 0 || K <= 0 || P < 0) return fail(GBW_ERR_SHAPE, "need T >= 0, K > 0, P >= 0");
  if (K % 32) return fail(GBW_ERR_SHAPE, "MXFP4 needs K % 32 == 0");
  if (K > (int64_t)1 << 24) return fail(GBW_ERR_SHAPE, "K must be at most 2^24");
  if (P > INT32_MAX || T > INT32_MAX)
    return fail(GBW_ERR_SHAPE, "sizes exceed the 32-bit row indices");
  if (!row_to_token && T < P) return fail(GBW_ERR_SHAPE, "row_to_token == NULL needs T >= P");
  if (row_to_token && P > 0 && T < 1) return fail(GBW_ERR_SHAPE, "T must be >= 1");
  if (P > 0 && (!x || !codes || !scales)) return fail(GBW_ERR_NULL, "NULL x, codes or scales");
  if (!aligned16(x)) return fail(GBW_ERR_ALIGN, "x must be 16-byte aligned");
  if (!aligned4(codes) || !aligned4(scales) || !aligned4(row_to_token))
    return fail(GBW_ERR_ALIGN, "codes, scales and row_to_token must be 4-byte aligned");
  int* err = nullptr;
  int sms = 0;
  gbw_status st = device_state(&err, &sms);
  if (st != GBW_OK) return st;
  const cudaError_t e = launch_quantize_rows(x, T, K, row_to_token, P, swiglu != 0, codes, scales,
                                             err, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GBW_OK : launch_error(e);
}

gbw_status gmxfp4_grouped_gemm_a4(const uint8_t* x_codes, const uint8_t* x_scales, int64_t P,
                                  int64_t K, const uint8_t* blocks, const uint8_t* scales,
                                  int32_t E, int64_t N, const int32_t* expert_offsets,
                                  uint16_t* out, void* stream) {
  if (P < 0 || K <= 0 || N <= 0 || E < 1)
    return fail(GBW_ERR_SHAPE, "need P >= 0, K > 0, N > 0, E >= 1");
  if (K % 32) return fail(GBW_ERR_SHAPE, "MXFP4 needs K % 32 == 0");
  if (N % 8) return fail(GBW_ERR_SHAPE, "N must be a multiple of 8");
  if (E > kMaxExperts) return fail(GBW_ERR_SHAPE, "at most 1024 experts");
  if (K > (int64_t)1 << 30 || N > (int64_t)1 << 30 || P > INT32_MAX || (int64_t)E * N > INT32_MAX)
    return fail(GBW_ERR_SHAPE, "sizes exceed the 32-bit row indices");
  if (!blocks || !scales || !expert_offsets) return fail(GBW_ERR_NULL, "NULL weights or offsets");
  if (P > 0 && (!x_codes || !x_scales || !out)) return fail(GBW_ERR_NULL, "NULL rows or out");
  if (!aligned16(x_codes) || !aligned16(blocks) || !aligned16(out))
    return fail(GBW_ERR_ALIGN, "x_codes, blocks and out must be 16-byte aligned");
  if (!aligned4(expert_offsets) || !aligned4(x_scales))
    return fail(GBW_ERR_ALIGN, "offsets and x_scales must be 4-byte aligned");
  int* err = nullptr;
  int sms = 0;
  gbw_status st = device_state(&err, &sms);
  if (st != GBW_OK) return st;
  const cudaError_t e = launch_gemm_a4(x_codes, x_scales, P, K, blocks, scales, E, N,
                                       expert_offsets, out, err, sms,
                                       static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GBW_OK : launch_error(e);
}

gbw_status gnf4_dequant(const uint8_t* packed, const float* absmax,
                        int64_t rows, int64_t K, uint16_t* w_out,
                        void* stream) {
  if (rows < 0 || K <= 0 || K % 64) return fail(GBW_ERR_SHAPE, "need rows >= 0, K % 64 == 0");
  if (rows > 0 && (!packed || !absmax || !w_out)) return fail(GBW_ERR_NULL, "NULL argument");
  if (!aligned16(packed) || !aligned16(w_out) || !aligned4(absmax))
    return fail(GBW_ERR_ALIGN, "packed / w_out must be 16-byte aligned");
  int* err = nullptr;
  int sms = 0;
  gbw_status st = device_state(&err, &sms);
  if (st != GBW_OK) return st;
  cudaError_t e = launch_dequant(Fmt::NF4, packed, absmax, rows, K, w_out,
                                 static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GBW_OK : launch_error(e);
}

gbw_status gmxfp4_dequant(const uint8_t* blocks, const uint8_t* scales,
                          int64_t rows, int64_t K, uint16_t* w_out,
                          void* stream) {
  if (rows < 0 || K <= 0 || K % 32) return fail(GBW_ERR_SHAPE, "need rows >= 0, K % 32 == 0");
  if (rows > 0 && (!blocks || !scales || !w_out)) return fail(GBW_ERR_NULL, "NULL argument");
  if (!aligned16(blocks) || !aligned16(w_out))
    return fail(GBW_ERR_ALIGN, "blocks / w_out must be 16-byte aligned");
  int* err = nullptr;
  int sms = 0;
  gbw_status st = device_state(&err, &sms);
  if (st != GBW_OK) return st;
  cudaError_t e = launch_dequant(Fmt::MXFP4, blocks, scales, rows, K, w_out,
                                 static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GBW_OK : launch_error(e);
}

gbw_status gnf4_quantize(const float* w, int64_t rows, int64_t K,
                         uint8_t* packed, float* absmax, void* stream) {
  if (rows < 0 || K <= 0 || K % 64) return fail(GBW_ERR_SHAPE, "need rows >= 0, K % 64 == 0");
  if (rows > 0 && (!w || !packed || !absmax)) return fail(GBW_ERR_NULL, "NULL argument");
  if (!aligned16(w) || !aligned4(absmax)) return fail(GBW_ERR_ALIGN, "w must be 16-byte aligned");
  int* err = nullptr;
  int sms = 0;
  gbw_status st = device_state(&err, &sms);
  if (st != GBW_OK) return st;
  cudaError_t e = launch_quantize(Fmt::NF4, w, rows, K, packed, absmax,
                                  static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GBW_OK : launch_error(e);
}

gbw_status gmxfp4_quantize(const float* w, int64_t rows, int64_t K,
                           uint8_t* blocks, uint8_t* scales, void* stream) {
  if (rows < 0 || K <= 0 || K % 32) return fail(GBW_ERR_SHAPE, "need rows >= 0, K % 32 == 0");
  if (rows > 0 && (!w || !blocks || !scales)) return fail(GBW_ERR_NULL, "NULL argument");
  if (!aligned16(w)) return fail(GBW_ERR_ALIGN, "w must be 16-byte aligned");
  int* err = nullptr;
  int sms = 0;
  gbw_status st = device_state(&err, &sms);
  if (st != GBW_OK) return st;
  cudaError_t e = launch_quantize(Fmt::MXFP4, w, rows, K, blocks, scales,
                                  static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GBW_OK : launch_error(e);
}

gbw_status gbw_device_status(void* stream, int32_t* host_err, int32_t clear) {
  int* err = nullptr;
  int* copy = nullptr;
  int sms = 0;
  gbw_status st = device_state(&err, &sms, &copy);
  if (st != GBW_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  take_error_word<<<1, 1, 0, s>>>(err, copy, clear ? 1 : 0);
  cudaError_t e = cudaGetLastError();
  int v = 0;
  if (e == cudaSuccess) e = cudaMemcpyAsync(&v, copy, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return launch_error(e);
  if (host_err) *host_err = v;
  return v ? GBW_ERR_DEVICE : GBW_OK;
}

const char* gbw_status_string(gbw_status s) {
  switch (s) {
    case GBW_OK: return "ok";
    case GBW_ERR_NULL: return g_msg[0] ? g_msg : "NULL pointer";
    case GBW_ERR_SHAPE: return g_msg[0] ? g_msg : "unsupported size";
    case GBW_ERR_ALIGN: return g_msg[0] ? g_msg : "misaligned pointer";
    case GBW_ERR_ARCH: return g_msg[0] ? g_msg : "device is not sm_100";
    case GBW_ERR_LAUNCH: return g_msg[0] ? g_msg : "CUDA launch failed";
    case GBW_ERR_DEVICE: return "device error word set (see GBW_DEVERR_* bits)";
  }
  return "unknown status";
}

int32_t gbw_version(void) { return 100; }

}  // extern "C"
