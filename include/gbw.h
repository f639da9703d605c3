/*
 * gbw.h -- C ABI of the B200 grouped 4-bit MoE matmul library (libgbw.so).
 *
 * One call multiplies bf16 activations by the 4-bit packed weights of every
 * active expert ("grouped-nf4-gemm 0.43.0" project page, opening lines: one
 * GPU launch for the active experts, no full-size bf16 weight copies;
 * "Receipts-driven engineering", opening paragraph: the codebook is decoded
 * in registers inside the GEMM mainloop, NF4 in the bitsandbytes packed
 * format unchanged, MXFP4 as OCP e2m1 on released checkpoint bytes, the NF4
 * path differentiable).
 *
 * Conventions for every entry point
 *  - All array arguments are DEVICE pointers owned by the caller; the library
 *    never allocates, frees or keeps them.  Inputs are only read.
 *  - bf16 arrays are passed as uint16_t bit patterns.
 *  - `stream` is a cudaStream_t (NULL = the legacy default stream).  Every
 *    call is asynchronous on that stream and does no host synchronisation.
 *  - Host-side checks (NULL pointers, sizes, alignment, device architecture)
 *    return an error code before anything is launched.
 *  - Checks that need device data (expert_offsets, row_to_token) run inside
 *    the kernels: offsets are clamped to a running maximum in [0, P] and
 *    token indices to [0, T), so no access leaves the caller's buffers; the
 *    violation is recorded in a per-device error word that
 *    gbw_device_status() reads.  The same word records a bounded wait that
 *    gave up (the kernel then returns instead of hanging).
 *  - The library runs only on sm_100 devices (B200); anything else returns
 *    GBW_ERR_ARCH.  There is no fallback path.
 */
#ifndef GBW_H_
#define GBW_H_

#include <stdint.h>

#if defined(__GNUC__)
#define GBW_API __attribute__((visibility("default")))
#else
#define GBW_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GBW_OK = 0,
  GBW_ERR_NULL = 1,   /* a required pointer is NULL */
  GBW_ERR_SHAPE = 2,  /* a size is negative or breaks a divisibility rule */
  GBW_ERR_ALIGN = 3,  /* a pointer or row stride is not 16-byte aligned */
  GBW_ERR_ARCH = 4,   /* the current device is not sm_100 */
  GBW_ERR_LAUNCH = 5, /* a CUDA call failed (cudaGetLastError text kept) */
  GBW_ERR_DEVICE = 6  /* gbw_device_status found a device-side error */
} gbw_status;

typedef enum {
  GBW_MODE_AUTO = 0, /* GEMV when P <= 4 * E (at most ~4 routed rows per
                        expert on average), else the tensor-core GEMM */
  GBW_MODE_GEMM = 1, /* force the tcgen05 grouped GEMM */
  GBW_MODE_GEMV = 2  /* force the bandwidth GEMV (no tensor cores) */
} gbw_mode;

/* Flag OR-ed into the mode argument of the grouped forward calls.
 * GBW_FLAG_OVERLAP_PREV: the caller guarantees that the packed weights, the
 * scales, expert_offsets and row_to_token of this call are not written by
 * the kernel launched immediately before it on the same stream (in a MoE
 * layer they come from the checkpoint and the router, launched earlier).
 * The bandwidth GEMV then reads them while that kernel is still finishing
 * (programmatic dependent launch); it reads x and writes out only after the
 * preceding kernel has completed, with or without the flag.  Passing the
 * flag when the guarantee does not hold gives undefined results. */
#define GBW_FLAG_OVERLAP_PREV 0x100

/* Bits of the device error word. */
#define GBW_DEVERR_OFFSETS 1 /* expert_offsets not 0 <= ... <= P (clamped) */
#define GBW_DEVERR_TOKEN 2   /* row_to_token[p] outside [0, T) (clamped) */
#define GBW_DEVERR_TIMEOUT 4 /* a pipeline wait gave up (or the whole layer's shared
                                memory does not start where it counts on);
                                output incomplete */
#define GBW_DEVERR_ROUTE 8   /* an expert id or a routed row out of range, or
                                slot_of_row not the inverse of row_of_slot
                                (the slot is left out) */

/* Types of the router logits. */
#define GBW_LOGITS_BF16 0
#define GBW_LOGITS_FP32 1

/* Grouped NF4 forward ("grouped-nf4-gemm 0.43.0", "Which entry point?":
 * nf4_grouped.gemm_4bit_grouped; the bandwidth route of the 0.43.0 notes is
 * GBW_MODE_GEMV).
 *   out[p, n] = bf16( sum_k x[tok(p), k] * W_e(p)[n, k] ),  fp32 accumulation
 *   W_e[n, k] = NF4[q] * absmax[e, n, k/64]  (q = code of element k)
 *   x              [T, K]   bf16, row-major
 *   packed         [E, N, K/2] uint8: byte j of a row holds elements 2j (high
 *                  nibble) and 2j+1 (low nibble) -- the bitsandbytes layout
 *   absmax         [E, N, K/64] fp32, one per 64 consecutive K elements
 *   expert_offsets [E+1] int32 (device): routed rows are sorted by expert;
 *                  rows expert_offsets[e] .. expert_offsets[e+1]-1 use expert
 *                  e; expert_offsets[0] = 0, expert_offsets[E] = P
 *   row_to_token   [P] int32 (device) or NULL: routed row p reads x row
 *                  row_to_token[p]; NULL means row p reads x row p (T >= P)
 *   out            [P, N] bf16, row-major, expert-sorted row order
 * mode           a gbw_mode, optionally OR-ed with GBW_FLAG_OVERLAP_PREV
 * Requires K % 64 == 0, N % 8 == 0, 1 <= E <= 1024, and 16-byte aligned x,
 * packed and out.  P == 0 is a no-op.  Experts with no rows cost nothing. */
GBW_API gbw_status gnf4_grouped_gemm(const uint16_t* x, int64_t T, int64_t K,
                             const uint8_t* packed, const float* absmax,
                             int32_t E, int64_t N,
                             const int32_t* expert_offsets,
                             const int32_t* row_to_token, int64_t P,
                             uint16_t* out, int32_t mode, void* stream);

/* Grouped MXFP4 forward ("grouped-nf4-gemm 0.43.0", "Which entry point?":
 * mxfp4_grouped.gemm_mxfp4_grouped; "native MXFP4 MoE inference": e2m1
 * blocks with e8m0 scales, no requantisation, no bf16 materialisation).
 *   W_e[n, k] = e2m1(code) * 2^(scales[e, n, k/32] - 127)
 *   blocks [E, N, K/32, 16] uint8 (= [E, N, K/2]): byte j holds elements 2j
 *          (LOW nibble) and 2j+1 (high nibble); bit 3 of a code is its sign
 *   scales [E, N, K/32] uint8, e8m0 (0xFF is NaN), 2-byte aligned
 * Everything else as gnf4_grouped_gemm; requires K % 32 == 0, N % 8 == 0.
 * K % 64 == 32 is taken by both paths: the tensor-core GEMM runs its last
 * 64-wide K stage half full, zeros in the upper half on both operands. */
GBW_API gbw_status gmxfp4_grouped_gemm(const uint16_t* x, int64_t T, int64_t K,
                               const uint8_t* blocks, const uint8_t* scales,
                               int32_t E, int64_t N,
                               const int32_t* expert_offsets,
                               const int32_t* row_to_token, int64_t P,
                               uint16_t* out, int32_t mode, void* stream);

/* Grouped NF4 activation gradient ("grouped-nf4-gemm 0.43.0", "Which entry
 * point?": dgrad_4bit_grouped; "Receipts-driven engineering": fine-tuning
 * never leaves the packed format).
 *   dx[p, k] = bf16( sum_n dy[p, n] * W_e(p)[n, k] ),  fp32 accumulation
 *   dy [P, N] bf16 row-major (expert-sorted rows), dx [P, K] bf16 row-major;
 *   packed / absmax / expert_offsets exactly as in gnf4_grouped_gemm (the
 *   weights are read packed, in the transposed orientation).
 * Requires K % 64 == 0, N % 64 == 0, 16-byte aligned dy, packed and dx. */
GBW_API gbw_status gnf4_grouped_dgrad(const uint16_t* dy, int64_t P, int64_t N,
                              const uint8_t* packed, const float* absmax,
                              int32_t E, int64_t K,
                              const int32_t* expert_offsets, uint16_t* dx,
                              void* stream);

/* Grouped MXFP4 activation gradient ("grouped-nf4-gemm 0.43.0", "Which
 * entry point?": the MXFP4 entry point; "Receipts-driven engineering":
 * training on the released MXFP4 bytes without requantisation).
 *   dx[p, k] = bf16( sum_n dy[p, n] * W_e(p)[n, k] ),  fp32 accumulation
 *   dy, dx, expert_offsets as in gnf4_grouped_dgrad; blocks / scales as in
 *   gmxfp4_grouped_gemm (read packed, in the transposed orientation).
 * Requires K % 64 == 0, N % 64 == 0, 16-byte aligned dy, blocks and dx,
 * 2-byte aligned scales. */
GBW_API gbw_status gmxfp4_grouped_dgrad(const uint16_t* dy, int64_t P, int64_t N,
                                const uint8_t* blocks, const uint8_t* scales,
                                int32_t E, int64_t K,
                                const int32_t* expert_offsets, uint16_t* dx,
                                void* stream);

/* Fused expert pass, NF4 ("Receipts-driven engineering", "The numbers":
 * the fused training row over all 48 Qwen3-30B-A3B layers -- the expert
 * MLP runs gate_up, the SwiGLU combine and down in one pass per routed row).
 *   gate_up[p, :] = x[tok(p)] @ Wgu_e(p)^T          (2I columns, bf16)
 *   h[p, j]       = bf16( silu(gate_up[p, j]) * gate_up[p, I + j] ),
 *                   silu(v) = v / (1 + e^-v), evaluated in fp32
 *   out[p, :]     = h[p] @ Wdn_e(p)^T                (H columns, bf16)
 * The page names the pass but prints neither the activation nor the
 * gate/up layout; the reading taken is the standard SwiGLU with the gate
 * rows [0, I) stacked above the up rows [I, 2I) of each expert's gate_up
 * weight.
 *   x          [T, H] bf16 row-major; row_to_token / expert_offsets / P as
 *              in gnf4_grouped_gemm
 *   gu_packed  [E, 2I, H/2] uint8, gu_absmax [E, 2I, H/64] fp32
 *   dn_packed  [E, H, I/2] uint8, dn_absmax [E, H, I/64] fp32
 *   h          [P, I] bf16 WORKSPACE supplied by the caller: written by the
 *              gate_up kernel, read by the down kernel (it keeps h)
 *   out        [P, H] bf16, expert-sorted row order
 *   mode       AUTO: both projections on the bandwidth GEMV when P <= 4 * E,
 *              else both on the tensor cores; GEMM / GEMV force a path.  No
 *              flags.  SwiGLU is computed where the gate and up sums meet
 *              (the GEMM epilogue pairs them in one tile, the GEMV in one
 *              warp), so gate_up is never written out.
 * Requires H % 64 == 0, I % 64 == 0, 16-byte aligned x, weights, h and out.
 * Two kernels are launched on `stream`, in order. */
GBW_API gbw_status gnf4_grouped_expert_mlp(const uint16_t* x, int64_t T, int64_t H,
                                   const uint8_t* gu_packed, const float* gu_absmax,
                                   const uint8_t* dn_packed, const float* dn_absmax,
                                   int32_t E, int64_t I, const int32_t* expert_offsets,
                                   const int32_t* row_to_token, int64_t P, uint16_t* h,
                                   uint16_t* out, int32_t mode, void* stream);

/* Fused expert pass, MXFP4 (gate_up blocks [E, 2I, H/32, 16] + scales
 * [E, 2I, H/32]; down blocks [E, H, I/32, 16] + scales [E, H, I/32], e8m0,
 * 2-byte aligned).  Everything else as gnf4_grouped_expert_mlp. */
GBW_API gbw_status gmxfp4_grouped_expert_mlp(const uint16_t* x, int64_t T, int64_t H,
                                     const uint8_t* gu_blocks, const uint8_t* gu_scales,
                                     const uint8_t* dn_blocks, const uint8_t* dn_scales,
                                     int32_t E, int64_t I, const int32_t* expert_offsets,
                                     const int32_t* row_to_token, int64_t P, uint16_t* h,
                                     uint16_t* out, int32_t mode, void* stream);

/* Fused NF4 expert pass that allocates nothing and takes no workspace.
 * This entry point has no counterpart on the source pages; it exists for
 * callers that cannot hand the library device memory at call time -- for
 * example a plugin running inside an inference engine that has already
 * reserved all device memory for itself, or a serving loop that forbids
 * allocation after warm-up (cudaMalloc may synchronise the device and
 * fragment memory held by a caching allocator).
 *   Same arguments and results as gnf4_grouped_expert_mlp, without h: the h
 *   rows go to a fixed scratch array inside the library's device image
 *   (4 MiB, which every device that loads the library keeps until the
 *   process exits).
 *   Limit: P * I <= 2,097,152; larger problems return GBW_ERR_SHAPE.
 *   The first call on a device looks up the scratch address for that device
 *   (cudaGetSymbolAddress); make that first call before any stream capture.
 *   All calls share the one array: calls whose kernels may overlap on the
 *   GPU (different streams, or several host threads) race on it and must be
 *   ordered by the caller.  No call depends on what an earlier call left
 *   there.  No device memory is allocated or freed. */
GBW_API gbw_status gnf4_grouped_expert_mlp_noalloc(const uint16_t* x, int64_t T, int64_t H,
                                           const uint8_t* gu_packed, const float* gu_absmax,
                                           const uint8_t* dn_packed, const float* dn_absmax,
                                           int32_t E, int64_t I, const int32_t* expert_offsets,
                                           const int32_t* row_to_token, int64_t P,
                                           uint16_t* out, int32_t mode, void* stream);

/* Routing: each token's k experts, their softmax weights, and the
 * expert-sorted plan that the grouped calls read.
 *   logits  [T, E] bf16 (logits_type GBW_LOGITS_BF16) or fp32
 *           (GBW_LOGITS_FP32), contiguous
 *   topk_ids      [T, k] int32: the k largest logits in falling order, ties
 *                 to the lowest index; a NaN counts as -inf
 *   topk_weights  [T, k] fp32: exp(l - max) over its sum, over the chosen
 *                 experts (renormalize != 0) or over all E; a row without any
 *                 logit above -inf gets ids 0 .. k-1 and weights 0; equal
 *                 infinite maxima share
 *   expert_offsets [E+1], row_to_token [P], P = T * k: as in
 *                 gnf4_grouped_gemm; routed rows are sorted by expert, stably
 *                 (rows of one expert in the order of their tokens)
 *   row_of_slot   [T, k] int32: routed row of slot s of token t
 *   slot_of_row   [P] int32: its inverse, t * k + s of each routed row
 *   workspace     gmoe_route_workspace(T, E) bytes of device memory (may be
 *                 NULL when that is 0), overwritten; calls that may overlap
 *                 need one each
 * Requires 1 <= E <= 1024, 1 <= k <= min(E, 32), T * k < 2^31.  T == 0 writes
 * expert_offsets (zeros) only.  One launch up to 128 tokens, two above. */
GBW_API gbw_status gmoe_route(const void* logits, int32_t logits_type, int64_t T, int32_t E,
                              int32_t k, int32_t renormalize, int32_t* topk_ids,
                              float* topk_weights, int32_t* expert_offsets,
                              int32_t* row_to_token, int32_t* row_of_slot, int32_t* slot_of_row,
                              void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace gmoe_route needs for T tokens and E experts. */
GBW_API int64_t gmoe_route_workspace(int64_t T, int32_t E);

/* Gradient of gmoe_route's weights:
 *   dlogits[t, e] = [e = ids[s]] w[s] dw[s] - q[e] * sum_s w[s] dw[s]
 * with q = w on the chosen experts (renormalize) or the softmax over all.
 *   logits, topk_ids, topk_weights   as gmoe_route took and gave them (logits
 *            is not read and may be NULL when renormalize != 0)
 *   dweights [T, k] fp32; dlogits [T, E], every element written, in the
 *            logits' type.  A slot of weight 0 passes nothing on, nor does one
 *            whose id is outside [0, E) (it raises GBW_DEVERR_ROUTE). */
GBW_API gbw_status gmoe_route_bwd(const void* logits, int32_t logits_type, int64_t T, int32_t E,
                                  int32_t k, int32_t renormalize, const int32_t* topk_ids,
                                  const float* topk_weights, const float* dweights, void* dlogits,
                                  void* stream);

/* Combine: out[t, :] = bf16( sum_s w[t, s] * y[row_of_slot[t, s], :] ), summed
 * in slot order in fp32.
 *   y [P, H] bf16 (the routed rows, e.g. the down projection's output),
 *   row_of_slot [T, k] int32, weights [T, k] fp32 or NULL (all 1: with it the
 *   call sums the routed rows' gradients dx back into their tokens), out
 *   [T, H] bf16.  A slot of weight 0 adds nothing, whatever its row holds.  A
 *   row outside [0, P) adds nothing and raises GBW_DEVERR_ROUTE.
 * Requires H % 8 == 0, 1 <= k <= 32, 16-byte aligned y and out. */
GBW_API gbw_status gmoe_combine(const uint16_t* y, int64_t P, int64_t H,
                                const int32_t* row_of_slot, const float* weights, int64_t T,
                                int32_t k, uint16_t* out, void* stream);

/* Gradient of gmoe_combine: for each slot, with r = row_of_slot[t, s],
 *   dy[r, :] = bf16( w[t, s] * dout[t, :] ),  dw[t, s] = sum_h y[r, h] dout[t, h]
 * (fp32).  slot_of_row is gmoe_route's inverse of row_of_slot: a row is
 * written by the slot it names, so each row once; a slot that is not named by
 * its row, or whose row is outside [0, P), gets dw = 0 and raises
 * GBW_DEVERR_ROUTE.  Rows of dy that no slot names are left as they were.
 * Requires H % 8 == 0, 16-byte aligned dout, y and dy. */
GBW_API gbw_status gmoe_combine_bwd(const uint16_t* dout, const uint16_t* y, int64_t P, int64_t H,
                                    const int32_t* row_of_slot, const int32_t* slot_of_row,
                                    const float* weights, int64_t T, int32_t k, uint16_t* dy,
                                    float* dweights, void* stream);

/* A whole mixture-of-experts layer for a few tokens, NF4 experts: router,
 * choice of experts, gate_up, SwiGLU, down and weighted combine, in two
 * launches.
 *   l[t, e] = sum_k x[t, k] router_w[e, k] + router_bias[e], fp32 accumulation;
 *   topk ids and weights as gmoe_route chooses them from l; for each slot with
 *   e = ids[t, s]:
 *     h = silu(x[t] @ Wg_e^T) * (x[t] @ Wu_e^T)   kept to 16 bits
 *   out[t, :] = bf16( sum_s w[t, s] * (h_s @ Wd_e^T) )
 *   x            [T, H] bf16; out [T, H] bf16
 *   router_w     [E, H] bf16; router_bias [E] fp32 or NULL
 *   gu_packed    [E, 2I, H/2], gu_absmax [E, 2I, H/64]: gate rows, then up rows
 *   dn_packed    [E, H, I/2], dn_absmax [E, H, I/64]
 *   workspace    gmoe_layer_workspace(T, E, k, H, I) bytes of 256-byte aligned
 *                device memory, overwritten; nothing is kept in it between
 *                calls; calls that may overlap need one each
 * The codebook enters the sums in bf16, off by 7.5e-4 of its root mean square,
 * with hardly a mean (9e-6).  A
 * slot of weight 0 adds nothing, whatever its expert gives.  A value of a token
 * that is not finite may make the whole of its output NaN, no other token's.  A
 * token without any logit above -inf gets an output of zeros when all its logits
 * are -inf, and of NaN when one of them is NaN (as a token that holds a NaN has).
 * Requires T <= 32 (larger batches: gmoe_route, gnf4_grouped_expert_mlp,
 * gmoe_combine), 1 <= E <= 1024, 1 <= k <= min(E, 16), H % 64 == 0,
 * I % 64 == 0, H * I <= 2^33, 16-byte aligned x, router_w, packed weights,
 * scales and out.  T == 0 is
 * a no-op. */
GBW_API gbw_status gnf4_moe_layer(const uint16_t* x, int64_t T, int64_t H,
                                  const uint16_t* router_w, const float* router_bias,
                                  const uint8_t* gu_packed, const float* gu_absmax,
                                  const uint8_t* dn_packed, const float* dn_absmax, int32_t E,
                                  int64_t I, int32_t k, int32_t renormalize, uint16_t* out,
                                  void* workspace, int64_t workspace_bytes, void* stream);

/* The same with MXFP4 experts (blocks [E, 2I, H/32, 16] + scales [E, 2I, H/32],
 * blocks [E, H, I/32, 16] + scales [E, H, I/32], e8m0).  From 100 MB of codes
 * of the experts that T tokens are expected to choose, seven launches: x and h
 * are kept to 2^-32 of the largest of each 32 columns (so a bf16 x whole, down to
 * 2^-24 of it). */
GBW_API gbw_status gmxfp4_moe_layer(const uint16_t* x, int64_t T, int64_t H,
                                    const uint16_t* router_w, const float* router_bias,
                                    const uint8_t* gu_blocks, const uint8_t* gu_scales,
                                    const uint8_t* dn_blocks, const uint8_t* dn_scales, int32_t E,
                                    int64_t I, int32_t k, int32_t renormalize, uint16_t* out,
                                    void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace the two calls above need. */
GBW_API int64_t gmoe_layer_workspace(int64_t T, int32_t E, int32_t k, int64_t H, int64_t I);

/* Activations to MXFP4: routed row p of the output is x row row_to_token[p]
 * (row p when row_to_token is NULL; T >= P then), packed like the weights.
 *   swiglu == 0: x [T, K] bf16, v = the row
 *   swiglu != 0: x [T, 2K] bf16 (a gate_up output, gate columns first),
 *                v[k] = silu(x[k]) * x[K + k] in fp32, not rounded in between
 *   codes  [P, K/32, 16] (= [P, K/2]) uint8, low nibble = even k
 *   scales [ceil(K/128), P, 4] uint8 e8m0: byte b of word (a, p) is the scale of
 *          row p's block 4 a + b, 127 past the last; the rows of a word are
 *          next to each other, as the product loads them
 * Per 32 values: X = floor(log2 max|v|) - 2 clamped to [-127, 127], scale byte
 * X + 127, codes = nearest e2m1 to v / 2^X (ties to the even code,
 * saturating, sign kept); an all-zero block gets scale 0 and codes 0, a block
 * with a value that is not finite scale 255 (NaN) and codes 0.  Token indices
 * are clamped to [0, T) and recorded as in gmxfp4_grouped_gemm.
 * Requires K % 32 == 0, K <= 2^24, 16-byte aligned x, 4-byte aligned codes and
 * scales. */
GBW_API gbw_status gmxfp4_quantize_rows(const uint16_t* x, int64_t T, int64_t K,
                                        const int32_t* row_to_token, int64_t P, int32_t swiglu,
                                        uint8_t* codes, uint8_t* scales, void* stream);

/* Grouped MXFP4 x MXFP4 product (W4A4) on the block-scaled tensor cores:
 *   out[p, n] = bf16( sum_k xq[p, k] * W_e(p)[n, k] ),  fp32 accumulation
 *   x_codes [P, K/2] uint8, x_scales [ceil(K/128), P, 4] uint8: expert-sorted
 *           rows as gmxfp4_quantize_rows writes them
 *   blocks, scales, expert_offsets, out: as in gmxfp4_grouped_gemm (scales
 *           need no alignment here), but expert_offsets[E] may be less than P
 * Requires K % 32 == 0, N % 8 == 0, 1 <= E <= 1024, 16-byte aligned x_codes,
 * blocks and out, 4-byte aligned x_scales.  P == 0 is a no-op.  Rows past
 * expert_offsets[E] (of a buffer padded to a fixed P) belong to no expert: their
 * codes and scales are not used and their rows of out are not written. */
GBW_API gbw_status gmxfp4_grouped_gemm_a4(const uint8_t* x_codes, const uint8_t* x_scales,
                                          int64_t P, int64_t K, const uint8_t* blocks,
                                          const uint8_t* scales, int32_t E, int64_t N,
                                          const int32_t* expert_offsets, uint16_t* out,
                                          void* stream);

/* Decode packed weights to bf16 ("grouped-nf4-gemm 0.43.0", "Try the
 * packers and byte checks on CPU", example 1: dequant_ref).  Bit-exact:
 * w[r, k] = bf16_rn(fp32(NF4[q] * absmax[r, k/64])).  rows counts all
 * expert rows (E*N).  Requires K % 64 == 0 and a 16-byte aligned w_out. */
GBW_API gbw_status gnf4_dequant(const uint8_t* packed, const float* absmax,
                        int64_t rows, int64_t K, uint16_t* w_out,
                        void* stream);

/* MXFP4 decode (same page, example 2: dequant_mxfp4):
 * w[r, k] = bf16_rn(e2m1(code) * 2^(s - 127)).  Requires K % 32 == 0. */
GBW_API gbw_status gmxfp4_dequant(const uint8_t* blocks, const uint8_t* scales,
                          int64_t rows, int64_t K, uint16_t* w_out,
                          void* stream);

/* NF4 packer on the GPU (same page, example 1: quantize_pack_nf4).
 * Per row and 64-block: a = max|w|, q = argmin_i |w/a - NF4[i]| (fp32,
 * lowest index on ties), all-zero block -> a = 0 and code 7.  Byte-identical
 * to the CPU packer.  w [rows, K] fp32; non-finite input is not checked
 * (its codes are unspecified).  Requires K % 64 == 0. */
GBW_API gbw_status gnf4_quantize(const float* w, int64_t rows, int64_t K,
                         uint8_t* packed, float* absmax, void* stream);

/* MXFP4 packer on the GPU (same page, example 2: quantize_pack_mxfp4).
 * Per 32-block: X = floor(log2 max|w|) - 2 clamped to [-127, 127], scale
 * byte X + 127, codes = nearest e2m1 to w / 2^X (ties to even, saturating,
 * sign kept); all-zero block -> scale 0, codes 0.  Requires K % 32 == 0. */
GBW_API gbw_status gmxfp4_quantize(const float* w, int64_t rows, int64_t K,
                           uint8_t* blocks, uint8_t* scales, void* stream);

/* Reads the current device's error word (GBW_DEVERR_* bits) on `stream`,
 * stores it in *host_err, and clears it when `clear` is non-zero.  The word
 * is taken in one atomic step on the device, so a bit that a kernel on
 * another stream raises meanwhile is either returned or kept, never lost.
 * Synchronises `stream`.  Returns GBW_ERR_DEVICE when a bit is set.  Calls
 * for the same device from several host threads at once share one copy
 * slot: serialise them. */
GBW_API gbw_status gbw_device_status(void* stream, int32_t* host_err, int32_t clear);

/* Static text for a status code; the last CUDA error text for
 * GBW_ERR_LAUNCH. */
GBW_API const char* gbw_status_string(gbw_status s);

/* Library version, major * 10000 + minor * 100 + patch. */
GBW_API int32_t gbw_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GBW_H_ */
