/*
 * moe.h - C ABI of the GB300 (sm_103a) local Mixture-of-Experts forward chain.
 *
 * The chain (ruDNN user guide, section 3 "MoE workflow"):
 *
 *     logits [T,E] -> softmax/top-k routing -> compact per-expert dispatch
 *                  -> SwiGLU experts -> routing-weighted combine -> out [T,H]
 *
 * Conventions shared by every entry point
 *   - All pointers named "device" are CUDA device pointers on the current
 *     device; the caller allocates and owns every buffer, including the
 *     workspaces. The library allocates no device memory on any call below.
 *   - Tensors are dense and row-major (C order) with the shapes given.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream). Every call only enqueues work on that stream and returns; no
 *     call waits for the device. Results are ready when the stream is.
 *   - Every argument check runs on the host before anything is launched; a
 *     failed check returns its status and enqueues nothing. MOE_ERR_CUDA
 *     means a launch was rejected by the CUDA runtime (the message is in
 *     moe_last_error()).
 *   - Dtypes: MOE_F32, MOE_F16, MOE_BF16 (non-quantised floats, ruDNN user
 *     guide section 4). Arithmetic: routing in FP32; expert projections
 *     accumulate in FP32 (tensor cores for F16/BF16, FP32 FMA for F32, never
 *     TF32); combine accumulates in FP32.
 *   - Indices are uint32 (ruDNN user guide section 4: "indices use U32").
 *   - Thread safety: calls on different streams may run concurrently when
 *     their buffers do not overlap. A moe_experts handle is read-only after
 *     creation and may be shared.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MOE_F32 = 0, MOE_F16 = 1, MOE_BF16 = 2 } moe_dtype;

/* Status codes: the C counterpart of MoeError (ruDNN user guide section 3:
 * "computation entry points return Result with MoeError for invalid shapes,
 * dtypes, or other arguments"). */
typedef enum {
  MOE_OK = 0,
  MOE_ERR_NULL = 1,          /* a required pointer is NULL                          */
  MOE_ERR_SHAPE = 2,         /* a size is out of range or sizes disagree             */
  MOE_ERR_DTYPE = 3,         /* unknown dtype, or dtypes that must agree do not      */
  MOE_ERR_TOP_K = 4,         /* top_k outside 1 <= top_k <= E (section 4)            */
  MOE_ERR_ALIGNMENT = 5,     /* a pointer or row pitch is not 16-byte aligned        */
  MOE_ERR_WORKSPACE = 6,     /* workspace pointer NULL or smaller than required      */
  MOE_ERR_UNSUPPORTED = 7,   /* a valid request this build does not implement        */
  MOE_ERR_CUDA = 8,          /* the CUDA runtime rejected a launch or query          */
  MOE_ERR_DEVICE_CHECK = 9   /* a device-side wait ran out of time (see moe_device_status) */
} moe_status;

/* Opaque expert-weight handle (SwiGluExperts::new, ruDNN user guide section 3). */
typedef struct moe_experts moe_experts;

/* Human-readable name of a status code; never NULL. */
const char* moe_status_string(int status);

/* Detail of the last failed call on this host thread (empty if none). */
const char* moe_last_error(void);

/* ABI version of this library (major * 10000 + minor * 100 + patch): 1.1.0
 * adds moe_experts_forward_combine, moe_route_dispatch,
 * moe_route_sigmoid_grouped_dispatch and moe_permute_rows to 1.0.0; nothing
 * was removed or changed. The moe_mxfp4_*, moe_experts_mxfp4_*,
 * moe_forward_mxfp4*, moe_grad_*, moe_block_*, moe_combine_join,
 * moe_orthogonalize* and moe_muon_step entry points came later under the same
 * number: a caller that has to know looks the symbols up. */
int moe_version(void);

/*
 * moe_route - softmax/top-k routing (RoutingPlan, ruDNN user guide section 4
 * "Routing contract"; restated in the Japanese guide section 4 and the
 * ruDNN 0.1.5 User Guide section 4).
 *
 *   logits        device, [T, E] in `dtype`.
 *   T, E          1 <= E <= 1024, T >= 0 (T = 0 enqueues nothing).
 *   top_k         1 <= top_k <= E, else MOE_ERR_TOP_K.
 *   renormalize   nonzero: divide the selected weights by their sum.
 *   indices       device, [T, top_k] uint32 out: selected experts, slot 0 the
 *                 largest logit, ties to the lower expert id.
 *   weights       device, [T, top_k] out in `dtype`: FP32 softmax over all E
 *                 experts, gathered, optionally renormalized, then rounded to
 *                 `dtype` (round to nearest even).
 *   weights_fp32  device, [T, top_k] float out before that rounding, or NULL.
 *
 * A row holding a NaN or +inf, or only -inf, gets NaN weights (no uniform
 * fallback) and indices 0..top_k-1. Selection compares the logits
 * themselves (softmax is strictly increasing, so this is "softmax then
 * top-k" without ties added by exp rounding).
 */
moe_status moe_route(const void* logits, moe_dtype dtype, int64_t T, int64_t E, int32_t top_k,
                     int32_t renormalize, uint32_t* indices, void* weights, float* weights_fp32,
                     void* stream);

/*
 * moe_dispatch - compact per-expert token layout with no capacity dropping
 * (RoutingPlan::dispatch; ruDNN user guide section 5 "Expert weights and
 * dispatch": tokens are never dropped, a saved mapping restores token order).
 *
 *   indices       device, [T, top_k] uint32 (from moe_route or the caller).
 *   x             device, [T, H] in `dtype`, or NULL to skip x_dispatched.
 *   counts        device, [E] uint32 out: rows per expert.
 *   offsets       device, [E + 1] uint32 out: exclusive prefix of counts.
 *   row_src       device, [T * top_k] uint32 out: dispatched row r holds slot
 *                 row_src[r] = t * top_k + j.
 *   inv           device, [T * top_k] uint32 out: slot t * top_k + j sits in
 *                 dispatched row inv[t * top_k + j].
 *   x_dispatched  device, [T * top_k, H] out (row r = x[row_src[r] / top_k]),
 *                 or NULL. Needs x.
 *   workspace     device scratch of moe_dispatch_workspace_size(T, E, top_k)
 *                 bytes (256-byte aligned); contents need not be initialised.
 *
 * Order within an expert is ascending t * top_k + j, so the maps are the
 * same on every run (the pages leave that order free). An index >= E is not
 * dispatched: its inv entry is 0xFFFFFFFF, counts exclude it, and
 * moe_combine writes a NaN row for that token. No out-of-range access, no
 * host synchronisation.
 */
size_t moe_dispatch_workspace_size(int64_t T, int64_t E, int32_t top_k);
moe_status moe_dispatch(const uint32_t* indices, int64_t T, int64_t E, int32_t top_k,
                        const void* x, moe_dtype dtype, int64_t H, uint32_t* counts,
                        uint32_t* offsets, uint32_t* row_src, uint32_t* inv, void* x_dispatched,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * moe_dispatch_noalloc - moe_dispatch without a workspace argument, for
 * callers that cannot allocate device memory when they dispatch: a plugin
 * that reaches the library through this C ABI from a host framework owning
 * every device allocation, or a serving loop whose memory budget is fixed at
 * start-up and may not grow afterwards. The pages have no counterpart; the
 * outputs are the same as moe_dispatch's, bit for bit.
 *
 * Arguments and outputs are those of moe_dispatch. The scratch instead lives
 * in a fixed 1 MiB (MOE_DISPATCH_NOALLOC_SCRATCH_BYTES) array inside the
 * library's device image; every GPU that loads the library holds it until the
 * process exits. Requests whose scratch, ceil(T*top_k/2048)*E*4 bytes, exceeds
 * it are rejected with MOE_ERR_SHAPE before anything is launched. No call
 * allocates or frees device memory. Every call looks up the array's device
 * address (cudaGetSymbolAddress) with the calling device current, so the
 * address stays right after a cudaDeviceReset; the first call on a device
 * also loads the library's device code there, so make it before any stream
 * capture. All calls on a device share
 * the array and it keeps the last call's contents (each call writes every
 * entry it reads, so nothing needs clearing): calls that may overlap on the
 * GPU, such as calls on different streams without ordering between them, race
 * on it and must not be issued.
 */
#define MOE_DISPATCH_NOALLOC_SCRATCH_BYTES (1u << 20)
moe_status moe_dispatch_noalloc(const uint32_t* indices, int64_t T, int64_t E, int32_t top_k,
                                const void* x, moe_dtype dtype, int64_t H, uint32_t* counts,
                                uint32_t* offsets, uint32_t* row_src, uint32_t* inv,
                                void* x_dispatched, void* stream);

/*
 * moe_route_dispatch - moe_route followed by moe_dispatch as one cooperative
 * launch (ruDNN user guide sections 4 "Routing contract" and 5 "Expert
 * weights and dispatch"): every output is the same, bit for bit, as those two
 * calls give. moe_forward runs this launch for its routing and dispatch.
 *
 *   logits, logits_dtype, T, E, top_k, renormalize, indices, weights,
 *   weights_fp32      as moe_route.
 *   x, x_dtype, H, counts, offsets, row_src, inv, x_dispatched
 *                     as moe_dispatch (x_dtype is x's dtype; x_dispatched
 *                     NULL writes the maps only).
 *   workspace         device scratch of moe_route_dispatch_workspace_size(T, E)
 *                     bytes (256-byte aligned); contents need not be
 *                     initialised (the call zeroes what it needs on the
 *                     stream).
 *
 * The blocks of the launch meet once at a grid-wide barrier (all of them are
 * resident: the launch is cooperative). Its wait is bounded (about one
 * second); a wait that runs out records 0x1B in the device status word
 * (moe_device_status) and the launch returns with its outputs incomplete.
 */
size_t moe_route_dispatch_workspace_size(int64_t T, int64_t E);
moe_status moe_route_dispatch(const void* logits, moe_dtype logits_dtype, int64_t T, int64_t E, int32_t top_k,
                              int32_t renormalize, uint32_t* indices, void* weights, float* weights_fp32,
                              const void* x, moe_dtype x_dtype, int64_t H, uint32_t* counts, uint32_t* offsets,
                              uint32_t* row_src, uint32_t* inv, void* x_dispatched, void* workspace,
                              size_t workspace_bytes, void* stream);

/*
 * moe_permute_rows - move whole rows by an index: the reorders of the
 * expert-parallel exchange (the received rows into expert-major order, the
 * experts' outputs back into the received order); the exchange itself is the
 * caller's collective. Not on the pages: they run every expert on one device.
 *
 *   src           device, [src_rows, row_bytes] (rows contiguous).
 *   dst           device, [dst_rows, row_bytes]; must not overlap src.
 *   index         device, [rows] int64.
 *   scatter       zero: gather, dst[r] = src[index[r]] for r < rows
 *                 (rows <= dst_rows); a row whose index is outside
 *                 0..src_rows-1 is written as zeros. Nonzero: scatter,
 *                 dst[index[r]] = src[r] for r < rows (rows <= src_rows); a
 *                 row whose index is outside 0..dst_rows-1 is skipped, and
 *                 repeated indexes leave one of their rows (unspecified).
 *   row_bytes     > 0; 16-byte rows and pointers move as 16-byte vectors.
 *
 * Errors: MOE_ERR_NULL, MOE_ERR_SHAPE (negative sizes, row_bytes < 1, rows
 * beyond the written or read side). Enqueued on the stream, no host sync.
 */
moe_status moe_permute_rows(const void* src, int64_t src_rows, void* dst, int64_t dst_rows, const int64_t* index,
                            int64_t rows, int64_t row_bytes, int32_t scatter, void* stream);

/*
 * moe_experts_create - validate and wrap bias-free SwiGLU expert weights
 * (SwiGluExperts::new; ruDNN user guide section 5: gate and up [E, I, H],
 * down [E, H, I], one float dtype, one device).
 *
 *   gate, up      device, [E, I, H] in `dtype`.
 *   down          device, [E, H, I] in `dtype`.
 *   E, H, I       1 <= E <= 1024; H, I >= 1. F16/BF16 need H and I to be
 *                 multiples of 8 (16-byte row pitch), else MOE_ERR_ALIGNMENT.
 *   out           receives the handle.
 *
 * The handle records the pointers (the caller keeps the weights alive and
 * unchanged while it is in use) and the prebuilt TMA descriptors. It is
 * reusable across batches and read-only; free it with moe_experts_destroy.
 * Device is the current device at creation.
 */
moe_status moe_experts_create(const void* gate, const void* up, const void* down, moe_dtype dtype,
                              int64_t E, int64_t H, int64_t I, moe_experts** out);
void moe_experts_destroy(moe_experts* experts);

/*
 * moe_experts_forward_dispatched - SwiGLU experts on dispatched rows
 * (SwiGluExperts::forward_dispatched; "tiny-llm deep dive 5: ops.rs",
 * section on SiLU: FFN(x) = W_down (SiLU(W_gate x) * W_up x)).
 *
 *   x_dispatched  device, [rows, H] in the experts' dtype (from moe_dispatch).
 *   offsets       device, [E + 1] uint32 (from moe_dispatch); expert e owns
 *                 rows offsets[e] .. offsets[e+1]-1; offsets[E] must equal
 *                 rows. The host never reads the counts.
 *   rows          T * top_k.
 *   y_dispatched  device, [rows, H] out in the experts' dtype:
 *                 y = W_down[e] h, h = SiLU(W_gate[e] x) * (W_up[e] x), FP32
 *                 accumulation, h rounded to the dtype before the down
 *                 projection.
 *   workspace     device scratch of
 *                 moe_experts_forward_dispatched_workspace_size(experts, rows)
 *                 bytes (holds h, the GEMMs' tile counter and one counter per
 *                 expert), 256-byte aligned.
 *
 * F16/BF16 run both GEMMs as one launch (after a reset of the counters):
 * tiles of the gate/up GEMM first, then tiles of the down GEMM, each of
 * which waits (bounded, about a second; on timeout the device status word
 * records 0x19) until every gate/up tile of its expert has stored its h
 * rows. The results are bit-identical to moe_experts_gate_up followed by
 * moe_experts_down.
 */
size_t moe_experts_forward_dispatched_workspace_size(const moe_experts* experts, int64_t rows);
moe_status moe_experts_forward_dispatched(const moe_experts* experts, const void* x_dispatched,
                                          const uint32_t* offsets, int64_t rows,
                                          void* y_dispatched, void* workspace,
                                          size_t workspace_bytes, void* stream);

/*
 * moe_experts_forward_combine - the experts and the weighted combine in one
 * launch: SwiGluExperts::forward_dispatched followed by
 * DispatchedTokens::combine (ruDNN user guide section 6), the combine run by
 * the down GEMM's epilogue warps ("PyTorch general ops", section "two ways
 * to write a contraction": the routing-weighted sum over a token's top_k
 * expert outputs is part of the expert contraction).
 *
 *   x_dispatched, offsets   as in moe_experts_forward_dispatched.
 *   inv           device, [T * top_k] uint32 (from moe_dispatch).
 *   weights       device, [T, top_k] in `weights_dtype` (from moe_route),
 *                 aligned to its element size.
 *   T, top_k      1 <= top_k <= min(E, 64); rows = T * top_k.
 *   out           device, [T, H] out in the experts' dtype, 16-byte aligned:
 *                 out[t] = sum over j = 0..top_k-1, in that order, of
 *                 w[t, j] * y[inv[t * top_k + j]], FP32 accumulation, then
 *                 rounded to the dtype, y being the expert outputs rounded to
 *                 the dtype. The bits equal moe_experts_forward_dispatched
 *                 followed by moe_combine.
 *   workspace     device scratch of
 *                 moe_experts_forward_combine_workspace_size(experts, T,
 *                 top_k) bytes (h, y_dispatched, the tile counter, one
 *                 counter per expert and the combine's counter), 256-byte
 *                 aligned.
 *
 * How: every epilogue warp of every down tile raises one done counter once
 * its y rows are stored; a CTA that has run out of tiles waits (bounded,
 * about a second: on timeout the device status word records 0x1A) until the
 * counter shows every down tile done, then its epilogue warps combine a
 * fixed stripe of the tokens, four tokens' slot rows in one stream of loads
 * per warp. It waits only on tiles already claimed by running CTAs, so it
 * cannot deadlock. The counters are reset on the stream first. F16/BF16
 * experts and top_k <= 64 only (else MOE_ERR_UNSUPPORTED; use
 * moe_experts_forward_dispatched and moe_combine). An inv entry >= rows
 * makes its token's row NaN, as in moe_combine.
 */
size_t moe_experts_forward_combine_workspace_size(const moe_experts* experts, int64_t T, int32_t top_k);
moe_status moe_experts_forward_combine(const moe_experts* experts, const void* x_dispatched,
                                       const uint32_t* offsets, const uint32_t* inv, const void* weights,
                                       moe_dtype weights_dtype, int64_t T, int32_t top_k, void* out,
                                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * moe_experts_gate_up / moe_experts_down - the two grouped-GEMM stages of
 * moe_experts_forward_dispatched, for callers that want h or want to time or
 * schedule the stages apart. Same arguments and checks as above.
 *
 *   gate_up:  x_dispatched [rows, H] -> h [rows, I],
 *             h = SiLU(W_gate[e] x) * (W_up[e] x), FP32 accumulation, rounded
 *             to the experts' dtype.
 *   down:     h [rows, I] -> y_dispatched [rows, H], y = W_down[e] h.
 *   workspace at least 256 bytes, 256-byte aligned (the tensor-core kernels'
 *             tile counter, reset on the stream by each call); two calls
 *             that may run at the same time need separate workspaces.
 */
moe_status moe_experts_gate_up(const moe_experts* experts, const void* x_dispatched,
                               const uint32_t* offsets, int64_t rows, void* h, void* workspace,
                               size_t workspace_bytes, void* stream);
moe_status moe_experts_down(const moe_experts* experts, const void* h, const uint32_t* offsets,
                            int64_t rows, void* y_dispatched, void* workspace, size_t workspace_bytes,
                            void* stream);

/*
 * moe_experts_gate_up_gather - the gate/up stage reading each dispatched row
 * straight from x: row r is x[row_src[r] / top_k] (row_src from
 * moe_dispatch), so no x_dispatched copy is needed. This is the stage
 * moe_forward runs; the pages have no separate entry for it (their split API
 * materialises x_dispatched). h is bit-identical to moe_experts_gate_up on
 * the x_dispatched that moe_dispatch would write.
 *
 *   x         device, [T, H] in the experts' dtype (16-byte aligned for F16/BF16).
 *   row_src   device, [rows] uint32 from moe_dispatch; an entry >= T * top_k
 *             reads as a zero row.
 *   top_k     >= 1; rows <= T * top_k.
 *   offsets, rows, h, workspace   as in moe_experts_gate_up.
 */
moe_status moe_experts_gate_up_gather(const moe_experts* experts, const void* x, int64_t T,
                                      const uint32_t* row_src, int32_t top_k, const uint32_t* offsets,
                                      int64_t rows, void* h, void* workspace, size_t workspace_bytes,
                                      void* stream);

/*
 * moe_combine - restore token order and take the routing-weighted sum
 * (DispatchedTokens::combine; ruDNN user guide section 6: combine uses the
 * dispatch mapping to restore token order and merges the expert outputs with
 * the routing weights).
 *
 *   y_dispatched  device, [T * top_k, H] in `dtype`.
 *   inv           device, [T * top_k] uint32 (from moe_dispatch).
 *   weights       device, [T, top_k] in `weights_dtype` (from moe_route).
 *   out           device, [T, H] out in `dtype`:
 *                 out[t] = sum over j = 0..top_k-1, in that order, of
 *                 w[t, j] * y[inv[t * top_k + j]], FP32 accumulation, then
 *                 rounded to `dtype`. Deterministic: no atomics.
 */
moe_status moe_combine(const void* y_dispatched, moe_dtype dtype, const uint32_t* inv,
                       const void* weights, moe_dtype weights_dtype, int64_t T, int32_t top_k,
                       int64_t H, void* out, void* stream);

/*
 * moe_forward - the whole local chain in one call (SwiGluExperts::forward;
 * ruDNN user guide section 6): route, dispatch, SwiGLU experts, combine.
 *
 *   experts       handle from moe_experts_create (its dtype is x's and out's).
 *   x             device, [T, H] in the experts' dtype.
 *   logits        device, [T, E] in `logits_dtype` (E from the handle).
 *   top_k, renormalize   as in moe_route.
 *   out           device, [T, H] out in the experts' dtype.
 *   indices_opt   device [T, top_k] uint32 out, or NULL (kept in workspace).
 *   weights_opt   device [T, top_k] out in `logits_dtype`, or NULL.
 *   workspace     device scratch of moe_forward_workspace_size(experts, T,
 *                 top_k) bytes, 256-byte aligned, uninitialised is fine.
 *
 * Same numerics as calling moe_route, moe_dispatch,
 * moe_experts_forward_dispatched and moe_combine in turn: the outputs are
 * bit-identical to that sequence. F16/BF16 run the two expert GEMMs as one
 * launch (as moe_experts_forward_dispatched does; the dispatch zeroes its
 * counters), then the combine as its own launch (measured faster than the
 * combine inside the experts' launch, moe_experts_forward_combine). For
 * decode-sized batches (T * top_k <= 8 * E) it dispatches the maps only and
 * the gate/up tiles gather x rows through row_src (as
 * moe_experts_gate_up_gather), so x_dispatched is never written.
 */
size_t moe_forward_workspace_size(const moe_experts* experts, int64_t T, int32_t top_k);
moe_status moe_forward(const moe_experts* experts, const void* x, const void* logits,
                       moe_dtype logits_dtype, int64_t T, int32_t top_k, int32_t renormalize,
                       void* out, uint32_t* indices_opt, void* weights_opt, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * moe_forward_host - moe_forward on host buffers: the inputs are copied from
 * host memory into device staging in the workspace, the chain runs, and out
 * is copied back to host memory. Every step is enqueued on `stream` (one
 * cudaMemcpyAsync per copy, then the kernels); nothing synchronises the host.
 *
 *   x_host       host, [T, H] in the experts' dtype.
 *   logits_host  host, [T, E] in `logits_dtype`.
 *   out_host     host, [T, H] out in the experts' dtype.
 *   indices_opt, weights_opt   device outputs as in moe_forward, or NULL.
 *   workspace    device scratch of moe_forward_host_workspace_size(experts,
 *                T, top_k, logits_dtype) bytes, 256-byte aligned.
 *
 * Same outputs as moe_forward on device copies of x and logits (bit for bit).
 * With page-locked host buffers the copies are asynchronous: a caller that
 * runs consecutive batches on two streams with two workspaces overlaps one
 * batch's copies with the other's kernels. Pageable host memory works, but
 * each copy then completes before the call returns. The host buffers stay
 * owned by the caller; they must not be changed (x_host, logits_host) or read
 * (out_host) until the stream has passed the call's work.
 */
size_t moe_forward_host_workspace_size(const moe_experts* experts, int64_t T, int32_t top_k,
                                       moe_dtype logits_dtype);
moe_status moe_forward_host(const moe_experts* experts, const void* x_host, const void* logits_host,
                            moe_dtype logits_dtype, int64_t T, int32_t top_k, int32_t renormalize,
                            void* out_host, uint32_t* indices_opt, void* weights_opt, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * moe_group_routing_options - GroupRoutingOptions of the group-limited
 * sigmoid routing (ruDNN user guide, section 10).
 *
 *   top_k            1..64, at most selected_groups * (E / groups).
 *   groups           1..128 and divides E.
 *   selected_groups  1..groups: groups whose experts may be chosen.
 *   group_top_two    nonzero: a group scores the sum of its two largest
 *                    corrected scores (needs E / groups >= 2); zero: its
 *                    largest corrected score.
 *   renormalize      nonzero: divide the chosen weights by their sum.
 *   scale            finite and > 0: multiplies the weights last.
 */
typedef struct {
  int32_t top_k;
  int32_t groups;
  int32_t selected_groups;
  int32_t group_top_two;
  int32_t renormalize;
  float scale;
} moe_group_routing_options;

/*
 * moe_route_sigmoid_grouped - group-limited, bias-corrected sigmoid routing
 * (route_sigmoid_grouped, ruDNN user guide section 10; the group steps
 * follow the DeepSeek-style routing of "PyTorch general ops").
 *
 *   logits        device, [T, E] in `dtype` (MOE_F32, MOE_F16, MOE_BF16),
 *                 1 <= E <= 1024, T >= 0 (T = 0 enqueues nothing).
 *   bias          device, [E] float (FP32), or NULL for no correction; it
 *                 steers the selection only. 4-byte aligned.
 *   options       host pointer, read during the call only.
 *   indices       device, [T, top_k] uint32 out: slot 0 the largest
 *                 corrected score; ties to the lower id (groups too).
 *   weights       device, [T, top_k] out in `dtype`: the uncorrected sigmoid
 *                 scores of the chosen experts, optionally renormalized,
 *                 times scale, rounded to `dtype` (round to nearest even).
 *   weights_fp32  device, [T, top_k] float out before that rounding, or NULL.
 *
 * Scores are FP32: s = 1 / (1 + exp(-l)), c = s + bias. A row with a NaN
 * logit (or any NaN bias) gets NaN weights and indices 0..top_k-1. A group
 * whose two largest corrected scores are +inf and -inf has a NaN score and
 * ranks below every other group. Errors: MOE_ERR_TOP_K for top_k outside
 * 1..64 or above the selected groups' experts, MOE_ERR_SHAPE for any other
 * option or size out of range, MOE_ERR_DTYPE, MOE_ERR_NULL, MOE_ERR_ALIGNMENT.
 */
moe_status moe_route_sigmoid_grouped(const void* logits, moe_dtype dtype, int64_t T, int64_t E,
                                     const float* bias, const moe_group_routing_options* options,
                                     uint32_t* indices, void* weights, float* weights_fp32, void* stream);

/*
 * moe_route_sigmoid_grouped_dispatch - moe_route_sigmoid_grouped followed by
 * moe_dispatch as one cooperative launch, as moe_route_dispatch is for the
 * softmax routing: every output is the same, bit for bit, as those two calls
 * give. Routing arguments as moe_route_sigmoid_grouped; x, x_dtype, H, the
 * maps and x_dispatched as moe_dispatch; the workspace is
 * moe_route_dispatch_workspace_size(T, E) bytes (256-byte aligned, contents
 * need not be initialised). The grid barrier's wait is bounded as in
 * moe_route_dispatch (status 0x1B).
 */
moe_status moe_route_sigmoid_grouped_dispatch(const void* logits, moe_dtype logits_dtype, int64_t T, int64_t E,
                                              const float* bias, const moe_group_routing_options* options,
                                              uint32_t* indices, void* weights, float* weights_fp32, const void* x,
                                              moe_dtype x_dtype, int64_t H, uint32_t* counts, uint32_t* offsets,
                                              uint32_t* row_src, uint32_t* inv, void* x_dispatched, void* workspace,
                                              size_t workspace_bytes, void* stream);

/*
 * moe_forward_sigmoid_grouped - the whole local chain with grouped sigmoid
 * routing (SwiGluExperts::forward_sigmoid_grouped, ruDNN user guide section
 * 10): the grouped routing and the dispatch (one launch, as
 * moe_route_sigmoid_grouped_dispatch), then SwiGLU experts and combine
 * exactly as moe_forward does. Arguments as in moe_forward, with `bias` and
 * `options` as in moe_route_sigmoid_grouped; the workspace is
 * moe_forward_workspace_size(experts, T, options->top_k) bytes.
 */
moe_status moe_forward_sigmoid_grouped(const moe_experts* experts, const void* x, const void* logits,
                                       moe_dtype logits_dtype, int64_t T, const float* bias,
                                       const moe_group_routing_options* options, void* out,
                                       uint32_t* indices_opt, void* weights_opt, void* workspace,
                                       size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * First-order training (ruDNN user guide, section 12). The backward runs in
 * the order the guide gives: combine_backward -> experts backward (the
 * forward cache's backward) -> dispatch_backward, and the FP32 dweights go
 * to moe_router_backward for the logits gradient.
 * ---------------------------------------------------------------------- */

typedef enum { MOE_ROUTER_SOFTMAX = 0, MOE_ROUTER_SIGMOID = 1 } moe_router_scoring;
typedef enum { MOE_INDEX_U32 = 0, MOE_INDEX_I32 = 1, MOE_INDEX_I64 = 2 } moe_index_type;

/* RouterWeightOptions: scoring, renormalize over the selected slots, and a
 * finite positive scale applied last. */
typedef struct {
  int32_t scoring;      /* moe_router_scoring */
  int32_t renormalize;  /* nonzero: divide by the sum over the slots */
  float scale;
} moe_router_weight_options;

/*
 * moe_router_weights - selected_router_weights: FP32 weights of a fixed
 * selection. Softmax: the FP32 softmax over all E experts (as moe_route
 * computes it) at each selected index; sigmoid: 1 / (1 + exp(-l)) of each
 * selected logit. Then optional renormalize (slot-ordered FP32 sum), then
 * times scale.
 *
 *   logits    device [T, E] in `dtype` (1 <= E <= 1024).
 *   indices   device [T, top_k] in `index_type` (uint32, int32 or int64),
 *             1 <= top_k <= min(E, 64). Repeated indices gather; any index
 *             outside 0..E-1 makes the token's whole row NaN (no out-of-range
 *             access, no host synchronisation).
 *   weights   device [T, top_k] float out.
 */
moe_status moe_router_weights(const void* logits, moe_dtype dtype, int64_t T, int64_t E, const void* indices,
                              moe_index_type index_type, int32_t top_k, const moe_router_weight_options* options,
                              float* weights, void* stream);

/*
 * moe_router_backward - selected_router_backward: dlogits [T, E] in the
 * logits dtype, the gradient of the moe_router_weights output (given as
 * FP32 grad_weights [T, top_k]) with respect to the logits, for the fixed
 * selection (the top-k itself, group choice and correction bias are not
 * differentiated). Every entry of dlogits is written. Same checks as
 * moe_router_weights; an invalid index makes the row of dlogits NaN.
 */
moe_status moe_router_backward(const void* logits, moe_dtype dtype, int64_t T, int64_t E, const void* indices,
                               moe_index_type index_type, int32_t top_k, const moe_router_weight_options* options,
                               const float* grad_weights, void* dlogits, void* stream);

/*
 * moe_experts_forward_training - forward_dispatched_training: the experts'
 * forward that also keeps the cache the backward needs.
 *
 *   x_dispatched, offsets, rows   as in moe_experts_forward_dispatched.
 *   h             device [rows, I] out: SiLU(g) * u in the dtype.
 *   y_dispatched  device [rows, H] out.
 *   cache_g, cache_u  device [rows, I] out: the pre-activations g = W_gate x
 *                 and u = W_up x, rounded to the dtype.
 *   workspace     device scratch of
 *                 moe_experts_forward_training_workspace_size(experts) bytes
 *                 (the GEMMs' counters), 256-byte aligned.
 * y_dispatched and h are bit-identical to moe_experts_forward_dispatched's
 * (F16/BF16: the same chained launch, whose gate/up tiles also store g, u).
 */
size_t moe_experts_forward_training_workspace_size(const moe_experts* experts);
moe_status moe_experts_forward_training(const moe_experts* experts, const void* x_dispatched,
                                        const uint32_t* offsets, int64_t rows, void* h, void* y_dispatched,
                                        void* cache_g, void* cache_u, void* workspace, size_t workspace_bytes,
                                        void* stream);

/*
 * moe_combine_backward - combine_backward: for each token t and slot j with
 * r = inv[t * top_k + j]: dexpert[r] = w[t, j] * grad_out[t] (rounded to the
 * dtype) and dweights[t, j] = <grad_out[t], y[r]> (FP32). A slot whose inv
 * entry is >= T * top_k gets a NaN dweight and writes no dexpert row;
 * dexpert rows no slot points at are not written.
 *
 *   y_dispatched  device [T * top_k, H] in `dtype` (the forward's expert output).
 *   inv, row_src  device [T * top_k] uint32, the two maps of moe_dispatch
 *                 (slot -> row and row -> slot). The work runs in row order;
 *                 a row r counts only when inv[row_src[r]] == r, so the
 *                 entries of row_src past the dispatched rows may hold
 *                 anything.
 *   weights       device [T, top_k] in `weights_dtype` (the forward's weights).
 *   grad_out      device [T, H] in `dtype`.
 *   dexpert       device [T * top_k, H] out in `dtype`.
 *   dweights      device [T, top_k] float out.
 */
moe_status moe_combine_backward(const void* y_dispatched, moe_dtype dtype, const uint32_t* inv,
                                const uint32_t* row_src, const void* weights, moe_dtype weights_dtype,
                                const void* grad_out, int64_t T, int32_t top_k, int64_t H, void* dexpert,
                                float* dweights, void* stream);

/*
 * moe_experts_backward - the forward cache's backward: from dexpert [rows, H]
 * (dy), the dispatched input gradient dx_dispatched [rows, H] (dtype) and the
 * FP32 weight gradients dgate, dup [E, I, H] and ddown [E, H, I] (every
 * entry written; experts without rows get zeros):
 *   dh = W_down^T dy; dg = dh * u * SiLU'(g); du = dh * SiLU(g);
 *   dx = W_gate^T dg + W_up^T du; ddown = dy h^T; dgate = dg x^T; dup = du x^T.
 *   workspace  moe_experts_backward_workspace_size(experts, rows) bytes,
 *              256-byte aligned (dg and du in the dtype; F32 experts also
 *              keep dh there in FP32, F16/BF16 experts turn dh into dg and du
 *              inside the dgrad GEMM).
 */
size_t moe_experts_backward_workspace_size(const moe_experts* experts, int64_t rows);
moe_status moe_experts_backward(const moe_experts* experts, const void* x_dispatched, const uint32_t* offsets,
                                int64_t rows, const void* h, const void* cache_g, const void* cache_u,
                                const void* dexpert, void* dx_dispatched, float* dgate, float* dup, float* ddown,
                                void* workspace, size_t workspace_bytes, void* stream);

/*
 * moe_dispatch_backward - dispatch_backward: dx[t] = sum over slots j of
 * dinput[inv[t * top_k + j]], added in slot order in FP32 and rounded to the
 * dtype; the routing weight is not applied again. A token with an inv entry
 * >= T * top_k gets a NaN row.
 */
moe_status moe_dispatch_backward(const void* dinput, moe_dtype dtype, const uint32_t* inv, int64_t T, int32_t top_k,
                                 int64_t H, void* dx, void* stream);

/* ------------------------------------------------------------------------
 * Experts in microscaled 4-bit floating point (MXFP4, OCP Microscaling
 * Formats v1.0: blocks of 32 E2M1 elements with one E8M0 scale). The pages
 * have float experts only; these entry points are added beside them.
 *
 * Layout of an MXFP4 matrix [rows, K], K a multiple of 32:
 *   codes    [rows, K / 2] bytes: element 2i in the low, 2i + 1 in the high
 *            four bits of byte i; bit 3 is the sign, 0..7 stand for 0, 0.5, 1,
 *            1.5, 2, 3, 4, 6. 16-byte aligned.
 *   scales   [rows, moe_mxfp4_scale_pitch(K)] bytes: byte b < K / 32 of a row
 *            is the scale 2^(byte - 127) of its elements 32b .. 32b + 31, 255
 *            is NaN. The pitch is K / 32 rounded up to 4; the bytes past K / 32
 *            are written as 0 and never read. 4-byte aligned. (Scales made
 *            elsewhere with K / 32 bytes a row have to be copied to this
 *            pitch where K / 32 is not a multiple of 4.)
 * ---------------------------------------------------------------------- */

/* 4 * ceil(K / 128), or 0 where K is not a positive multiple of 32. */
int64_t moe_mxfp4_scale_pitch(int64_t K);

/*
 * moe_mxfp4_quantize - float rows to MXFP4, optionally straight into
 * dispatched order.
 *
 *   x         device, [rows, K] in `dtype`, 16-byte aligned.
 *   K         a multiple of 32, 32 .. 262144.
 *   inv       NULL: row r is written to row r (top_k must be 1). Else device,
 *             [rows * top_k] uint32, moe_dispatch's slot -> row map: row t is
 *             written to the rows inv[t * top_k + j], j < top_k, and codes and
 *             scales hold rows * top_k rows. An entry >= rows * top_k is
 *             skipped; rows that no entry names are left as they were; a row
 *             that two entries name (moe_dispatch's maps have none) ends with
 *             bytes of either.
 *   codes, scales   device, out (layout above).
 *
 * For a block with a = max |x_i|: byte = clamp(floor(log2 a) - 2 + 127, 0,
 * 254) (0 where a = 0); each element is x_i / 2^(byte - 127) rounded to the
 * nearest E2M1 value, ties to the even mantissa, saturated to 6. A block that
 * holds a NaN or an infinity gets byte 255 and zero codes.
 * Errors: MOE_ERR_DTYPE, MOE_ERR_SHAPE, MOE_ERR_TOP_K, MOE_ERR_NULL,
 * MOE_ERR_ALIGNMENT.
 */
moe_status moe_mxfp4_quantize(const void* x, moe_dtype dtype, int64_t rows, int64_t K, const uint32_t* inv,
                              int32_t top_k, void* codes, void* scales, void* stream);

/*
 * moe_mxfp4_dequantize - the values an MXFP4 matrix stands for, [rows, K] in
 * `dtype` (16-byte aligned), rounded to nearest even (exact in F32 but for
 * scales above 2^125, whose largest elements overflow to infinity).
 */
moe_status moe_mxfp4_dequantize(const void* codes, const void* scales, int64_t rows, int64_t K, void* out,
                                moe_dtype dtype, void* stream);

/* Opaque handle of MXFP4 expert weights. */
typedef struct moe_experts_mxfp4 moe_experts_mxfp4;

/*
 * moe_experts_mxfp4_create - validate and wrap bias-free SwiGLU expert
 * weights in MXFP4: gate and up [E, I, H], down [E, H, I] (as E * I, or E * H
 * rows of the layout above).
 *
 *   E, H, I       1 <= E <= 1024; H and I multiples of 32, 32 .. 262144.
 *   storage       device, moe_experts_mxfp4_storage_size(E, H, I) bytes,
 *                 256-byte aligned: the weights' scales in the tensor cores'
 *                 order, written by kernels enqueued on `stream`; uses of the
 *                 handle on other streams have to be ordered after them.
 *   out           receives the handle.
 *
 * The handle keeps the code pointers and `storage` (the caller keeps them
 * alive and unchanged); the scale arrays are not used after the stream has
 * passed the call. It is read-only and may be shared between streams; free it
 * with moe_experts_mxfp4_destroy. Device is the current device at creation.
 */
size_t moe_experts_mxfp4_storage_size(int64_t E, int64_t H, int64_t I);
moe_status moe_experts_mxfp4_create(const void* gate_codes, const void* gate_scales, const void* up_codes,
                                    const void* up_scales, const void* down_codes, const void* down_scales, int64_t E,
                                    int64_t H, int64_t I, void* storage, size_t storage_bytes, void* stream,
                                    moe_experts_mxfp4** out);
void moe_experts_mxfp4_destroy(moe_experts_mxfp4* experts);

/*
 * moe_experts_mxfp4_gate_up - h = SiLU(W_gate[e] x) * (W_up[e] x) on
 * dispatched MXFP4 rows, FP32 accumulation.
 *
 *   x_codes, x_scales   device, MXFP4 [rows, H] (moe_mxfp4_quantize with inv).
 *   offsets       device, [E + 1] uint32 (from moe_dispatch), ascending.
 *   rows          rows of the buffers, at most 2^31 - 1024; offsets[E] of them
 *                 are computed, the others are left as they were.
 *   h             device, [rows, I] out in `dtype`, or NULL.
 *   h_codes, h_scales   device, MXFP4 [rows, I] out, or both NULL: h rounded
 *                 to `dtype` and then quantised, the same bytes as
 *                 moe_mxfp4_quantize gives on h. At least one of the two
 *                 outputs is needed.
 *   dtype         MOE_F32, MOE_F16 or MOE_BF16.
 *
 * No workspace. A row with a NaN block gives NaN outputs for its token only.
 * SiLU's relative error: below 2^-20 for FP32 h, 2^-20 + |g| 2^-23 for 16-bit
 * h (the hardware's exponential), and 2^-142 more; a SiLU below 2^-126, where
 * g < -92, may count as 0.
 */
moe_status moe_experts_mxfp4_gate_up(const moe_experts_mxfp4* experts, const void* x_codes, const void* x_scales,
                                     const uint32_t* offsets, int64_t rows, moe_dtype dtype, void* h, void* h_codes,
                                     void* h_scales, void* stream);

/* moe_experts_mxfp4_down - y = W_down[e] h on MXFP4 [rows, I] -> [rows, H] in
 * `dtype`, FP32 accumulation. Arguments as moe_experts_mxfp4_gate_up. */
moe_status moe_experts_mxfp4_down(const moe_experts_mxfp4* experts, const void* h_codes, const void* h_scales,
                                  const uint32_t* offsets, int64_t rows, moe_dtype dtype, void* y, void* stream);

/*
 * moe_experts_mxfp4_forward_dispatched - both stages: h goes from gate/up to
 * down as MXFP4 (rounded to `dtype` before). The same bits as
 * moe_experts_mxfp4_gate_up with h_codes followed by moe_experts_mxfp4_down.
 *   workspace     device, moe_experts_mxfp4_forward_dispatched_workspace_size
 *                 bytes (h as MXFP4), 256-byte aligned.
 */
size_t moe_experts_mxfp4_forward_dispatched_workspace_size(const moe_experts_mxfp4* experts, int64_t rows);
moe_status moe_experts_mxfp4_forward_dispatched(const moe_experts_mxfp4* experts, const void* x_codes,
                                                const void* x_scales, const uint32_t* offsets, int64_t rows,
                                                moe_dtype dtype, void* y, void* workspace, size_t workspace_bytes,
                                                void* stream);

/*
 * moe_forward_mxfp4 - the whole local chain on MXFP4 experts: route +
 * dispatch (one launch, as moe_forward), x quantised into dispatched order,
 * the two expert products, combine. The same bits as moe_route_dispatch,
 * moe_mxfp4_quantize (with inv), moe_experts_mxfp4_forward_dispatched and
 * moe_combine in turn.
 *
 *   x, out        device, [T, H] in `dtype` (MOE_F32, MOE_F16, MOE_BF16),
 *                 16-byte aligned; h is rounded to `dtype` before it is
 *                 quantised (in MOE_F16 an h beyond 65504 is an infinity, as
 *                 in moe_forward, and its block of 32 channels NaN).
 *   logits, logits_dtype, T, top_k, renormalize, indices_opt, weights_opt
 *                 as in moe_forward.
 *   workspace     device, moe_forward_mxfp4_workspace_size(experts, T, top_k,
 *                 dtype) bytes, 256-byte aligned.
 */
size_t moe_forward_mxfp4_workspace_size(const moe_experts_mxfp4* experts, int64_t T, int32_t top_k, moe_dtype dtype);
moe_status moe_forward_mxfp4(const moe_experts_mxfp4* experts, const void* x, moe_dtype dtype, const void* logits,
                             moe_dtype logits_dtype, int64_t T, int32_t top_k, int32_t renormalize, void* out,
                             uint32_t* indices_opt, void* weights_opt, void* workspace, size_t workspace_bytes,
                             void* stream);

/* ------------------------------------------------------------------------
 * Gradient norm and clipping over many tensors: what a training step runs
 * between the backward (moe_experts_backward's dgate, dup, ddown and the
 * caller's other gradients) and the optimizer. Added beside the pages'
 * training calls.
 * ---------------------------------------------------------------------- */

/* One dense gradient of `numel` elements (0 is allowed), aligned to its
 * element size. `dst` is used by moe_grad_clip only: where the clipped
 * gradient goes, src itself to clip in place. */
typedef struct {
  const void* src;
  void* dst;
  int64_t numel;
  int32_t dtype;  /* moe_dtype of src and dst */
} moe_grad_tensor;

/*
 * moe_grad_norm - the L2 norm over all elements of n tensors.
 *
 *   tensors    host, n entries, read during the call only (n >= 0).
 *   norm       device, one float out: sqrt of the sum of squares (a thread's
 *              16 or 32 squares in FP32, its running sum as a compensated FP32
 *              pair, or in FP64 where FP32 does not hold the squares; threads
 *              and blocks in FP64; the same bits on every run). 0 without
 *              elements; NaN or infinity where the gradients hold one,
 *              infinity also where the norm exceeds FP32.
 *   workspace  device, moe_grad_norm_workspace_size(n) bytes, 256-byte
 *              aligned; contents need not be initialised. Calls that may
 *              overlap need separate workspaces.
 */
size_t moe_grad_norm_workspace_size(int64_t n);
moe_status moe_grad_norm(const moe_grad_tensor* tensors, int64_t n, float* norm, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * moe_grad_clip - dst = src * max_norm / norm for every tensor if norm is
 * finite and larger than max_norm; otherwise dst = src (in place: nothing is
 * written). FP32 arithmetic, rounded to the tensor's dtype.
 *
 *   norm       device, one float: moe_grad_norm's result, or that of a larger
 *              set of gradients (for sharded experts, the root of the ranks'
 *              summed squares). A NaN or infinite norm leaves the gradients as
 *              they are: the caller sees it in *norm and skips the step.
 *   max_norm   finite and >= 0.
 *
 * dst ranges must not overlap one another, another entry's src or norm, and a
 * dst that is not its own src must not overlap it (MOE_ERR_SHAPE).
 */
moe_status moe_grad_clip(const moe_grad_tensor* tensors, int64_t n, const float* norm, float max_norm, void* stream);

/* ------------------------------------------------------------------------
 * The norms around a block of a residual stream: before the layer (its input),
 * after it (its output, gated and scaled, back into the stream) and the next
 * block's, forward and backward. Not on the pages, which stop at the layer.
 *
 *   norm(v; w) = v * w / sqrt(mean(v^2) + eps)      over the H columns of a row
 *
 * Rows are [T, H] in `dtype`, H <= 32768, aligned to their element size (16-byte
 * aligned rows, H a multiple of 8, take the wide loads). Weight vectors are
 * MOE_F32 or of the rows' dtype. Arithmetic and sums are FP32, each output is
 * rounded once; a row whose sum of squares passes FP32's range is normed to
 * zeros. An output may be the same [T, H] tensor as an input; any other overlap
 * with an output is MOE_ERR_SHAPE. Gradients of weights and channel gates are
 * FP32; every sum has a fixed order (the same bits on every run).
 * ---------------------------------------------------------------------- */

/*
 * moe_block_norm - y = norm(x; weight).
 *   x, y      device, [T, H] in `dtype` (T = 0 enqueues nothing).
 *   weight    device, [H] in `weight_dtype`.
 *   eps       finite, > 0.
 */
moe_status moe_block_norm(const void* x, moe_dtype dtype, const void* weight, moe_dtype weight_dtype, float eps,
                          int64_t T, int64_t H, void* y, void* stream);

/*
 * moe_block_norm_backward - from dy: dx = (dy's gradient of x) + dresidual, and
 * dweight[h] = sum over rows of dy * x / sqrt(mean(x^2) + eps).
 *   eps         the forward's, at least 2^-80.
 *   dresidual   device, [T, H]: the gradient that reaches x past the block, or
 *               NULL for none.
 *   dx          device, [T, H] out in `dtype`.
 *   dweight     device, [H] float out (zeros for T = 0).
 *   workspace   device, moe_block_norm_backward_workspace_size(T, H) bytes,
 *               256-byte aligned; contents need not be initialised.
 */
size_t moe_block_norm_backward_workspace_size(int64_t T, int64_t H);
moe_status moe_block_norm_backward(const void* dy, const void* x, moe_dtype dtype, const void* weight,
                                   moe_dtype weight_dtype, const void* dresidual, float eps, int64_t T, int64_t H,
                                   void* dx, float* dweight, void* workspace, size_t workspace_bytes, void* stream);

/* What a join's gate is shared by. */
typedef enum {
  MOE_GATE_NONE = 0,
  MOE_GATE_CHANNEL = 1,  /* [H], in vec_dtype      */
  MOE_GATE_TOKEN = 2,    /* [T], in vec_dtype      */
  MOE_GATE_ELEMENT = 3   /* [T, H], in the rows' dtype */
} moe_gate_kind;

typedef struct {
  const void* norm_weight;  /* device, [H], or NULL: the branch is not normed   */
  const void* next_weight;  /* device, [H], or NULL: no norm of the joined rows */
  const void* gate;         /* device, by gate_kind                             */
  int32_t gate_kind;        /* moe_gate_kind                                    */
  int32_t vec_dtype;        /* of norm_weight, next_weight, channel and token gates: MOE_F32 or the rows' dtype */
  float residual_scale;     /* finite */
  float branch_scale;       /* finite */
  float eps;                /* of both norms; finite, > 0 */
} moe_block_join_params;

/*
 * moe_block_join - the block's output back into the residual stream, and the
 * next block's norm:
 *   out    = residual_scale * residual + branch_scale * gate * norm(branch; norm_weight)
 *   normed = norm(out; next_weight), of out as stored
 *   branch, residual, out   device, [T, H] in `dtype`.
 *   params    host, read during the call only.
 *   normed    device, [T, H] out, exactly when next_weight is given.
 */
moe_status moe_block_join(const void* branch, const void* residual, moe_dtype dtype, const moe_block_join_params* params,
                          int64_t T, int64_t H, void* out, void* normed, void* stream);

/*
 * moe_combine_join - moe_combine and moe_block_join in one launch: the branch
 * is sum over slots j, in order, of weights[t, j] * y_dispatched[inv[t * top_k
 * + j]] in FP32 (not rounded to `dtype` in between, as moe_combine's result
 * is). A token with an inv entry >= T * top_k gets NaN rows.
 *   y_dispatched, inv, weights, weights_dtype, top_k   as moe_combine.
 */
moe_status moe_combine_join(const void* y_dispatched, moe_dtype dtype, const uint32_t* inv, const void* weights,
                            moe_dtype weights_dtype, const void* residual, const moe_block_join_params* params,
                            int64_t T, int32_t top_k, int64_t H, void* out, void* normed, void* stream);

/*
 * moe_block_join_backward - from dout (the gradient that reaches out past the
 * next norm; NULL for none, with next_weight only) and dnormed:
 *   dbranch, dresidual   device, [T, H] out in `dtype`.
 *   dnorm_weight, dnext_weight   device, [H] float out, exactly when their
 *             weights are given.
 *   dgate     device, out, exactly when there is a gate: [H] or [T] float, or
 *             [T, H] in `dtype`.
 *   params    the forward's, with eps at least 2^-80.
 *   branch    the forward's (moe_combine's result for a combined branch).
 *   joined    the forward's out; it and dnormed are read with next_weight only.
 *   workspace moe_block_join_backward_workspace_size(T, H) bytes, 256-byte
 *             aligned.
 */
size_t moe_block_join_backward_workspace_size(int64_t T, int64_t H);
moe_status moe_block_join_backward(const void* dout, const void* dnormed, const void* branch, const void* joined,
                                   moe_dtype dtype, const moe_block_join_params* params, int64_t T, int64_t H,
                                   void* dbranch, void* dresidual, float* dnorm_weight, void* dgate,
                                   float* dnext_weight, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Orthogonalised updates: what a training step runs between the gradients
 * (moe_experts_backward's dgate, dup, ddown, clipped) and the weights. Added
 * beside the pages' training calls.
 *
 * Newton-Schulz steps on each matrix G of a batch [E, rows, cols]:
 *   X = G / (|G|_F + eps), then `steps` times, with A = X X^T,
 *   X <- 3.4445 X + (-4.7750 A + 2.0315 A A) X
 * (five steps take the singular values that are not much below the largest
 * into about [0.7, 1.2] and keep the singular vectors). Products run on the
 * tensor cores with FP16 pairs as operands (22 bits) and FP32 accumulators:
 * the result is right to about its type's rounding, to some 2^-13 (2-norm over
 * the matrix) where it goes into FP32 weights. A matrix with a NaN or an
 * infinity becomes NaN as a whole, the others of the batch are not touched by
 * it; a matrix of zeros stays zero.
 *
 *   E           0 .. 65535 matrices, dense, one behind the other.
 *   rows, cols  0 .. 65536, either may be the longer (no element: nothing is
 *               enqueued); E times the square of max(rows, cols) / 128, rounded
 *               up, at most 2^31 - 1.
 *   steps       1 .. 100.
 *   eps         finite, > 0. Entries of X under 2^-38 count as zero: a matrix
 *               whose norm is that far below eps comes out as zeros.
 *   workspace   device, moe_orthogonalize_workspace_size(E, rows, cols) bytes,
 *               256-byte aligned, of both calls below: about 8 bytes per
 *               element, 16 min(rows, cols)^2 per matrix, and up to 34 MB for
 *               batches of few matrices. Contents need not be initialised.
 *               Calls that may overlap need separate ones.
 * Tensors are aligned to their element size. The same bits on every run.
 * ---------------------------------------------------------------------- */
size_t moe_orthogonalize_workspace_size(int64_t E, int64_t rows, int64_t cols);

/*
 * moe_orthogonalize - out = the orthogonalised matrices.
 *   matrices   device, [E, rows, cols] in `dtype`.
 *   out        device, the same shape in out_dtype, MOE_F16 or MOE_BF16 (the
 *              steps' accuracy is that of 16-bit results, so FP32 is not
 *              offered); may be the matrices' own memory.
 */
moe_status moe_orthogonalize(const void* matrices, moe_dtype dtype, int64_t E, int64_t rows, int64_t cols,
                             int32_t steps, float eps, void* out, moe_dtype out_dtype, void* workspace,
                             size_t workspace_bytes, void* stream);

typedef struct {
  float lr;               /* finite, as lr * weight_decay and lr * update_scale */
  float momentum_decay;   /* in [0, 1) */
  float weight_decay;     /* finite */
  float update_scale;     /* finite; commonly sqrt(max(1, rows / cols)) */
  float eps;
  int32_t steps;
  int32_t nesterov;       /* nonzero: orthogonalise grad + momentum_decay * momentum, else the momentum */
} moe_muon_params;

/*
 * moe_muon_step - one optimizer step on a batch of weight matrices:
 *   momentum <- momentum_decay * momentum + grad
 *   O = the orthogonalised (nesterov ? grad + momentum_decay * momentum : momentum)
 *   weight <- (1 - lr * weight_decay) * weight - lr * update_scale * O
 * in FP32 (O is not rounded in between), weight rounded to its dtype once.
 *   weight     device, [E, rows, cols] in weight_dtype, updated in place.
 *   grad       device, in grad_dtype.
 *   momentum   device, float, updated in place (zeros before the first step).
 * A matrix whose grad or momentum holds a NaN or an infinity gets NaN weights:
 * moe_grad_norm tells before the step.
 *   params     host, read during the call only.
 * The tensors and the workspace must not overlap. A call that fails leaves them
 * as they were, unless a launch after its first was rejected (MOE_ERR_CUDA):
 * then the momentum may have been updated.
 */
moe_status moe_muon_step(void* weight, moe_dtype weight_dtype, const void* grad, moe_dtype grad_dtype, float* momentum,
                         int64_t E, int64_t rows, int64_t cols, const moe_muon_params* params, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * moe_device_status - read (and clear, if `clear` is nonzero) the device
 * status word. The expert GEMM kernels bound every pipeline wait (about one
 * second); a wait that runs out stops its kernel's remaining work, lets the
 * copies and MMAs already issued finish, frees its tensor memory, returns,
 * and records a code here instead of hanging the GPU. Codes (first one
 * wins): 0x11 producer waiting for a free stage, 0x12 MMA waiting for a
 * loaded stage, 0x13 MMA waiting for a drained accumulator, 0x14 epilogue
 * waiting for a finished accumulator, 0x15 / 0x16 teardown drains, 0x17 a
 * wait on the shared-memory tile ring of the tile scheduler, 0x18 a gather
 * loader waiting for a free stage, 0x19 a down tile of the chained gate/up +
 * down launch waiting for its expert's h rows, 0x1A the combine of
 * moe_experts_forward_combine waiting for the last down tile, 0x1B the grid
 * barrier of moe_route_dispatch and moe_route_sigmoid_grouped_dispatch (and
 * of the forward calls' routing), 0x31 - 0x3B the waits of the MXFP4 expert
 * products (0x31 producer, 0x32 MMA for a loaded stage, 0x33 MMA for a drained
 * accumulator, 0x34 epilogue, 0x35 / 0x36 teardown drains, 0x37 scale loader
 * for a free ring slot, 0x38 scale warps for a free scale buffer, 0x39 for a
 * loaded ring slot, 0x3A MMA for a stage's scales, 0x3B a teardown drain of
 * the scale loader), 0x41 - 0x47 the waits of the Newton-Schulz products (0x41
 * producer, 0x42 MMA for a loaded stage, 0x43 MMA for a drained accumulator,
 * 0x44 epilogue, 0x45 / 0x46 teardown drains, 0x47 a product of the one-launch
 * kernel), 0x51 / 0x52 the norms around a
 * block waiting for their rows, 0x100 moe_selftest_bounded_wait. Synchronises
 * the current device; *code = 0 when no wait has timed out.
 */
moe_status moe_device_status(uint32_t* code, int32_t clear);

/*
 * moe_selftest_bounded_wait - launch one thread that waits on an mbarrier
 * nothing ever arrives on, with a limit of `limit_us` microseconds
 * (1 .. 10^7). The wait gives up, records 0x100 in the device status word
 * and the kernel returns; the CUDA context stays usable. Exercises the same
 * bounded-wait routine the expert GEMMs use.
 */
moe_status moe_selftest_bounded_wait(uint32_t limit_us, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
