/*
 * tlq.h -- C ABI of the GB300 (sm_103a) weight-only quantized linear layer.
 *
 * One shared library (libtlq.so) implements the hot path of the TinyLoop
 * looped-transformer runtime: the quantized linear layer quant_gemm (routed
 * to the INT4 or INT2 kernels) and the shared-weight loop block that reapplies
 * one set of projections L times.
 *
 * Data types in this header are plain C: FP16 values are passed as their
 * IEEE-754 binary16 bit patterns (uint16_t), FP32 as float.  Every pointer
 * argument is a DEVICE pointer (cudaMalloc / torch CUDA tensor memory)
 * unless the comment says otherwise; `stream` is a cudaStream_t passed as
 * void* (NULL = the legacy default stream).
 *
 * Conventions shared by every entry point
 *  - Ownership: the caller owns every input, output, scratch and workspace
 *    buffer; the library allocates no device memory in any call.  A GEMM
 *    with M > 16 whose tiles would leave SMs idle splits K over a
 *    thread-block cluster and exchanges partial tiles through an FP32
 *    workspace that the caller passes (tl_quant_gemm_ws, the workspace fields
 *    of tl_gemm_desc, tl_block and tl_swiglu_block); the size it wants comes
 *    from tl_quant_gemm_workspace_size.  With no workspace, or one too small,
 *    the kernel keeps K whole (same arithmetic per output, possibly slower).
 *    tl_loop_block_forward_static_scratch also needs no caller scratch: it
 *    uses a static array the library owns.  Host state: the library keeps
 *    the launch descriptions (tensor maps, work lists) of recent calls, keyed
 *    by their full argument lists, and for tl_quant_gemm_batched up to three
 *    side streams per caller stream; it keeps no device state between calls.
 *  - Ordering: calls are asynchronous and ordered on `stream`.  Apart from
 *    tl_loop_block_forward_static_scratch the library holds no shared
 *    scratch, so calls on different streams with disjoint buffers may run
 *    concurrently; one model instance is meant to drive one
 *    stream ("Model", section "Thread safety": a single CUDA stream for all
 *    forward-pass work).
 *  - Errors: arguments are checked on the host before anything is launched.
 *    A rejected call returns TLQ_EINVAL (bad argument) or TLQ_EUNSUPPORTED
 *    (valid but not implemented, e.g. a group size the kernels do not take)
 *    and launches nothing; a failed launch returns TLQ_ECUDA.  The message of
 *    the last failure on the calling thread names the failing argument or
 *    step ("Model", section "Raises": errors name the failure point).
 *  - Device waits are bounded: a kernel that gives up on a wait records
 *    TLQ_ETIMEOUT in a device status word and returns; tl_check_status()
 *    reports it.
 *  - Determinism: identical inputs give bit-identical outputs on every call
 *    (no floating-point atomics, fixed reduction order) -- "Model", section
 *    "Determinism".
 *  - Environment (read by the library; none is needed): TLQ_LOG=1 prints each
 *    launch's configuration to stderr; TLQ_PDL=0 turns programmatic dependent
 *    launch off; TLQ_PREFILL_NMT=1|2, TLQ_PREFILL_KSPLIT=1|2|4|8 and
 *    TLQ_DECODE_ROWS=16|32|64 force the kernels' tiling choices (for tests
 *    and measurements; the results of the decode kernel do not depend on
 *    TLQ_DECODE_ROWS); TLQ_DECODE_GENERIC=1 and TLQ_PREFILL_GENERIC=1 force
 *    the kernels' general forms instead of the forms built for whole blocks
 *    (the same results, bit for bit).
 */
#ifndef TLQ_H_
#define TLQ_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  TLQ_OK = 0,
  TLQ_EINVAL = 1,       /* an argument is invalid; nothing was launched      */
  TLQ_EUNSUPPORTED = 2, /* valid request this build does not implement       */
  TLQ_ECUDA = 3,        /* a CUDA runtime/driver call failed                 */
  TLQ_ETIMEOUT = 4      /* a device-side wait hit its limit (see status)     */
} tlq_status;

/* Message of the last failure on the calling thread ("" if none).  The
 * string is owned by the library and valid until the next call on the same
 * thread. */
const char* tl_last_error(void);

/* Library version string, e.g. "tlq 0.1 sm_103a". */
const char* tl_version(void);

/*
 * tl_quant_gemm -- the quantized linear layer (quant_gemm).
 *
 *   C[m][n] = fp16( sum_k A[m][k] * w[n][k] ),  w[n][k] = (q[n][k] - z[n][g]) * s[n][g],
 *   g = k / group, accumulated in FP32 on the GPU.
 *
 * Source: "Model" (TinyLoop Python API), "VRAM cost", Weights -- each
 * quantized layer holds INT2 / INT4 packed data, FP16 scales and FP16 zeros;
 * "beta-Informed Deployment Features", CTX-TIER, "What Phase 2 ships" -- the
 * dispatcher routes on the weight's bit width (INT4 kernel or int2_gemm).
 *
 *   A       FP16 [M][K], row-major, row stride K elements, 16-byte aligned.
 *   Wpacked uint32 [N][K*bits/32], the format tl_pack_weights writes: row n
 *           is K-contiguous, code j of a word at bits [bits*j, bits*j+bits).
 *           16-byte aligned.
 *   scales  FP16 [N][K/group], row-major.
 *   zeros   FP16 [N][K/group], row-major (zero points, need not be integral).
 *   C       FP16 [M][N], row-major, row stride N; must not overlap A.
 *   M >= 1; N >= 1 and a multiple of 8; K >= 1 with K % group == 0.
 *   bits    4 or 2.
 *   group   a multiple of 32 (bits = 4) or 64 (bits = 2), dividing K;
 *           group = K (one scale per row) is allowed.
 *   M <= 16 runs the bandwidth-bound decode kernel, larger M the tensor-core
 *   (tcgen05) prefill kernel, here without a k split (no workspace; see
 *   tl_quant_gemm_ws).
 * Returns TLQ_OK, TLQ_EINVAL (null pointer, misalignment, bad shape/bits/
 * group), or TLQ_ECUDA.
 */
tlq_status tl_quant_gemm(const uint16_t* A, const uint32_t* Wpacked, const uint16_t* scales,
                         const uint16_t* zeros, uint16_t* C, int M, int N, int K, int bits,
                         int group, void* stream);

/*
 * tl_quant_gemm_workspace_size -- bytes of FP32 workspace with which the
 * tensor-core kernel would split K for this problem (its planner's choice
 * with no limit on the workspace); 0 when it would not split (always for
 * M <= 16) or for an invalid shape.  Honors TLQ_PREFILL_NMT / _KSPLIT.
 * A library choice (launch shape), not an operation of the pages.
 */
size_t tl_quant_gemm_workspace_size(int M, int N, int K, int bits, int group);

/*
 * tl_prefill_plan -- the launch plan the library would use for `count`
 * problems: per problem the token tiles per CTA of the tensor-core kernel
 * (1 or 2) and its k split (1, 2, 4 or 8), or 0 and 0 when M <= 16 (the
 * decode kernel).  count = 1 plans a single call (tl_quant_gemm_ws with the
 * given workspace); count = 2..4 with every M > 16 gives the joint plan of a
 * batched call whose launches run side by side; otherwise each problem is
 * planned alone.
 *   M, N, K, ws_bytes  HOST arrays of `count` entries (ws_bytes: the bytes of
 *                      workspace each problem is given, 0 = none).
 *   device             NULL: the current device.  Else a HOST int[9]: the SM
 *                      count, then how many clusters of 1, 2, 4 and 8 CTAs
 *                      fit at once with one token tile per CTA, then the same
 *                      with two.  With a device description no CUDA call is
 *                      made (the planners are host code).
 *   nmt_out, ks_out    HOST arrays of `count` entries, written.
 * TLQ_PREFILL_NMT / TLQ_PREFILL_KSPLIT force the choice as they do for the
 * launches.  A library choice (launch shape), not an operation of the pages.
 * Returns TLQ_OK or TLQ_EINVAL (count outside 1..16, null arrays, a size
 * below 1, a device entry below 1, or a forced split without the workspace
 * it needs).
 */
tlq_status tl_prefill_plan(const int* M, const int* N, const int* K, const size_t* ws_bytes, int count,
                           const int* device, int* nmt_out, int* ks_out);

/*
 * tl_quant_gemm_ws -- tl_quant_gemm with a caller-owned workspace for the
 * tensor-core kernel's k split (same operation, layouts and errors).
 *   workspace        device buffer, 16-byte aligned, or NULL; must not
 *                    overlap A, C or the weights.  Its contents on entry do
 *                    not matter; on return they are undefined.  Calls whose
 *                    executions overlap on the GPU need separate workspaces.
 *   workspace_bytes  its size.  The kernel splits K only with a split whose
 *                    workspace fits (the largest it wants is
 *                    tl_quant_gemm_workspace_size); results of each output do
 *                    not depend on it beyond FP32 summation order.
 */
tlq_status tl_quant_gemm_ws(const uint16_t* A, const uint32_t* Wpacked, const uint16_t* scales,
                            const uint16_t* zeros, uint16_t* C, int M, int N, int K, int bits, int group,
                            void* workspace, size_t workspace_bytes, void* stream);

/* One problem of tl_quant_gemm_batched: the arguments of one
 * tl_quant_gemm_ws call (device pointers, same layouts and rules), plus the
 * packed weight's row stride.
 *   ldw        row stride of Wpacked in 32-bit words; 0 = compact rows of
 *              K*bits/32 words; else >= K*bits/32 and a multiple of 4 (an
 *              INT2 weight converted in place keeps the INT4 stride K/8).
 *   workspace  this problem's own k-split workspace (NULL / 0: none); the
 *              problems of one call may run at the same time, so their
 *              workspaces must not overlap. */
typedef struct {
  const uint16_t* A;
  const uint32_t* Wpacked;
  const uint16_t* scales;
  const uint16_t* zeros;
  uint16_t* C;
  int M, N, K, bits, group;
  int ldw;
  void* workspace;
  size_t workspace_bytes;
} tl_gemm_desc;

/*
 * tl_quant_gemm_batched -- several independent quant_gemm problems in as few
 * launches as possible: every problem with M <= 16 of one bit width goes into
 * one persistent decode launch (up to 16 problems per launch), each larger
 * problem gets its own tensor-core launch.  Those launches run side by side
 * on up to three library-owned streams per caller stream, forked from
 * `stream` and joined back with events (so the call's work still completes in
 * `stream` order, and a graph capture of `stream` records the fork and join).
 * When two to four such launches run at once, their token tiles per CTA and
 * k splits are planned together for the shared GPU (within the workspace
 * each descriptor gives); otherwise each is planned as a single call would
 * plan it.  Results equal `count` separate tl_quant_gemm_ws calls within the
 * layer's tolerance, and M <= 16 problems bit for bit (a tensor-core
 * problem's k split, and so its FP32 summation order, may differ from the
 * one a single call picks); repeated calls give the same bits.  Same source passages as tl_quant_gemm; batching is a
 * launch-overhead measure of this library (the layers of one decode step that
 * do not depend on each other, or several requests at once).
 *   descs  HOST array of `count` descriptors (count >= 0; 0 is a no-op).
 *   No C may overlap any A or another C.  Every descriptor is validated
 *   before anything is launched (TLQ_EINVAL names the offending index).
 */
tlq_status tl_quant_gemm_batched(const tl_gemm_desc* descs, int count, void* stream);

/*
 * tl_quant_gemm_batched_host -- tl_quant_gemm_batched on HOST activations and
 * outputs: one host -> device copy of the step's activations, the batched
 * GEMMs, one device -> host copy of the outputs, in that order on `stream`.
 * Same source passages as tl_quant_gemm.
 *   hostA   a_bytes of activations (pinned host memory for asynchronous
 *           copies; pageable memory works but the copy blocks the caller).
 *   devA    device staging of a_bytes; every descriptor's A lies inside it.
 *   hostC   c_bytes of outputs (pinned host memory); written when the stream
 *           reaches the copy.
 *   devC    device staging of c_bytes; every descriptor's C lies inside it.
 *   Calls on two streams with two staging sets overlap one call's copies with
 *   the other's GEMMs.  Returns the errors of tl_quant_gemm_batched, TLQ_EINVAL
 *   for null or misplaced buffers, TLQ_ECUDA for a failed copy.
 */
tlq_status tl_quant_gemm_batched_host(const tl_gemm_desc* descs, int count, const void* hostA, void* devA,
                                      size_t a_bytes, void* hostC, const void* devC, size_t c_bytes, void* stream);

/*
 * tl_pack_weights -- pack quantization codes into the kernels' weight format.
 *
 * Source: "beta-Informed Deployment Features", CTX-TIER, "Details of the
 * shipped kernel": an INT4 row takes K/2 bytes, an INT2 row K/4 bytes, four
 * INT2 codes per byte.  The bit order is this library's reading (LSB first).
 *
 *   codes   uint8 [N][K] device array, one code per byte; only the low `bits`
 *           bits of each byte are stored.
 *   Wpacked uint32 [N][K*bits/32] output.
 *   K % (32/bits) == 0.  Bit-exact; deterministic.
 */
tlq_status tl_pack_weights(const uint8_t* codes, uint32_t* Wpacked, int N, int K, int bits,
                           void* stream);

/* Inverse of tl_pack_weights: codes[n][k] = code k of row n (0 .. 2^bits-1). */
tlq_status tl_unpack_weights(const uint32_t* Wpacked, uint8_t* codes, int N, int K, int bits,
                             void* stream);

/*
 * tl_requant_int4_to_int2 -- re-quantize an INT4 weight to INT2, the weight
 * conversion of the context-length tier switch after which quant_gemm routes
 * the layer to the INT2 kernel.
 *
 * Source: "beta-Informed Deployment Features", CTX-TIER, "Details of the
 * shipped kernel" (Phase 2 / 2b): per quantization group the INT4 weights are
 * dequantized, an asymmetric INT2 grid with scale = (max - min) / 3 and
 * zero = min is fitted, and each weight is rounded to the nearest of its four
 * levels; the group size is kept; the INT2 rows are compact so the INT4
 * buffer can be released afterwards.
 *
 * In this library's (q - z) * s form, per group of row n (binary32, rounded
 * to nearest even after every step, in this order):
 *   w  = (q4 - z4) * s4;  lo, hi = min, max of w over the group
 *   s2 = fp16((hi - lo) / 3), or 1.0 when that is zero;  z2 = fp16(-lo / s2)
 *   q2 = clamp(rint(w / s2 + z2), 0, 3)
 * so (q2 - z2) * s2 is the INT2 GEMM's weight.  Codes, s2 and z2 are
 * bit-exact and deterministic.
 *
 *   W4      uint32 [N][K/8] INT4 weight in the tl_pack_weights format;
 *           16-byte aligned; read only.
 *   s4, z4  FP16 [N][K/group] scales / zeros of W4; finite values.
 *   W2      uint32 [N][K/16] output, compact INT2 rows; 16-byte aligned; must
 *           not overlap any other argument -- or exactly W4: converted in
 *           place ("Details of the shipped kernel", storage reuse), the INT2
 *           rows keeping the INT4 row stride of K/8 words with the second
 *           half of every row left untouched; GEMMs then read it with
 *           ldw = K/8 (tl_qproj, tl_gemm_desc).
 *   s2, z2  FP16 [N][K/group] output scales / zeros.  Each may be exactly its
 *           input (s2 == s4, z2 == z4: converted in place) or overlap nothing.
 *   N >= 1; K >= 1; group a multiple of 64 dividing K (the INT2 kernel's
 *   rule); the INT2 weight keeps the INT4 weight's group.
 *   The caller owns every buffer; W4 may be freed once the stream has passed
 *   an out-of-place call.  Returns TLQ_OK, TLQ_EINVAL (null, misaligned, overlapping or
 *   bad shape) or TLQ_ECUDA.
 */
tlq_status tl_requant_int4_to_int2(const uint32_t* W4, const uint16_t* s4, const uint16_t* z4, uint32_t* W2,
                                   uint16_t* s2, uint16_t* z2, int N, int K, int group, void* stream);

/* One weight of tl_requant_int4_to_int2_batched (device pointers, the same
 * layouts and rules as tl_requant_int4_to_int2). */
typedef struct {
  const uint32_t* W4;
  const uint16_t* s4;
  const uint16_t* z4;
  uint32_t* W2;
  uint16_t* s2;
  uint16_t* z2;
  int N, K;
} tl_requant_desc;

/*
 * tl_requant_int4_to_int2_batched -- up to 16 weights of one group size
 * re-quantized in a single launch (the tier switch converts all projections
 * of the loop block at once).  Results equal `count` separate
 * tl_requant_int4_to_int2 calls.
 *   descs  HOST array of `count` descriptors (0 <= count <= 16; 0 is a no-op).
 *   No output (W2, s2, z2) may overlap any other buffer of any descriptor,
 *   except s2 == s4 / z2 == z4 of the same descriptor.  Everything is
 *   validated before the launch (TLQ_EINVAL names the offending index).
 */
tlq_status tl_requant_int4_to_int2_batched(const tl_requant_desc* descs, int count, int group, void* stream);

/*
 * tl_quant_gemm_swiglu -- the SwiGLU feed-forward's gate and up projections as
 * one GEMM with the gate*up product in its epilogue.
 *
 *   C[m][i] = fp16( silu(g) * u ),  g = fp16(acc[m][2i]),  u = fp16(acc[m][2i+1]),
 *   silu(g) = g / (1 + exp(-g)),  acc = A . dequant(Wgu)^T in FP32.
 *
 * Source: "Model", ffn_dim -- "For SwiGLU this is the width of the gate and up
 * projections"; the loop block's mlp_gate / mlp_up weights ("beta-Informed
 * Deployment Features", CTX-TIER, Phase 2b).  g and u are rounded to FP16 like
 * any GEMM output of the block; the product is formed in FP32 (the pages fix
 * neither).
 *   Wgu     packed weights [N2][K] whose rows alternate gate and up: row 2i is
 *           gate row i, row 2i+1 up row i (tl_interleave_rows builds it from
 *           the two packed weights; scales and zeros are interleaved the same
 *           way).  N2 = 2F, a multiple of 16.
 *   C       FP16 [M][N2/2], row stride N2/2; must not overlap A.
 *   Other arguments and errors as tl_quant_gemm.
 */
tlq_status tl_quant_gemm_swiglu(const uint16_t* A, const uint32_t* Wgu, const uint16_t* scales,
                                const uint16_t* zeros, uint16_t* C, int M, int N2, int K, int bits, int group,
                                void* stream);

/* tl_quant_gemm_swiglu with a caller-owned k-split workspace (the rules of
 * tl_quant_gemm_ws; its size from tl_quant_gemm_workspace_size(M, N2, K, ...)). */
tlq_status tl_quant_gemm_swiglu_ws(const uint16_t* A, const uint32_t* Wgu, const uint16_t* scales,
                                   const uint16_t* zeros, uint16_t* C, int M, int N2, int K, int bits, int group,
                                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * tl_dequant_fp16 -- the FP16 body of a quantized weight: out[n][k] =
 * fp16_RNE((q - z) * s), each weight rounded once from its exact value, +0
 * for an exact zero.  Bit-exact and deterministic.
 *
 * Source: "Model", section "VRAM cost": the opt-in FP16 body cache (a dense
 * FP16 copy of the loop-block weights, about 3x their quantized memory).
 * This library offers it as a comparison point for the quantized GEMM: a
 * plain FP16 GEMM on the body.
 *   Wpacked, scales, zeros  as tl_quant_gemm (16-byte aligned Wpacked).
 *   out     FP16 [N][K], row-major, 16-byte aligned, caller-owned; must not
 *           overlap the inputs.
 *   bits, group, N, K: the rules of tl_quant_gemm (N need not be a multiple
 *   of 8).  Returns TLQ_OK, TLQ_EINVAL or TLQ_ECUDA.
 */
tlq_status tl_dequant_fp16(const uint32_t* Wpacked, const uint16_t* scales, const uint16_t* zeros, uint16_t* out,
                           int N, int K, int bits, int group, void* stream);

/*
 * tl_interleave_rows -- out row 2i = row i of a, out row 2i+1 = row i of b
 * (device buffers of `rows` rows of `row_bytes` bytes; out holds 2*rows).
 * Lays out the gate and up weights (packed words, scales, zeros) for
 * tl_quant_gemm_swiglu.  out must not overlap a or b.  Asynchronous on
 * `stream`.  Returns TLQ_OK, TLQ_EINVAL or TLQ_ECUDA.
 */
tlq_status tl_interleave_rows(const void* a, const void* b, void* out, int rows, size_t row_bytes, void* stream);

/* One quantized projection of the loop block: weights [N][K] in the packed
 * format, FP16 scales/zeros [N][K/group]; ldw is the weight's row stride in
 * 32-bit words (0 = compact rows of K*bits/32 words; else >= that and a
 * multiple of 4, e.g. K/8 for an INT2 weight converted in place). */
typedef struct {
  const uint32_t* W;
  const uint16_t* s;
  const uint16_t* z;
  int N;
  int K;
  int ldw;
} tl_qproj;

/*
 * The shared-weight loop block (one weight set reused every iteration).
 *   qkv  : N = 3*D, K = D        o    : N = D, K = D
 *   up   : N = F,   K = D        down : N = D, K = F
 * Scratch buffers are caller-owned device FP16 arrays with at least M rows:
 *   h [M][D], qkv_out [M][3D], o_out [M][D], up_out [M][F].
 * normalize = 1 applies the per-row RMS pre-norm h = fp16(x / sqrt(mean x^2 +
 * 1e-5)) before the QKV projection (the block's LayerNorm position, "Model",
 * "VRAM cost", with buf.norm as its FP16 output); 0 feeds fp16(x) directly.
 * workspace / workspace_bytes: the caller's k-split workspace for the block's
 * GEMMs with M > 16 (they run one after another and share it; NULL / 0 = no
 * k split); the largest tl_quant_gemm_workspace_size of the four GEMMs at M
 * rows is what they can use.  Must not overlap any other buffer.
 */
typedef struct {
  tl_qproj qkv, o, up, down;
  int bits;
  int group;
  int D;
  uint16_t* h;
  uint16_t* qkv_out;
  uint16_t* o_out;
  uint16_t* up_out;
  int normalize;
  void* workspace;
  size_t workspace_bytes;
} tl_block;

/*
 * The five-weight SwiGLU loop block (attn_qkv, attn_out, mlp_gate, mlp_up,
 * mlp_down -- "beta-Informed Deployment Features", CTX-TIER, Phase 2b;
 * "Model", ffn_dim):
 *   h = norm(x); qkv = Q(h); o = Q(qkv[:, :D]);
 *   a = fp16(silu(Q_gate(o)) * Q_up(o)); x += float(Q_down(a))
 * with every GEMM output rounded to FP16 and the residual add in FP32.
 *   qkv     : N = 3*D, K = D          o    : N = D, K = D
 *   gate_up : N = 2*F, K = D, rows interleaved (see tl_quant_gemm_swiglu)
 *   down    : N = D, K = F
 * Scratch (caller-owned device FP16, at least M rows): h [M][D],
 * qkv_out [M][3D], o_out [M][D], act_out [M][F].  normalize and workspace as
 * tl_block.
 */
typedef struct {
  tl_qproj qkv, o, gate_up, down;
  int bits;
  int group;
  int D;
  uint16_t* h;
  uint16_t* qkv_out;
  uint16_t* o_out;
  uint16_t* act_out;
  int normalize;
  void* workspace;
  size_t workspace_bytes;
} tl_swiglu_block;

/*
 * tl_loop_block_forward -- apply the shared block L times to the FP32
 * residual stream x[M][D] in place:
 *
 *   for l in 0..L-1:
 *     h   = fp16(rmsnorm(x))            (or fp16(x) when normalize = 0)
 *     qkv = quant_gemm(h, qkv)          [M][3D]
 *     o   = quant_gemm(qkv[:, :D], o)   [M][D]   (row stride 3D)
 *     u   = relu(quant_gemm(o, up))     [M][F]   relu(v) = v > 0 ? v : +0
 *     x  += float(quant_gemm(u, down))  FP32 add of the FP16 result
 *
 * Source: "Model", "VRAM cost", Runtime buffers (buf.main is the FP32
 * residual, the scratch buffers are FP16); "Warm-start mid-loop", internal
 * flow, "Extend loop" (the block is re-run in place on the residual, so
 * running L1 then L - L1 iterations equals running L, bit for bit).
 *   x      FP32 [M][D] device array, updated in place.
 *   block  HOST pointer to a tl_block describing device buffers.
 *   L >= 0 (L = 0 is a no-op); M >= 1.
 * L2 residency (see tl_loop_block_l2_plan): the projections the plan keeps
 * resident are streamed with an evict-last policy, the others evict-first.
 * With TLQ_LOG=1 in the environment the first call prints the plan.
 */
tlq_status tl_loop_block_forward(float* x, const tl_block* block, int L, int M, void* stream);

/*
 * tl_loop_block_l2_plan -- the loop block's L2 residency plan ("Model",
 * "Returns", item 4: auto tile sizing reports loop-block vs L2 cache
 * residency).  The block's weights (packed words plus FP16 scales and zeros)
 * are re-read every iteration; the plan keeps projections resident, in
 * iteration order (qkv, o, up, down), while their running total fits a
 * budget of half the device's L2, and only when L > 1.
 *   block          HOST pointer; only the projections' N and K, bits and
 *                  group are read (no device memory is touched).
 *   resident_mask  out: bit i set when projection i is kept resident.
 *   weight_bytes, budget_bytes  out (may be NULL): the block's weight bytes
 *                  and the budget.
 * The SwiGLU block uses the same plan over (qkv, o, gate_up, down).
 * Returns TLQ_OK or TLQ_EINVAL.
 */
tlq_status tl_loop_block_l2_plan(const tl_block* block, int L, int* resident_mask, size_t* weight_bytes,
                                 size_t* budget_bytes);

/*
 * tl_swiglu_block_forward -- the five-weight SwiGLU loop block applied L times
 * to the FP32 residual x [M][D] in place (same rules, errors and L2 policy as
 * tl_loop_block_forward; the gate/up GEMM runs with the SwiGLU epilogue, so a
 * block iteration is five launches like the ReLU block).
 */
tlq_status tl_swiglu_block_forward(float* x, const tl_swiglu_block* block, int L, int M, void* stream);

/*
 * tl_loop_block_forward_chunked / tl_swiglu_block_forward_chunked -- chunked
 * prefill: the M rows of x are split into chunks of `chunk` rows and each
 * chunk runs through all L iterations before the next one starts, so the
 * scratch buffers need only min(chunk, M) rows.
 *
 * Source: "Model", section "Chunked prefill": prompts longer than
 * prefill_chunk are split into chunks that each run through all blocks and
 * loop iterations in turn; the buffer VRAM shrinks with the chunk while the
 * launch count grows with the number of chunks.  The block's rows are
 * independent (no attention on this path), so every chunk is the block on a
 * row slice; results match single-shot within the GEMM tolerance (the kernel
 * choice and summation order depend on the row count: M <= 16 takes the
 * decode kernel).
 *   chunk <= 0 or chunk >= M: single shot.  Other arguments and errors as the
 *   unchunked calls; scratch rows must cover min(chunk, M).
 */
tlq_status tl_loop_block_forward_chunked(float* x, const tl_block* block, int L, int M, int chunk, void* stream);
tlq_status tl_swiglu_block_forward_chunked(float* x, const tl_swiglu_block* block, int L, int M, int chunk,
                                           void* stream);

/*
 * tl_loop_block_to_int2 / tl_swiglu_block_to_int2 -- the context-length tier
 * switch of a loop block: its four weights (the SwiGLU block's fused gate/up
 * weight re-quantizes row by row like the two it holds) are re-quantized
 * INT4 -> INT2 as tl_requant_int4_to_int2 does, and the HOST block
 * description is rewritten (bits = 2, each projection's W / s / z / ldw) so
 * later forwards run the INT2 kernels.
 *
 * Source: "beta-Informed Deployment Features", CTX-TIER, "What Phase 2
 * ships", item 2 (apply_tier_to_model: the loop block's weights re-quantized,
 * the bit width flipped so the dispatcher routes to int2_gemm) and Phase 2b
 * (compact INT2 buffers, the INT4 ones released).
 *   block  HOST pointer; an INT4 block (bits = 4, compact INT4 rows, a group
 *          that is a multiple of 64).
 *   dst    HOST array of four destinations (qkv, o, up or gate_up, down), each
 *          with the weight's N and K: W compact INT2 rows (K/16 words) or the
 *          INT4 weight itself (in place, ldw = K/8 afterwards); s / z new
 *          arrays or the INT4 ones (converted in place).  NULL: everything in
 *          place (no new memory at all).
 *   Every check happens before the launch; on an error the block is left as
 *   it was.  Out of place, the INT4 buffers may be freed once `stream` has
 *   passed the call.  Returns TLQ_OK, TLQ_EINVAL or TLQ_ECUDA.
 */
tlq_status tl_loop_block_to_int2(tl_block* block, const tl_qproj* dst, void* stream);
tlq_status tl_swiglu_block_to_int2(tl_swiglu_block* block, const tl_qproj* dst, void* stream);

/*
 * tl_loop_block_forward_static_scratch -- tl_loop_block_forward for callers
 * that cannot allocate device memory or provide scratch buffers (a serving
 * runtime that forbids allocation after start-up, a plugin interface that only
 * passes a layer its inputs and outputs).  There is no counterpart on the
 * pages: it is a packaging choice of this library.
 *
 * Identical arithmetic to tl_loop_block_forward; block->h, qkv_out, o_out,
 * up_out and workspace are ignored (may be NULL): the GEMMs run without a k
 * split.  The four FP16 intermediates live in one
 * 4 MiB static device array inside the library, which every GPU that loads
 * the library holds until the process exits.  The call allocates nothing
 * (no cudaMalloc, cudaFree or allocating library routine).
 *   Size limit: 2*M*(5*D + F) bytes (each buffer rounded up to 256 bytes)
 *   must fit in 4 MiB -- e.g. M <= 113 at D = 2048, F = 8192 -- otherwise
 *   TLQ_EINVAL with a message that names the sizes, and nothing is launched.
 *   First call on a device: looks up the array's device address (once per
 *   device, with that device current) and keeps it for the life of the
 *   process; make that first call before any stream capture.  A device reset
 *   (cudaDeviceReset) invalidates the kept address: after one, this entry
 *   point must not be called again in the same process.
 *   All calls on a device share the one array, which keeps whatever the last
 *   call left in it; every intermediate is fully written before it is read,
 *   so nothing needs clearing.  Calls whose executions overlap on the GPU
 *   (other streams, other threads) race on the array: serialize them.
 */
tlq_status tl_loop_block_forward_static_scratch(float* x, const tl_block* block, int L, int M, void* stream);

/*
 * tl_probe_read_bandwidth -- a measurement helper, no operation of the pages:
 * `reps` passes of 16-byte L2-only loads (ld.global.cg) over buf, folded into
 * one word per thread of sink (2 x SMs x 512 words, caller-owned).  With buf
 * small enough to stay in L2 it measures the L2 read bandwidth that bounds
 * the loop block (its packed weights fit in L2 and are re-read every
 * iteration); the benchmark times it with CUDA events.
 *   buf    device buffer, 16-byte aligned; bytes a positive multiple of 16.
 * Returns TLQ_OK, TLQ_EINVAL or TLQ_ECUDA.
 */
tlq_status tl_probe_read_bandwidth(const void* buf, size_t bytes, int reps, uint32_t* sink, void* stream);

/*
 * ---------------------------------------------------------------------------
 * Multi-request serving beside the quantized projections: a paged cache of
 * keys and values in 4 bits with the attention that reads it, the tables of a
 * step's requests, and low-rank adapters per request.
 *
 * Source: "Model", section "VRAM cost" (INT4 cache mode) and "Chunked
 * prefill" (queries of a chunk over everything cached before it);
 * "Prefix pool" (requests of different lengths over shared cached pages).
 * The pages fix neither layout nor formulas; the ones below are this
 * library's.  Activations are FP16 like those of every GEMM here.
 *
 * Cache blocks.  `blocks` is [num_pages][heads][tl_kv4_block_bytes] bytes; the
 * block of one page and key head holds, one after another,
 *   key codes    [page_size][head_dim/2] bytes
 *   value codes  [page_size][head_dim/2] bytes
 *   key parameters   [page_size][head_dim/group] pairs of FP16 (scale, minimum)
 *   value parameters [page_size][head_dim/group] pairs of FP16 (scale, minimum)
 * Code rows pack channels as tl_pack_weights packs a weight row (least
 * significant first); a channel stands for code * scale + minimum, scales are
 * at least 2^-24, and neither is infinite.  A token's slot is page * page_size
 * + offset.
 * ---------------------------------------------------------------------------
 */
typedef struct {
  void* blocks;      /* device, 16-byte aligned */
  int64_t num_pages; /* 1 .. 2^31 - 1, and so num_pages * heads */
  int heads;         /* key (and value) heads, 1 .. 4096 */
  int head_dim;      /* 64 or 128 */
  int page_size;     /* tokens of a page: 16, 32, 64, 128 or 256 */
  int group;         /* channels that share a scale and a minimum: 64 or 128, dividing head_dim */
} tl_kv4_cache;

/* Bytes of one page and head of the cache; 0 for a geometry the library does
 * not take (tl_last_error says why). */
size_t tl_kv4_block_bytes(int page_size, int head_dim, int group);

/*
 * tl_kv_plan -- block tables, slots and positions of one step's tokens, from
 * the requests' lengths, on the GPU (no host copy of a length is needed).
 *
 *   Request b has cached[b] tokens in the cache and brings added[b] (either
 *   may be 0; negative counts as 0).  The step's tokens are laid out request
 *   after request.  Pages that a request does not hold yet are taken from
 *   free_pages in request order, beginning at *free_head:
 *     held = ceil(cached/page_size), need = ceil((cached+added)/page_size) - held
 *     table[b][held + i] = free_pages[*free_head + (need of earlier requests) + i]
 *
 *   cached, added  int32 [requests]
 *   table          int32 [requests][ld_table], read for pages held, written
 *                  for new ones (other entries are left as they are)
 *   free_pages     int32 [num_free] page ids; free_head: device int32 or NULL
 *                  (0; negative counts as 0)
 *   num_pages      pages of the cache; a page id outside it gives slot -1
 *   q_start        out int32 [requests + 1], exclusive sums of added
 *   seq_lens       out int32 [requests], cached + added
 *   token_req, token_pos, slots   out [capacity] (int32, int32, int64): each
 *                  token's request, its position in the request and its slot;
 *                  -1 behind the last token
 *   counts         out int32 [4]: tokens, pages taken, the free list's next
 *                  head, and pages that were needed but not to be had (the
 *                  list ended, or the table row did): their entries and slots
 *                  are -1
 *   Tokens beyond capacity are left out of the token arrays.  Outputs overlap
 *   neither an input nor each other (free_head may not point into counts: two
 *   counts buffers in turn carry the head from step to step).  page_size: a
 *   power of two.  Deterministic; the same inputs give the same tables, so a
 *   call can be repeated.  Returns TLQ_OK, TLQ_EINVAL or TLQ_ECUDA.
 */
tlq_status tl_kv_plan(const int32_t* cached, const int32_t* added, int requests, int32_t* table, int ld_table,
                      const int32_t* free_pages, int num_free, const int32_t* free_head, int page_size,
                      int64_t num_pages, int32_t* q_start, int32_t* seq_lens, int32_t* token_req, int32_t* token_pos,
                      int64_t* slots, int capacity, int32_t* counts, void* stream);

/*
 * tl_kv4_append -- keys and values of `tokens` tokens quantized into the cache.
 *
 *   Per token, head and group of channels (binary32, rounded to nearest even
 *   after every step):
 *     minimum = fp16(min x), scale = max(fp16((max x - min x) / 15), 2^-24)
 *     code = clamp(rint((x - minimum) / scale), 0, 15)
 *   k, v   FP16 [tokens][heads][head_dim] with token strides ldk, ldv (in
 *          elements, multiples of 8; the columns of a fused qkv projection's
 *          rows are taken as they lie); 16-byte aligned; a group with a value
 *          that is not finite has NaN for scale and minimum and stands for
 *          NaN throughout
 *   slots  int64 [tokens]; slots outside the cache (-1) are passed over; a
 *          call's slots are distinct
 *   Bit-exact; deterministic.  Returns TLQ_OK, TLQ_EINVAL, TLQ_EUNSUPPORTED
 *   (a head_dim or group that is not taken) or TLQ_ECUDA.
 */
tlq_status tl_kv4_append(const tl_kv4_cache* cache, const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                         const int64_t* slots, int tokens, void* stream);

/*
 * tl_kv4_read -- the values that cached tokens stand for: k, v FP16
 * [tokens][heads][head_dim] compact, fp16(code * scale + minimum) rounded once
 * more from binary32; zeros for slots outside the cache.  Errors as
 * tl_kv4_append.
 */
tlq_status tl_kv4_read(const tl_kv4_cache* cache, const int64_t* slots, int tokens, uint16_t* k, uint16_t* v,
                       void* stream);

/*
 * tl_kv4_attention -- causal attention of a step's queries over the cache.
 *
 *   Request b's queries are rows q_start[b] .. q_start[b+1] - 1; the last of
 *   them sits at position seq_lens[b] - 1, and a query at position p sees the
 *   request's tokens 0 .. p (window > 0: the last `window` of them).  Query
 *   head i reads key head i / (q_heads / heads).
 *     out = softmax(scale * q . k) v
 *   Sums and softmax statistics are FP32; weights are rounded to FP16 for the
 *   second product.  A NaN in the cache shows in the queries that see its token
 *   and in no others.  A query that sees no key (seq_lens[b] smaller than the
 *   request's queries, or none of its pages in the cache) gives zeros.
 *
 *   q, out    FP16 [tokens][q_heads][head_dim], token strides ldq, ldo
 *             (elements, multiples of 8), 16-byte aligned; out overlaps no
 *             other buffer
 *   q_start   int32 [requests + 1], seq_lens int32 [requests], table int32
 *             [requests][ld_table]: page ids of each request's tokens (device;
 *             what tl_kv_plan writes).  seq_lens counts the step's own tokens,
 *             which tl_kv4_append has put into the cache.  Entries that no
 *             visible token lies in are not read as pages; a page id outside
 *             the cache counts as holding no tokens, and so do those behind
 *             the table's row (positions are still those of seq_lens).
 *             A request's context is at most 2^30 tokens
 *   tokens    rows of q; queries outside [0, tokens) count as none, rows of
 *             no request are not written
 *   max_q     the most queries that a request has (an upper bound will do; of
 *             a request with more, the last ones are left out and their rows
 *             are not written)
 *   workspace device, 16-byte aligned, of tl_kv4_attention_workspace_size
 *             bytes or more; undefined afterwards, no contents needed before.
 *             Calls whose executions overlap need separate workspaces
 *   Lengths are read on the GPU only, so a captured call can be replayed as
 *   requests grow.  Deterministic.  Returns TLQ_OK, TLQ_EINVAL,
 *   TLQ_EUNSUPPORTED or TLQ_ECUDA.
 */
tlq_status tl_kv4_attention(const tl_kv4_cache* cache, const uint16_t* q, int64_t ldq, int q_heads, uint16_t* out,
                            int64_t ldo, const int32_t* q_start, const int32_t* seq_lens, const int32_t* table,
                            int ld_table, int requests, int tokens, int max_q, float scale, int window,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace that tl_kv4_attention takes (the same for every batch of
 * up to max_q queries a request); 0 for arguments it would not take. */
size_t tl_kv4_attention_workspace_size(int q_heads, int heads, int head_dim, int max_q);

/*
 * tl_kv4_attention_prefix -- attention of requests that share a prefix, whose
 * pages are read once for all of them.
 *
 *   A query sees the whole prefix, and of its request's own tokens those that
 *   tl_kv4_attention would show it: the request's own tokens are positions
 *   0 .. seq_lens[b] - 1 of its table row, the prefix lies before them.
 *     out = softmax(scale * q . k) v  over both together
 *   prefix_len    device int32: tokens of the prefix (may end inside a page:
 *                 own tokens begin with a page of their own; below 1: none)
 *   prefix_table  int32 [prefix_pages] page ids of the prefix; a page id
 *                 outside the cache counts as holding no tokens, and so do
 *                 those behind the table
 *   The other arguments, what is not written, and what a NaN does are as in
 *   tl_kv4_attention (without a window).  A batch whose queries are few for the
 *   prefix's table (a choice by both sizes; any where rows hold two groups)
 *   reads the prefix once for each 8 or 16 rows of a key head, from L2; prompts
 *   and long prefixes once for each 256.  The choice goes by prefix_pages and,
 *   in batches with prompts, by ld_table: tables much longer than what they hold
 *   can cost time.
 *   workspace     of tl_kv4_attention_prefix_workspace_size bytes or more
 *   Lengths are read on the GPU only, the prefix's too.  Deterministic.
 *   Returns as tl_kv4_attention.
 */
tlq_status tl_kv4_attention_prefix(const tl_kv4_cache* cache, const uint16_t* q, int64_t ldq, int q_heads,
                                   uint16_t* out, int64_t ldo, const int32_t* q_start, const int32_t* seq_lens,
                                   const int32_t* table, int ld_table, const int32_t* prefix_len,
                                   const int32_t* prefix_table, int prefix_pages, int requests, int tokens, int max_q,
                                   float scale, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace that tl_kv4_attention_prefix takes for up to that many
 * tokens; 0 for arguments it would not take. */
size_t tl_kv4_attention_prefix_workspace_size(int q_heads, int heads, int head_dim, int tokens, int max_q);

/*
 * Rotary positions.  Pair i (0 .. rot_dim/2 - 1) of a head's first rot_dim
 * channels, (a, b), turns by the angle of its position:
 *   (a, b) -> (a cos - b sin, b cos + a sin),  (cos, sin) = table[position][i]
 * Other channels are left.  With several axes (time, height and width of
 * images and video) the first sections[0] pairs go by a token's position on
 * the first axis, the next sections[1] by that on the second, and so on.
 */
typedef struct {
  const float* table;    /* device, FP32 [num_positions][rot_dim/2][2], 16-byte aligned: cos and sin */
  int64_t num_positions; /* 1 .. 2^30 */
  int rot_dim;           /* a multiple of 16, up to the head size */
  int interleaved;       /* pairs: 0 channels (i, i + rot_dim/2), else (2i, 2i + 1) */
  int axes;              /* 1 .. 3 */
  int sections[3];       /* pairs of each axis; they add up to rot_dim/2 */
} tl_rope;

/*
 * tl_rope_table -- table[p][i] = (cos, sin)(p * inv_freq[i]) * scale, in 64 bits
 * and rounded once to FP32 (angles of far positions keep their digits).
 *   inv_freq  device FP64 [rot_dim/2];  table  device, 4 * num_positions *
 *             rot_dim bytes, 16-byte aligned;  scale  1 for plain rotations
 * Returns TLQ_OK, TLQ_EINVAL or TLQ_ECUDA.
 */
tlq_status tl_rope_table(const double* inv_freq, int64_t num_positions, int rot_dim, double scale, float* table,
                         void* stream);

/*
 * tl_qk_norm_rope -- the query and key heads of `tokens` tokens normed and
 * rotated, one pass.
 *
 *   Per head x of head_dim channels (FP32, rounded after every operation):
 *     y = (x * r) * weight,  r = 1 / sqrt(sum(x^2) / head_dim + eps)
 *   (weight NULL: y = x), then the rotation, its products rounded and then
 *   their sum, and one rounding to FP16.  The squares are added up as a tree:
 *   each 8 channels by halves (j and j + 4, then j and j + 2, then the two),
 *   then these sums by halves.  So results are defined to the bit.
 *
 *   q, q_out   FP16 [tokens][q_heads][head_dim], token strides ldq, ldqo (in
 *              elements, multiples of 8); k, k_out likewise.  Either heads may
 *              be 0 (its pointers are not looked at).  An output may be exactly
 *              its input, else it shares no byte with an input or the other
 *              output (columns of the same fused rows do not)
 *   weights    FP16 [head_dim] or NULL; all pointers 16-byte aligned
 *   head_dim   64, 128 or 256;  eps  finite, not negative
 *   rope       NULL: no rotation;  positions  int32 [axes][tokens]
 *   A token with a negative position on an axis (tl_kv_plan's entries behind
 *   the last token) is passed over: its rows are not written.  A position at
 *   or past num_positions gives NaN in the rotated channels.
 *   Bit-exact; deterministic.  Returns TLQ_OK, TLQ_EINVAL, TLQ_EUNSUPPORTED (a
 *   head_dim that is not taken, 2^31 rows or more) or TLQ_ECUDA.
 */
tlq_status tl_qk_norm_rope(const tl_rope* rope, const int32_t* positions, const uint16_t* q, int64_t ldq, int q_heads,
                           const uint16_t* q_weight, uint16_t* q_out, int64_t ldqo, const uint16_t* k, int64_t ldk,
                           int k_heads, const uint16_t* k_weight, uint16_t* k_out, int64_t ldko, int head_dim,
                           float eps, int tokens, void* stream);

/*
 * tl_kv4_append_rope -- what tl_qk_norm_rope does with keys, on their way into
 * the cache: the bits are those of tl_qk_norm_rope followed by tl_kv4_append,
 * in one launch and without the keys' way through memory.  The queries of the
 * same tokens are normed and rotated beside them (q_heads 0: none).
 *   k, v, slots  as in tl_kv4_append;  the rest as in tl_qk_norm_rope.  A token
 *   with a negative position is passed over altogether, one whose slot is
 *   outside the cache brings its queries only; a position at or past
 *   num_positions gives a key that stands for NaN.  Behind a shared prefix,
 *   tl_kv_plan's positions count from the prefix on: a rope whose table begins
 *   at the row behind the prefix's last takes them as they are, its -1 too.
 *   Bit-exact; deterministic.  Returns as tl_kv4_append.
 */
tlq_status tl_kv4_append_rope(const tl_kv4_cache* cache, const tl_rope* rope, const int32_t* positions,
                              const uint16_t* k, int64_t ldk, const uint16_t* k_weight, const uint16_t* v, int64_t ldv,
                              const int64_t* slots, const uint16_t* q, int64_t ldq, int q_heads,
                              const uint16_t* q_weight, uint16_t* q_out, int64_t ldqo, float eps, int tokens,
                              void* stream);

/*
 * tl_sample -- one token a row of logits, from a given uniform number.
 *
 *   With w_i = exp((x_i - max x) / T) and the row's values in the order of x
 *   falling, equal ones by index rising, a token is kept if it is
 *     among the first top_k, and
 *     in the shortest run from the first on whose weights reach top_p times
 *     those of the first top_k, and
 *     of weight min_p or more;
 *   the first is always kept.  The row's token is the first kept one, by index,
 *   at which the running sum of the kept weights passes uniform times their
 *   sum; its log-probability is ln(w / that sum).  Weights below 2^-40 count as
 *   none.  They are held as whole numbers, 2^43 for the largest: each to about
 *   2^-39 of its own value and one unit, 2^-43 of the largest (min_p is compared
 *   with these), so sums are exact whatever their order.  A difference x - max x
 *   past FP32's range counts as -infinity.
 *
 *   logits       FP16 (fp16 = 1) or FP32 (0) [rows][vocab], row stride ld
 *                (elements); -infinity: a token that is not to be drawn.  A row
 *                with a NaN or +infinity, or with nothing else than -infinity,
 *                gives token -1 and log-probability NaN
 *   vocab        1 .. 2^20
 *   uniform      FP32 [rows], taken into [0, 1 - 2^-24]
 *   temperature  FP32 [rows] or NULL (1); not above 0 (or NaN): the row's
 *                greatest logit, the first of equal ones, log-probability 0
 *   top_k        int32 [rows] or NULL; below 1: all
 *   top_p, min_p FP32 [rows] or NULL; top_p of 1 or more and min_p of 0 or less
 *                (or NaN) leave every token, min_p above 1 counts as 1
 *   tokens       out int32 [rows];  logprobs  out FP32 [rows] or NULL
 *   Outputs overlap no input and not each other.  Deterministic.  Returns
 *   TLQ_OK, TLQ_EINVAL, TLQ_EUNSUPPORTED (a longer row) or TLQ_ECUDA.
 */
tlq_status tl_sample(const void* logits, int fp16, int64_t ld, int rows, int vocab, const float* uniform,
                     const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                     int32_t* tokens, float* logprobs, void* stream);

/*
 * tl_lora_add -- low-rank adapters of many requests beside a shared projection:
 *
 *   out[t] = fp16( y[t] + scales[a] * B[a] (A[a] x[t]) ),  a = adapters[b] of
 *   the token's request b; both products in FP32, one rounding.
 *
 *   x        FP16 [tokens][K], stride ldx; the projection's input
 *   y, out   FP16 [tokens][N], strides ldy, ldo; the projection's output; out
 *            may be exactly y, else overlaps no input
 *   A        FP16 [num_adapters][rank][K];  B  FP16 [num_adapters][N][rank]
 *   scales   FP32 [num_adapters]
 *   q_start  int32 [requests + 1] as in tl_kv4_attention; adapters int32
 *            [requests], outside 0 .. num_adapters - 1: none (out = y)
 *   K, N     multiples of 8; rank a multiple of 8 up to 64
 *   x, A, B, y and out 16-byte aligned, strides multiples of 8 elements.
 *   max_q as in tl_kv4_attention; rows of no request are not written.
 *   Deterministic.  Returns TLQ_OK, TLQ_EINVAL, TLQ_EUNSUPPORTED (rank above
 *   64) or TLQ_ECUDA.
 */
tlq_status tl_lora_add(const uint16_t* x, int64_t ldx, const uint16_t* A, const uint16_t* B, const float* scales,
                       const int32_t* q_start, const int32_t* adapters, int requests, int tokens, int max_q, int K,
                       int N, int rank, int num_adapters, const uint16_t* y, int64_t ldy, uint16_t* out, int64_t ldo,
                       void* stream);

/*
 * Synchronize `stream` and report the device status word: TLQ_OK, or
 * TLQ_ETIMEOUT if a kernel gave up on a bounded wait since the last
 * tl_reset_status().  Also returns TLQ_ECUDA on an asynchronous CUDA error.
 */
tlq_status tl_check_status(void* stream);

/* Clear the device status word of the current device; synchronizes `stream`. */
tlq_status tl_reset_status(void* stream);

/*
 * Self-test of the bounded device waits (no counterpart on the pages; it
 * backs the library's own failure-detection contract).  Launches a one-thread
 * kernel that waits on a shared-memory barrier nothing ever arrives at; the
 * wait gives up after limit_us microseconds (1 .. 1,000,000), records
 * TLQ_ETIMEOUT in the status word and the kernel returns normally, leaving the
 * context usable.  Read the result with tl_check_status().
 */
tlq_status tl_selftest_wait_timeout(unsigned limit_us, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TLQ_H_ */
