/*
 * qmoe.h -- C ABI of the INT4 block-quantized mixture-of-experts FFN layer
 * library for NVIDIA GB300 (sm_103a).
 *
 * The layer (source: "Qwen MoE BringUp", IREE ONNX Runtime EP issue #34,
 * the Qwen1.5-MoE-A2.7B-Chat INT4 IR Guide, section 3 "MoE Block"):
 *   logits = x . router_w (+ router_bias)          (Router: gate linear)
 *   p      = softmax(logits) over all E experts     (Router, kernel step 1)
 *   top-k  = the k largest p, best first            (Router, kernel step 2)
 *   for each chosen expert e of token t:
 *     g = x . Wg_e^T, u = x . Wu_e^T                (Expert Computation, step 4)
 *     act = g * sigmoid(g) * u                      (step 5, SwiGLU)
 *     y = act . Wd_e^T                              (step 6)
 *   out[t] = sum_j p[t, j] * y_j                    (step 7, not renormalised)
 * with every expert weight dequantised per DequantizeLinear with block_size
 * along the input dimension: w = (q - zp) * scale ("Qwen MoE BringUp",
 * local fix A1: extui -> uitofp -> subf -> mulf).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Pointers.  Every tensor pointer is a DEVICE pointer owned by the caller
 *   (cudaMalloc, torch, ...), on the current CUDA device, contiguous
 *   row-major.  The library never allocates, frees or copies host memory
 *   and never synchronises; all work is enqueued on `stream` (a
 *   cudaStream_t passed as void*, NULL = the legacy default stream).
 * Packed weights.  A projection with N outputs and K inputs, for all E
 *   experts, is three tensors:
 *     w      uint8  [E, N, K/2]   two uint4 codes per byte; element k of a
 *                                 row is in byte k/2, LOW nibble for even k
 *     scales fp16 or bf16 [E, N, K/block_size]
 *     zp     uint8  [E, N, K/block_size], values 0..15, or NULL meaning
 *                                 zero point 8 (signed symmetric int4)
 *   This is the IR guide's pre-transposed layout ([out, in], Optimization
 *   Opportunities item 5); gate/up have N = I, K = H; down has N = H, K = I.
 * Alignment.  x, out, router_w and every w must be 16-byte aligned; K must
 *   be a multiple of 32 and of block_size; block_size is 32, 64 or 128.
 * Errors.  Arguments are checked on the host before anything is enqueued;
 *   a bad argument returns QMOE_ERR_INVALID_ARG / QMOE_ERR_UNSUPPORTED /
 *   QMOE_ERR_WORKSPACE and enqueues nothing.  A failed launch returns
 *   QMOE_ERR_CUDA.  Conditions found on the device (a bounded wait that ran
 *   out) set bits in a status word kept in the workspace; read and clear it
 *   with qmoe_get_device_status.  No C++ exception crosses this ABI.
 * Device.  Compute capability 10.3 (sm_103a) only; any other device
 *   returns QMOE_ERR_UNSUPPORTED.  There is no CPU fallback.
 * Concurrency.  Calls that share a workspace must be ordered on one stream.
 */
#ifndef QMOE_H_
#define QMOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  QMOE_OK = 0,
  QMOE_ERR_INVALID_ARG = 1,  /* NULL / out-of-range / misaligned argument   */
  QMOE_ERR_UNSUPPORTED = 2,  /* valid but not supported (device, shape)     */
  QMOE_ERR_WORKSPACE = 3,    /* workspace NULL or smaller than required     */
  QMOE_ERR_CUDA = 4,         /* a CUDA runtime call or launch failed        */
  QMOE_ERR_TIMEOUT = 5,      /* device status: a bounded wait ran out       */
  QMOE_ERR_DEVICE_CHECK = 6  /* device status: an index or range check failed */
} qmoe_status;

/* Bits of a device status word (qmoe_get_device_status's *bits_out). */
typedef enum {
  QMOE_ST_TIMEOUT = 1, /* a bounded wait ran out                                 -> QMOE_ERR_TIMEOUT */
  QMOE_ST_INDEX = 2,   /* an index check failed                                  -> QMOE_ERR_DEVICE_CHECK */
  QMOE_ST_RANGE = 4    /* a value outside a format's or accumulator's range       -> QMOE_ERR_DEVICE_CHECK */
} qmoe_status_bit;

/* QMOE_F32 is taken by the microscaled and FP8 entry points that say so, no others. */
typedef enum { QMOE_F16 = 0, QMOE_BF16 = 1, QMOE_F32 = 2 } qmoe_dtype;

/* Path selection for qmoe_forward_ex.
 *   DECODE        per-token GEMV on CUDA cores, fp32 throughout (small T).
 *                 At T = 1 (gate/up and down either all with or all without
 *                 zero points, and a shared-memory plan that fits) the whole
 *                 layer runs as one kernel; otherwise as three kernels
 *                 (router; gate-up + SwiGLU; down + weighted sum).  The one
 *                 kernel splits the down projection along I over clusters of
 *                 4 CTAs and adds the partial outputs into an integer
 *                 fixed-point accumulator (2^-32), so the sum does not depend
 *                 on arrival order; it has no grid-wide wait, so it runs
 *                 with any number of SMs available, and its results are
 *                 bit-reproducible.
 *   PREFILL       tokens grouped by expert, grouped GEMM on the tensor cores
 *                 with fp32 accumulation and exact operands: with bf16 block
 *                 scales the operands are fp16 (bf16 activations convert
 *                 exactly within fp16's normal range) and, without zero
 *                 points, each dequantised weight is one fp16 operand
 *                 (s (q - 8) has at most 11 significant bits); with zero
 *                 points or fp16 scales each weight is the exact sum of two
 *                 operands (hi = RN(w), lo = w - hi) of fp16, or of bf16
 *                 for bf16 activations with fp16 scales.  The SwiGLU
 *                 output enters the down projection as hi + lo of the
 *                 operand type.  So the only roundings are fp32
 *                 accumulation, the hi + lo SwiGLU output and the final
 *                 output (on the fp16 operands, values below fp16's
 *                 normal range, 2^-14, round to its subnormals: an absolute
 *                 error of at most 2^-25).  A bf16 activation or SwiGLU value beyond fp16's
 *                 range (65504) on the fp16-operand form sets a device
 *                 status bit (QMOE_ERR_DEVICE_CHECK).  (Value 3 of this
 *                 enum is not used: a single-rounded-operand form that
 *                 missed the elementwise tolerance was withdrawn.)
 *   DECODE_SPLIT  DECODE as three kernels always.
 *   DECODE_FUSED  DECODE as the one kernel (for T <= 4 where a CTA's share
 *                 of the selected experts fits in shared memory: at the
 *                 Qwen1.5-MoE-A2.7B layer shape only T = 1);
 *                 QMOE_ERR_UNSUPPORTED where it does not fit.  Its routing
 *                 equals DECODE_SPLIT's bit for bit; its output differs from
 *                 DECODE_SPLIT's only by the order of fp32 sums in the down
 *                 projection.
 *   AUTO          DECODE for T <= QMOE_AUTO_DECODE_MAX_TOKENS, else PREFILL
 *                 (DECODE where PREFILL's shape rules do not hold). */
typedef enum {
  QMOE_PATH_AUTO = 0,
  QMOE_PATH_DECODE = 1,
  QMOE_PATH_PREFILL = 2,
  QMOE_PATH_DECODE_SPLIT = 4,
  QMOE_PATH_DECODE_FUSED = 5
} qmoe_path;

/* One projection for all E experts (see "Packed weights" above). */
typedef struct {
  const uint8_t* w;
  const void* scales;
  const uint8_t* zp; /* may be NULL: zero point 8 */
} qmoe_qweight;

/* Largest shapes accepted: E <= 256 experts, 1 <= k <= 8. */
#define QMOE_MAX_EXPERTS 256
#define QMOE_MAX_TOPK 8
/* Most tokens the decode (GEMV) path takes (QMOE_PATH_DECODE). */
#define QMOE_DECODE_MAX_TOKENS 16
/* Tokens at or below this count take the decode path under QMOE_PATH_AUTO,
 * more take the grouped GEMM (when its shape rules hold, else decode up to
 * QMOE_DECODE_MAX_TOKENS).  Measured on GB300 at the Qwen1.5-MoE-A2.7B layer
 * shape (H 2048, I 1408, E 60, k 4, block 32, fp16, zero points), per layer:
 * decode 80 / 132 / 182 / 234 us and grouped GEMM 88 / 122 / 150 / 172 us at
 * T = 4 / 8 / 12 / 16. */
#define QMOE_AUTO_DECODE_MAX_TOKENS 5

/* Human-readable name of a status code.  Never NULL. */
const char* qmoe_status_string(int status);

/* Text of the last CUDA runtime error an entry point on this thread turned
 * into QMOE_ERR_CUDA / QMOE_ERR_UNSUPPORTED ("no error" if none).  Never NULL. */
const char* qmoe_last_cuda_error(void);

/* Bytes of device workspace qmoe_route / qmoe_forward need for these
 * shapes (covers both paths).  The workspace is caller-owned, 256-byte
 * aligned device memory.  Before its FIRST use it must be prepared with
 * qmoe_workspace_init; every call leaves it ready for the next one. */
size_t qmoe_workspace_size(int T, int H, int I, int E, int k);

/* Zero the workspace's control block (device status, counters, and the
 * one-kernel decode layer's 128 KB output accumulator) on `stream`.  Every
 * call leaves the control block ready for the next one; after a call whose
 * device status reports QMOE_ERR_TIMEOUT or QMOE_ERR_DEVICE_CHECK, run this
 * again before the workspace's next use (a call that gave up part-way can
 * leave counters or the accumulator mid-update). */
int qmoe_workspace_init(void* workspace, size_t workspace_bytes, void* stream);

/* Diagnostics of the failure path, kept in the workspace's control block
 * (qmoe_workspace_init clears both; callers otherwise leave them).
 *   wait_limit_kilocycles  the grouped GEMM's bounded waits (prefill path and
 *                          the tensor-core matmul_nbits_ex) give up after
 *                          this many x 1024 SM cycles; 0: the default,
 *                          about 2 s.
 *   flags                  QMOE_DIAG_STALL_GEMM: the GEMM's dequantiser warps
 *                          wait for a copy that cannot arrive, so that wait
 *                          runs out; 0: none.
 * A wait that gives up sets QMOE_ST_TIMEOUT; the kernel's roles then drain
 * their copies and MMAs in flight, free TMEM and return (no trap, no hang);
 * qmoe_get_device_status reports QMOE_ERR_TIMEOUT and that call's output is
 * undefined.  The workspace stays usable: with the diagnostics cleared the
 * next call computes normally.  Asynchronous on `stream` (an 8-byte copy
 * into the control block).  QMOE_ERR_INVALID_ARG for unknown flags. */
#define QMOE_DIAG_STALL_GEMM 1u
int qmoe_workspace_set_diagnostics(void* workspace, size_t workspace_bytes, uint32_t wait_limit_kilocycles,
                                   uint32_t flags, void* stream);

/* Router: logits = x[T,H] . router_w[H,E] (+ router_bias[E]) accumulated in
 * fp32 (on CUDA cores for T <= 16; on the tensor cores for T > 16 when H is
 * a multiple of 64, E <= 128 and x is 16-byte aligned: exact 16-bit products
 * summed in fp32, the sum of the K-split partials in a fixed order);
 * softmax over all E in fp32; the k largest probabilities, best first,
 * equal probabilities ordered by lower expert id; weights are the raw
 * probabilities (not renormalised).  Then the assignments a = t*k + j are
 * grouped by expert ("sort tokens by expert", IR guide Optimization
 * Opportunities item 9 step 1).
 *   x, router_w : act_dtype (fp16 or bf16), [T,H] and [H,E]
 *   router_bias : fp32 [E] or NULL
 *   topk_w      : fp32 [T,k] out;  topk_ids : int32 [T,k] out
 *   expert_offsets : int32 [E+1] out or NULL: offsets[e] = number of
 *                 assignments to experts < e, offsets[E] = T*k
 *   perm        : int32 [T*k] out or NULL: assignment ids grouped by
 *                 expert, increasing within an expert
 * Requires 1 <= T, 1 <= k <= min(E, 8), E <= 256. */
int qmoe_route(const void* x, const void* router_w, int act_dtype, const float* router_bias,
               int T, int H, int E, int k, float* topk_w, int32_t* topk_ids,
               int32_t* expert_offsets, int32_t* perm, void* workspace, size_t workspace_bytes,
               void* stream);

/* MatMulNBits: y[M,N] = x[M,K] . dequant(W)[N,K]^T with W one packed
 * [N, K/2] matrix (E = 1 in the layout above), fp32 accumulation, y rounded
 * to act_dtype.  Small M streams W through CUDA cores; no workspace. */
int matmul_nbits(const void* x, int act_dtype, const uint8_t* w, const void* scales,
                 int scale_dtype, const uint8_t* zp, int M, int N, int K, int block_size, void* y,
                 void* stream);

/* matmul_nbits with an explicit path and a workspace, for any M (MatMulNBits,
 * IR guide section 2 "Quantization Scheme" for the weight format and the
 * dequantize-then-matmul definition).  path:
 *   DECODE        the CUDA-core path above (workspace unused, may be NULL);
 *   PREFILL       tensor cores (tcgen05) with exact operands as in the
 *                 layer's prefill path (one fp16 weight operand for bf16
 *                 scales without zero points, else hi + lo) and x as one
 *                 operand;
 *   AUTO          DECODE for M <= QMOE_DECODE_MAX_TOKENS, else PREFILL.
 * The tensor-core path needs N % 128 == 0, K % 64 == 0, x, y, scales and
 * zero points 16-byte aligned and an initialised workspace (qmoe_workspace_init)
 * of at least qmoe_workspace_size(M, N, K, 1, 1) bytes (QMOE_ERR_WORKSPACE if
 * smaller); other shapes return QMOE_ERR_UNSUPPORTED.  y is fully written;
 * x, w, scales and zp are read only.  Stream-ordered. */
int matmul_nbits_ex(const void* x, int act_dtype, const uint8_t* w, const void* scales,
                    int scale_dtype, const uint8_t* zp, int M, int N, int K, int block_size,
                    void* y, int path, void* workspace, size_t workspace_bytes, void* stream);

/* The whole layer: out[T,H] (act_dtype) = sum over the k chosen experts of
 * p * SwiGLU-FFN_e(x).  gate/up are [E, I, H/2] (N = I, K = H), down is
 * [E, H, I/2] (N = H, K = I); all three share scale_dtype and block_size.
 * topk_w_out / topk_ids_out ([T,k], may be NULL) return the routing used.
 * If accumulate is non-zero, out = out + layer(x) (residual add).
 * Requires H and I multiples of 32 and of block_size. */
int qmoe_forward(const void* x, int act_dtype, const void* router_w, const float* router_bias,
                 qmoe_qweight gate, qmoe_qweight up, qmoe_qweight down, int scale_dtype, int T,
                 int H, int I, int E, int k, int block_size, void* out, float* topk_w_out,
                 int32_t* topk_ids_out, int accumulate, void* workspace, size_t workspace_bytes,
                 void* stream);

/* qmoe_forward with an explicit path (QMOE_PATH_*); AUTO picks decode for
 * T <= QMOE_AUTO_DECODE_MAX_TOKENS. */
int qmoe_forward_ex(const void* x, int act_dtype, const void* router_w, const float* router_bias,
                    qmoe_qweight gate, qmoe_qweight up, qmoe_qweight down, int scale_dtype, int T,
                    int H, int I, int E, int k, int block_size, void* out, float* topk_w_out,
                    int32_t* topk_ids_out, int accumulate, int path, void* workspace,
                    size_t workspace_bytes, void* stream);

/* Number of kernels one qmoe_forward_ex call with these sizes and this path
 * launches on the current device: 1 (decode layer fused into one
 * kernel), 3 (decode: router, gate-up, down) or 5 (prefill:
 * router, token permutation, two grouped GEMMs, output conversion).  Host
 * only, nothing launched.  Negative status (-QMOE_ERR_*) if the arguments
 * are invalid or the shape is unsupported.  Pointer alignment is not known
 * here and is assumed to meet the call's rules. */
int qmoe_forward_kernels(int T, int H, int I, int E, int k, int block_size, int act_dtype,
                         int scale_dtype, int gate_up_has_zp, int down_has_zp, int path);

/* qmoe_forward_ex for profiling: records events[0] before the first kernel
 * and events[i] after kernel i (router, gate-up, down on the decode path),
 * for i < n_events (cudaEvent_t passed as void*; NULL entries skipped).  The
 * kernels run back to back without programmatic overlap, so event pairs
 * bracket one kernel each.  Same arguments and results as qmoe_forward. */
int qmoe_forward_profiled(const void* x, int act_dtype, const void* router_w,
                          const float* router_bias, qmoe_qweight gate, qmoe_qweight up,
                          qmoe_qweight down, int scale_dtype, int T, int H, int I, int E, int k,
                          int block_size, void* out, int path, void* workspace,
                          size_t workspace_bytes, void* stream, void* const* events,
                          int n_events);

/* Shared expert of the MoE block ("Qwen MoE BringUp", IR guide section 3,
 * "Shared Expert"): every token goes through one more SwiGLU expert whose
 * output, scaled by a sigmoid gate, is added to the block's output:
 *   out[t] (+)= sigmoid(x[t] . shared_gate_w) * FFN(x[t])
 * shared_gate_w is a [H] vector in act_dtype.  The expert's weights use the
 * same INT4 block format as the routed experts with E = 1: gate/up
 * [1, I, H/2], down [1, H, I/2] (the pages' model keeps this expert in fp16;
 * here it is quantised like the others).  It runs as the layer with one
 * expert, top-1, the gate vector as its router and a sigmoid in place of the
 * softmax, so the whole MoE block is
 *   qmoe_forward(..., out, accumulate)  then
 *   qmoe_shared_expert(..., out, accumulate = 1).
 * Workspace: qmoe_workspace_size(T, H, I, 1, 1).  Same conventions and
 * errors as qmoe_forward; shared_gate_w NULL -> QMOE_ERR_INVALID_ARG. */
int qmoe_shared_expert(const void* x, int act_dtype, const void* shared_gate_w, qmoe_qweight gate,
                       qmoe_qweight up, qmoe_qweight down, int scale_dtype, int T, int H, int I,
                       int block_size, void* out, int accumulate, void* workspace, size_t workspace_bytes,
                       void* stream);

/* qmoe_forward without a caller workspace.  An engineering addition with no
 * counterpart in the method's sources: it serves callers that cannot give
 * the library device memory, such as a plain C host program with no device
 * allocator, or a plugin hook that receives no workspace argument and must
 * not call cudaMalloc (which synchronises the whole device).
 *
 * The workspace is a library-owned static device array of
 * QMOE_NOALLOC_SCRATCH_BYTES (2 MiB) per device; the call allocates
 * nothing.  Its control block (device status word, counters, the one-kernel
 * decode layer's output accumulator) starts at zero when the library is
 * loaded and every call leaves the counters and the accumulator at zero
 * again.  The first call on a device
 * looks the array's address up (cudaGetSymbolAddress), so make that first
 * call, with the device current, before any stream capture.
 *
 * Same arguments and results as qmoe_forward (path chosen as by
 * QMOE_PATH_AUTO), minus the workspace.  Shapes whose workspace
 * (qmoe_workspace_size) exceeds QMOE_NOALLOC_SCRATCH_BYTES return
 * QMOE_ERR_UNSUPPORTED and enqueue nothing; the Qwen1.5-MoE-A2.7B layer
 * shape fits up to T = 16.  Overlapping calls on one device (two streams,
 * or two host threads without ordering) share the array and race: order
 * them on one stream.  Device-side conditions (a bounded wait that ran out)
 * are recorded in the scratch's status word: read it with
 * qmoe_noalloc_status. */
#define QMOE_NOALLOC_SCRATCH_BYTES (2u << 20)
int qmoe_forward_noalloc(const void* x, int act_dtype, const void* router_w, const float* router_bias,
                         qmoe_qweight gate, qmoe_qweight up, qmoe_qweight down, int scale_dtype, int T,
                         int H, int I, int E, int k, int block_size, void* out, float* topk_w_out,
                         int32_t* topk_ids_out, int accumulate, void* stream);

/* The device status word of qmoe_forward_noalloc's static scratch on the
 * current device, read and cleared like qmoe_get_device_status (blocking:
 * synchronises `stream`).  Returns QMOE_OK, or the first QMOE_ERR_* a kernel
 * recorded since the last read (a bounded wait that ran out, a failed index
 * or launch-shape check: the output of that call is not valid); *bits_out
 * (may be NULL) gets the raw bits.  After QMOE_ERR_TIMEOUT the scratch's
 * counters may be left mid-count: the library has no allocation-free way to
 * reset them, so such a process should stop using this entry point. */
int qmoe_noalloc_status(uint32_t* bits_out, void* stream);

/* DequantizeLinear of one [N, K] matrix (packed [N, K/2]) to fp32 out[N,K]:
 * (q - zp) * scale, which fp32 holds exactly. */
int qmoe_dequant(const uint8_t* w, const void* scales, int scale_dtype, const uint8_t* zp, int N,
                 int K, int block_size, float* out, void* stream);

/* RMSNorm of the layer stack ("IR guide", 1. RMSNorm) with unit weight:
 * out[t,h] = x[t,h] / sqrt(mean_h(x[t,h]^2) + eps), computed in fp32 and
 * rounded to act_dtype.  x and out may alias. */
int qmoe_rmsnorm(const void* x, void* out, int act_dtype, int T, int H, float eps, void* stream);

/* ---- Weight-format adapters (one-time conversion at model load).
 *
 * GPTQ checkpoints into the canonical layout above ("Qwen MoE BringUp",
 * "Bugs/Issues Found", item 1: GPTQ zero points are stored with an offset
 * of +1 or +0 depending on the exporter, told apart by the median stored
 * zero).  Source layout, per expert e (E experts stacked, input-major):
 *   qweight [E, K/8, N]    int32: bits 4j..4j+3 of word (i, n) = q[8i + j, n]
 *   qzeros  [E, K/bs, N/8] int32: bits 4j..4j+3 of word (g, i) = stored zero
 *                          of block g, column 8i + j; or NULL (symmetric
 *                          int4 without zero points)
 *   scales  [E, K/bs, N]   16-bit (fp16 or bf16, copied bit for bit)
 * Output: w_out [E, N, K/2], scales_out [E, N, K/bs], zp_out [E, N, K/bs]
 * (NULL exactly when qzeros is NULL; the canonical layout then implies
 * zero point 8).  zp = stored + offset: the offset is *zero_offset_dev
 * when that device pointer is given (for example the output of
 * qmoe_gptq_zero_offset, read by the kernel, so no host round trip), else
 * zero_offset (0 or 1).  A zero point of 16 (a stored 15 with offset 1)
 * does not fit the canonical 4-bit zero point: it is written as 15 and, if
 * status_dev (a 4-byte device word, may be NULL) is given, QMOE_ST_RANGE is
 * OR-ed into it; read it with qmoe_get_device_status(status_dev, ...),
 * which returns QMOE_ERR_DEVICE_CHECK when the bit is set.  The weights of
 * such blocks differ from the checkpoint's by one scale step, so a caller
 * should refuse the checkpoint.  Requires N a multiple of 8, K a
 * multiple of 32 and of block_size (32, 64, 128); 4-byte aligned int32
 * buffers and w_out, 2-byte aligned scales.  Asynchronous on `stream`;
 * input and output must not overlap.  Bound by HBM (every byte read and
 * written once). */
int qmoe_repack_gptq(const int32_t* qweight, const int32_t* qzeros, const void* scales, int E, int K,
                     int N, int block_size, int zero_offset, const int32_t* zero_offset_dev,
                     uint8_t* w_out, void* scales_out, uint8_t* zp_out, uint32_t* status_dev, void* stream);

/* The GPTQ zero-point offset of a qzeros tensor (n_words int32 words, all
 * experts and projections the caller wants to judge together), written to
 * the device int *offset_out: 1 if the lower median of the stored zero
 * points is 7 (the exporter stored zero - 1), else 0.  Asynchronous; pass
 * offset_out to qmoe_repack_gptq as zero_offset_dev. */
int qmoe_gptq_zero_offset(const int32_t* qzeros, size_t n_words, int32_t* offset_out, void* stream);

/* Packed 4-bit zero points [rows, ceil(nb/2)] (two per byte, block 2b in
 * the low nibble, 2b + 1 in the high nibble, each row padded to a byte)
 * into the canonical one byte per block [rows, nb].  The pages' model
 * already stores one byte per block; this is the packing ONNX MatMulNBits
 * uses for 4-bit zero points.  rows = E * N for a stacked projection. */
int qmoe_unpack_zero_points(const uint8_t* zp_packed, int rows, int nb, uint8_t* zp_out, void* stream);

/* ---- Microscaled (MX) formats: OCP Microscaling v1.0 blocks of 32 elements.
 *
 * An MX tensor [R, K] (K a multiple of 32) is two device buffers:
 *   codes   MXFP8: uint8 [R, K], one e4m3 code per element;
 *           MXFP4: uint8 [R, K/2], two e2m1 codes per byte, element k of a
 *           row in byte k/2, LOW nibble for even k;
 *   scales  one e8m0 byte s per block of 32 elements along K: the block's
 *           scale is X = 2^(s - 127), 255 is NaN.  They lie in tiles of 128
 *           rows x 4 blocks, 512 bytes each, tiles row-major over
 *           [ceil(R/128), ceil(K/128)]; row r, block b is at byte
 *             (r/128 * ceil(K/128) + b/4) * 512 + r%32 * 16 + r%128/32 * 4 + b%4.
 *           Tensor memory holds a product's scales in this order, so the
 *           tiles are copied there as they are.  Bytes for rows >= R and
 *           blocks >= K/32 are padding: the calls below write zeros there.
 *           qmoe_mx_scale_bytes(R, K) gives the size.
 * An element's value is code * X.  R and K are at most 2^30
 * (QMOE_ERR_UNSUPPORTED).  Every codes and scales pointer is 16-byte aligned;
 * codes, scales, inputs and outputs of one call must not overlap
 * (qmoe_rmsnorm_mx's residual_out is the exception). */
typedef enum { QMOE_MXFP8 = 0, QMOE_MXFP4 = 1 } qmoe_mx_format;

/* Bytes of the scale tiles of an MX tensor [R, K]; 0 for R < 1, K < 32 or K
 * not a multiple of 32.  Host only. */
size_t qmoe_mx_scale_bytes(int R, int K);

/* Quantise x [M, K] (fp16, bf16 or fp32; finite or not) to an MX tensor:
 *   s    = clamp(floor(log2(max |v| of the block)) - emax, -127, 127) + 127,
 *          emax = 8 (e4m3, largest 448) or 2 (e2m1, largest 6); an all-zero
 *          block has s = 0;
 *   code = v / X rounded to nearest even, saturating at the largest value.
 * A block that holds a NaN or an infinity gets s = 255 and zero codes: all
 * its elements read as NaN.  x is 16-byte aligned.  Bound by HBM. */
int qmoe_mx_quantize(const void* x, int x_dtype, int format, int M, int K, uint8_t* codes, uint8_t* scales,
                     void* stream);

/* The values of an MX tensor: out [M, K] (fp16, bf16 or fp32) = code * X,
 * exact in fp32 and rounded once to out_dtype.  out is 16-byte aligned. */
int qmoe_mx_dequant(const uint8_t* codes, const uint8_t* scales, int format, int M, int K, void* out, int out_dtype,
                    void* stream);

/* RMSNorm of the layer stack with the residual's addition and microscaled
 * output, for a product that takes it (qmoe_mx_matmul):
 *   h = x + residual (fp32);  residual_out = h rounded to act_dtype;
 *   y = h / sqrt(mean_h(h^2) + eps) * weight (fp32, from the unrounded h);
 *   codes, scales = y [T, H] quantised as by qmoe_mx_quantize.
 * x, residual, residual_out [T, H] and weight [H] are fp16 or bf16
 * (act_dtype).  residual may be NULL (h = x), weight may be NULL (unit
 * weight), residual_out may be NULL (not wanted) and may be x or residual
 * itself.  Requires H a multiple of 32; pointers 16-byte aligned.  A NaN makes
 * its whole row read as NaN; an infinity makes its own block NaN and the rest
 * of its row 0 (also where the sum of squares leaves fp32's range).  With eps
 * = 0, rows whose largest |h| is below 2^-60 lose accuracy, and read as NaN
 * where their squares vanish in fp32. */
int qmoe_rmsnorm_mx(const void* x, const void* residual, const void* weight, int act_dtype, int T, int H, float eps,
                    int format, void* residual_out, uint8_t* codes, uint8_t* scales, void* stream);

/* Product with MXFP4 weights: y[M, N] = x . W^T, x an MX tensor [M, K] of
 * x_format (MXFP8 or MXFP4), W an MXFP4 tensor [N, K]; products are exact,
 * sums are fp32, and y is rounded once to y_dtype (fp16, bf16 or fp32;
 * y aligned to its element size).  Any M and N >= 1.  A NaN scale makes the
 * outputs of its row NaN; the scales' padding behind K has to be zeros (the
 * calls here write it so), that behind the last row may be anything.
 * One kernel.  Its tile and the split of K are chosen by M, N, K, x_format,
 * whether w_codes lies on a 32-byte boundary (MXFP8 x), and the device: calls
 * that agree in these give the same bits, others sum in another order.
 * status_dev (a 4-byte device word that the caller set to 0): a bounded wait of the kernel that ran out sets QMOE_ST_TIMEOUT
 * there (y is then undefined); read it with qmoe_get_device_status(status_dev,
 * ...).  NULL: the same in a word of the library's, one per device
 * (qmoe_mx_status). */
int qmoe_mx_matmul(const uint8_t* x_codes, const uint8_t* x_scales, int x_format, const uint8_t* w_codes,
                   const uint8_t* w_scales, int M, int N, int K, void* y, int y_dtype, uint32_t* status_dev,
                   void* stream);

/* The form of the kernel that qmoe_mx_matmul runs for such a call on the
 * current device (no launch): variant_out[0] tokens per tile, [1] 1 for pairs
 * of CTAs, [2] CTAs that share a tile's K, [3] 1 where warps spread the
 * weights' codes.  w_codes is looked at for its alignment alone. */
int qmoe_mx_matmul_variant(int x_format, const uint8_t* w_codes, int M, int N, int K, int variant_out[4]);

/* The status word, on the current device, of the products that were given
 * none: read and cleared like qmoe_get_device_status (blocking: synchronises
 * `stream`, on which those products should have run).  QMOE_ERR_TIMEOUT: a
 * product since the last read is not valid. */
int qmoe_mx_status(uint32_t* bits_out, void* stream);

/* qmoe_mx_matmul with diagnostics of its failure path (all zero: the same).
 *   wait_limit_kilocycles  the kernel's bounded waits give up after this many
 *                          x 1024 SM cycles; 0: the default, about 2 s.
 *   flags                  the named role waits for what cannot arrive before
 *                          its first step, so that waits run out: the copies
 *                          of codes or of scales, the MMAs, the output, the
 *                          spreading of ragged rows' codes (MXFP8 x with K
 *                          not a multiple of 128 or w_codes off a 32-byte
 *                          boundary; else there is no such role).
 * The roles then drain, free tensor memory and return (no trap, no hang), and
 * the status reads QMOE_ST_TIMEOUT; the next call computes normally.
 * QMOE_ERR_INVALID_ARG for unknown flags. */
#define QMOE_DIAG_STALL_MX_CODES 1u
#define QMOE_DIAG_STALL_MX_SCALES 2u
#define QMOE_DIAG_STALL_MX_MMA 4u
#define QMOE_DIAG_STALL_MX_OUTPUT 8u
#define QMOE_DIAG_STALL_MX_SPREAD 16u
int qmoe_mx_matmul_diagnosed(const uint8_t* x_codes, const uint8_t* x_scales, int x_format, const uint8_t* w_codes,
                             const uint8_t* w_scales, int M, int N, int K, void* y, int y_dtype, uint32_t* status_dev,
                             uint32_t wait_limit_kilocycles, uint32_t flags, void* stream);

/* Scale-layout adapters (one-time conversion at model load): row-major
 * scales [R, K/32], as checkpoints store them, into the tiles above, and
 * back.  in and out are separate buffers of any alignment on the row-major
 * side. */
int qmoe_mx_tile_scales(const uint8_t* scales_rowmajor, int R, int K, uint8_t* scales, void* stream);
int qmoe_mx_untile_scales(const uint8_t* scales, int R, int K, uint8_t* scales_rowmajor, void* stream);

/* ---- FP8 tensors with a scale for each block of 128 (e4m3), and experts in
 * that format: quantisation, products (dense or grouped by expert), tokens put
 * in the order of their experts and brought back.  A layer of them:
 *   qmoe_route                    topk_w, topk_ids
 *   qmoe_sort_experts             offsets, pos
 *   qmoe_fp8_quantize (pos)       the tokens in 8 bits, in the experts' order
 *   qmoe_fp8_matmul (offsets)     gate and up: weights [E, 2 I, H]
 *   qmoe_fp8_quantize_swiglu      silu(gate) * up in 8 bits
 *   qmoe_fp8_matmul (offsets)     down: weights [E, H, I]
 *   qmoe_combine (pos, topk_w)    the weighted sum, onto a residual
 *
 * An FP8 tensor is two device buffers:
 *   codes   uint8, one e4m3 code per element (largest 448; 127 and 255: NaN);
 *           activations [M, K], weights [E, N, K], K a multiple of 16; 16-byte
 *           aligned;
 *   scales  fp32, row-major; activations [M, ceil(K/128)]: one per row and 128
 *           columns; weights [E, ceil(N/128), ceil(K/128)]: one per 128 rows of
 *           an expert and 128 columns.  The last block of a row or column may be
 *           shorter.  4-byte aligned.
 * An element's value is code * scale.  Quantisation, with a the largest
 * magnitude of the block, at least 2^-100:
 *   scale = fp32(a / 448),  code = v * fp32(448 / a) rounded to nearest even
 * (the product rounded once, as if it were exact before).  A block with a NaN
 * or an infinity gets a NaN scale and zero codes.
 * K is at most 2^30 and so are M and E * N (QMOE_ERR_UNSUPPORTED).  Inputs and
 * outputs of one call must not overlap (but for qmoe_combine's out, which may be
 * its residual, and qmoe_combine_backward's dys, which may be its ys).
 *
 * pos int32 [T, k] gives the place of each assignment t * k + j among the rows
 * of the experts' order, T * k of them: row pos[t, j] belongs to token t.  An
 * entry outside 0 .. T * k - 1 goes nowhere; no row may be named twice.  Rows
 * that no entry names are left as they were. */

/* Tokens to FP8.  x [T, K] (fp16, bf16 or fp32; 16-byte aligned).  pos NULL (k
 * then 0): codes and scales of T rows.  Else pos [T, k] and T * k rows: token
 * t is quantised once and written to each row pos[t, j].  Bound by HBM. */
int qmoe_fp8_quantize(const void* x, int x_dtype, int T, int K, const int32_t* pos, int k, uint8_t* codes, float* scales,
                      void* stream);

/* silu(gate) * up = gate / (1 + exp(-gate)) * up of h [M, 2 I] (gate in the
 * first I columns; fp16, bf16 or fp32; 16-byte aligned), computed in fp32 (within
 * 9 2^-24 of itself, whatever the gate) and quantised to codes [M, I] without a
 * rounding in between.  I a multiple of 16.
 * Bound by its instructions at many rows. */
int qmoe_fp8_quantize_swiglu(const void* h, int h_dtype, int M, int I, uint8_t* codes, float* scales, void* stream);

/* Weights w [E, N, K] (fp16, bf16 or fp32; 16-byte aligned) to FP8, a scale for
 * each 128 x 128 elements of an expert.  (The transposed weights' codes and
 * scales are the transposed ones, so the gradient of a product with respect to
 * x is a product with them.)  Bound by HBM. */
int qmoe_fp8_quantize_weights(const void* w, int w_dtype, int E, int N, int K, uint8_t* codes, float* scales, void* stream);

/* Values of an FP8 tensor: out (fp16, bf16 or fp32; 16-byte aligned) = code *
 * scale in fp32, rounded once to out_dtype.  block_rows 1: activations [E * N,
 * K]; 128: weights [E, N, K]. */
int qmoe_fp8_dequant(const uint8_t* codes, const float* scales, int E, int N, int K, int block_rows, void* out,
                     int out_dtype, void* stream);

/* Product of FP8 tensors: y[m, n] = sum_k x[m, k] W[n, k], the codes' products
 * summed in fp32 over each block of 128 k, these sums times their scales summed
 * in fp32, y rounded once to y_dtype (fp16, bf16 or fp32; aligned to its
 * element size).
 *   offsets NULL  dense: E is 1, y [M, N] = x [M, K] . W [N, K]^T.
 *   offsets       int32 [E + 1] on the device, as qmoe_sort_experts and
 *                 qmoe_route give them: rows offsets[e] .. offsets[e + 1] - 1 of
 *                 x and y belong to expert e, whose weights are W[e]; rows
 *                 outside every expert's are not read, and y's are left as they
 *                 were.  Offsets that decrease or leave 0 .. M set QMOE_ST_INDEX,
 *                 and all of y is left as it was.  At most QMOE_MAX_EXPERTS
 *                 experts.
 * A NaN scale or code makes the outputs that it enters NaN, and no others.  Scales
 * may be any fp32 numbers: a token with a pair of scales whose product fp32 does not
 * hold as a normal number is computed by a slow path (some 300 times the time).
 * One kernel.  Its tile and the split of K are chosen by E, M, N, K, whether
 * there are offsets, and the device: calls that agree in these give the same
 * bits, others sum in another order.
 * status_dev (a 4-byte device word that the caller set to 0, or NULL): collects
 * QMOE_ST_INDEX, and QMOE_ST_TIMEOUT where a bounded wait ran out (y is then
 * undefined); read it with qmoe_get_device_status(status_dev, ...).  NULL: the
 * same in a word of the library's, one per device (qmoe_fp8_status). */
int qmoe_fp8_matmul(const uint8_t* x_codes, const float* x_scales, const uint8_t* w_codes, const float* w_scales,
                    const int32_t* offsets, int E, int M, int N, int K, void* y, int y_dtype, uint32_t* status_dev,
                    void* stream);

/* The form of the kernel that qmoe_fp8_matmul runs for such a call on the
 * current device (no launch): variant_out[1] 0: tiles of variant_out[0] tokens
 * by 128 outputs, 1: of 128 tokens by variant_out[0] outputs; [2] CTAs that share
 * a tile's K. */
int qmoe_fp8_matmul_variant(int grouped, int E, int M, int N, int K, int variant_out[3]);

/* qmoe_fp8_matmul with diagnostics of its failure path, as
 * qmoe_mx_matmul_diagnosed: the named roles (the copies of codes, the scales,
 * the MMAs, the sums and outputs) wait for what cannot arrive before their
 * first step, the waits give up after wait_limit_kilocycles x 1024 SM cycles (0:
 * about 2 s), and the status reads QMOE_ST_TIMEOUT.  QMOE_ERR_INVALID_ARG for
 * unknown flags. */
#define QMOE_DIAG_STALL_FP8_CODES 1u
#define QMOE_DIAG_STALL_FP8_SCALES 2u
#define QMOE_DIAG_STALL_FP8_MMA 4u
#define QMOE_DIAG_STALL_FP8_OUTPUT 8u
int qmoe_fp8_matmul_diagnosed(const uint8_t* x_codes, const float* x_scales, const uint8_t* w_codes,
                              const float* w_scales, const int32_t* offsets, int E, int M, int N, int K, void* y,
                              int y_dtype, uint32_t* status_dev, uint32_t wait_limit_kilocycles, uint32_t flags,
                              void* stream);

/* The status word, on the current device, of the FP8 products that were given
 * none: as qmoe_mx_status. */
int qmoe_fp8_status(uint32_t* bits_out, void* stream);

/* Assignments by expert: ids int32 [T, k] (from any router; the same expert may
 * come twice in a row), those outside 0 .. E - 1 (padding) go nowhere.
 *   offsets  int32 [E + 1] out or NULL: assignments to experts < e
 *   perm     int32 [T * k] out or NULL: assignments t * k + j by expert,
 *            increasing within an expert; -1 behind the last
 *   pos      int32 [T, k] out or NULL: the place of each in perm, or -1
 * 1 <= E <= QMOE_MAX_EXPERTS, 1 <= T * k <= 2^30.  One kernel, no workspace. */
int qmoe_sort_experts(const int32_t* ids, int T, int k, int E, int32_t* offsets, int32_t* perm, int32_t* pos,
                      void* stream);

/* Tokens in the experts' order: xs[pos[t, j]] = x[t].  x [T, H] and xs [T * k,
 * H] of dtype (fp16, bf16 or fp32), 16-byte aligned, H a multiple of 8.  Bound
 * by HBM. */
int qmoe_dispatch(const void* x, int dtype, int T, int H, int k, const int32_t* pos, void* xs, void* stream);

/* Its gradient: dx[t] = sum_j dxs[pos[t, j]], summed in fp32 in the order of j
 * and rounded once; qmoe_combine without weights and residual. */
int qmoe_dispatch_backward(const void* dxs, int dtype, const int32_t* pos, int T, int H, int k, void* dx, void* stream);

/* The experts' outputs back to their tokens:
 *   out[t] = residual[t] + sum_j w[t, j] ys[pos[t, j]]
 * in fp32, in this order, rounded once.  ys [T * k, H] of ys_dtype, residual
 * (NULL: none) and out [T, H] of out_dtype (each fp16, bf16 or fp32), w fp32 [T,
 * k] (NULL: ones).  out may be residual.  H a multiple of 8, tensors 16-byte
 * aligned.  Rows that go nowhere are not read.  Bound by HBM. */
int qmoe_combine(const void* ys, int ys_dtype, const int32_t* pos, const float* w, const void* residual, int T, int H, int k,
                 void* out, int out_dtype, void* stream);

/* Its gradients, from dout [T, H] of dout_dtype:
 *   dys[pos[t, j]] = w[t, j] dout[t]                 [T * k, H], ys_dtype; NULL: not wanted
 *   dw[t, j] = sum_h dout[t, h] ys[pos[t, j], h]     fp32 [T, k]; 0 where j goes nowhere; NULL: not wanted
 * (the residual's gradient is dout).  ys may be NULL where dw is.  Sums are
 * fp32, in a fixed order.  dys may be ys.  H a multiple of 8.  Bound by HBM. */
int qmoe_combine_backward(const void* dout, int dout_dtype, const void* ys, int ys_dtype, const int32_t* pos,
                          const float* w, int T, int H, int k, void* dys, float* dw, void* stream);

/* Read (blocking: synchronises `stream`) and clear the device status word
 * of `workspace` (its first 4 bytes; also any 4-byte status word such as
 * qmoe_repack_gptq's status_dev).  Returns QMOE_OK, or QMOE_ERR_TIMEOUT
 * if a wait ran out, else QMOE_ERR_DEVICE_CHECK if an index or range check
 * failed since the last read; *bits_out (may be NULL) gets the raw bits
 * (QMOE_ST_*). */
int qmoe_get_device_status(void* workspace, uint32_t* bits_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QMOE_H_ */
