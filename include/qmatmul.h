/*
 * qmatmul.h -- C ABI of the MI355X (gfx950) GGUF quantized matmul library.
 *
 * Computes y[M x N] = x[M x K] . W[N x K]^T where W is stored as GGUF
 * quantized blocks exactly as a GGUF file stores a weight tensor: N rows, each
 * row K/QK consecutive blocks cut along K (page "自己量化", section
 * "2. q、k 投影的行重排": blocks run along a row).  x and y are f32, row-major,
 * contiguous.  y is overwritten.
 *
 * Two numerical modes, the two forms the page "同一个 GGUF，CPU 和 Metal
 * 生成的文字不一样" (section 出处) contrasts:
 *   QMM_MODE_F32ACT (a)  activations stay f32; weight blocks are dequantized
 *                        inside the kernel (the Metal form).  Accurate to f32.
 *   QMM_MODE_QACT   (b)  each activation row is first quantized on its own
 *                        (Q8_0 for Q8_0 weights, Q8K for Q4_K weights, per 32 or
 *                        256 values), then integer block dot products are
 *                        scaled by the weight and activation block scales (the
 *                        CPU form).
 * and the third form the same page (section 修法) sets against them:
 *   QMM_MODE_DEQUANT     every weight block decoded to f32 once, then a plain
 *                        f32 matmul (CANDLE_DEQUANTIZE_ALL): no activation
 *                        quantization, f32-sized weights.
 *
 * Block formats (little-endian; byte sizes fixed by the page "自己量化",
 * sections 和下载的 Q8_0 逐字节比 and 大小和误差):
 *   QMM_Q8_0   34 B per 32 values: f16 d, int8 q[32].
 *   QMM_Q4_K  144 B per 256 values: f16 d, f16 dmin, 12 B packed 6-bit
 *             sub-block scales and mins, 128 B of 4-bit values.
 *   QMM_Q8_K  292 B per 256 values (activations only): f32 d, int8 q[256],
 *             int16 bsums[16].
 * and the other formats of the pages' files (Q4_0 and Q5_0 sizes fixed by the
 * same page's byte counts, section 大小和误差 and the Q5_0 tensor totals of
 * 和下载的 Q8_0 逐字节比; Q6_K named there among the downloaded file's
 * tensors; the packings are the public GGUF layout, not printed by the pages):
 *   QMM_Q4_0   18 B per 32 values: f16 d, 16 B of 4-bit values (element j < 16
 *             in the low nibble of byte j, element j+16 in its high nibble);
 *             w = d*(q - 8).
 *   QMM_Q5_0   22 B per 32 values: f16 d, u32 of fifth bits (bit j of element
 *             j), 16 B of 4-bit values as Q4_0; w = d*(q - 16).
 *   QMM_Q6_K  210 B per 256 values: 128 B low 4 bits, 64 B high 2 bits, int8
 *             scales[16] (one per 16 values), f16 d; w = d*sc*(q - 32).
 * Mode (b) pairs Q4_0 and Q5_0 with Q8_0 activations and Q6_K with Q8K (page
 * "同一个 GGUF，CPU 和 Metal 生成的文字不一样", section 出处).  K must be a
 * multiple of the block size: 32 for Q8_0, Q4_0 and Q5_0, 256 for the
 * K-quants.  The kernels read 32-value blocks in pairs: rows with an odd
 * number of blocks run on copies one all-zero block longer, made in the plan's
 * workspace at every run (correct at any such K; the throughput is that of
 * the even case plus the copies).
 *
 * Pointers named "device" must be device memory of the current HIP device
 * (e.g. torch tensor data pointers); `stream` is a hipStream_t (NULL = the
 * null stream).  Every call that takes a stream is asynchronous: it enqueues
 * kernels and returns without synchronizing.  No call throws or aborts; each
 * returns a status code, and qmatmul_last_error() gives a message for the
 * calling thread.  Argument checks happen on the host before any HIP call.
 */
#ifndef QMATMUL_H
#define QMATMUL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* formats: the GGUF (ggml) type ids */
#define QMM_Q4_0 2
#define QMM_Q5_0 6
#define QMM_Q8_0 8
#define QMM_Q4_K 12
#define QMM_Q6_K 14
#define QMM_Q8_K 15

/* modes */
#define QMM_MODE_F32ACT 0
#define QMM_MODE_QACT 1
#define QMM_MODE_DEQUANT 2

/* status codes */
#define QMM_OK 0
#define QMM_EINVAL 1       /* null pointer, non-positive size, M > M_max, misaligned pointer */
#define QMM_EBLOCK 2       /* K not a multiple of the format's block size */
#define QMM_EUNSUPPORTED 3 /* unknown format or mode, or a format/mode pairing not offered */
#define QMM_ENOMEM 4       /* device allocation failed */
#define QMM_EHIP 5         /* a HIP runtime call or kernel launch failed */

typedef struct qmm_plan qmm_plan;

/*
 * Create a plan for one weight shape: format, N output rows, K inputs, up to
 * M_max activation rows per run, and a mode.  The mode is fixed here, as the
 * pages' QMatMul fixes its form when it is built (page "同一个 GGUF，CPU 和
 * Metal 生成的文字不一样", section 修法).  K must be a multiple of the block
 * size, 32 (Q8_0, Q4_0, Q5_0) or 256 (Q4_K, Q6_K), the shape check of page
 * "自己量化", section "3. 量化" (QMM_EBLOCK).
 * Allocates the plan's device workspace on the current device (hipMalloc).
 * On success *out receives the plan; on failure *out is set to NULL.
 */
int qmatmul_create(qmm_plan** out, int format, int64_t N, int64_t K, int64_t M_max, int mode);

/*
 * Run y = x . W^T on `stream`.  w_blocks: device, N * qmatmul_row_bytes(format, K)
 * bytes, 16-byte aligned.  x: device f32 [M x K].  y: device f32 [M x N],
 * overwritten.  0 <= M <= M_max; M == 0 enqueues nothing.  M <= 8 takes the
 * decode (GEMV) kernels, larger M the prefill (GEMM) kernels.  The caller owns
 * w, x and y; the plan keeps no pointer after the call.  The plan's workspace
 * is shared by its runs: do not run one plan concurrently on two streams.
 * At M > 8, Q8_0, Q4_0, Q5_0 and Q4_K runs with short rows (K <= 1536, at
 * most 8192 rows of W, a grid of at most one workgroup per compute unit) take
 * one launch that prepares its own activations; other Q4_0 and Q5_0 runs
 * first rewrite the weights as Q8_0 blocks (the same dequantized values) in
 * the plan's workspace and take the Q8_0 prefill kernels; Q6_K runs with
 * M > 8 take their own prefill kernel (both modes) on the f16 matrix cores.
 * A run only enqueues kernels (no allocation, memset or synchronization), so
 * runs may be captured in a HIP graph once each kernel has run eagerly (its
 * launch attributes are set on first use); the exception is a
 * QMM_MODE_DEQUANT plan, whose product is a rocBLAS call.
 */
int qmatmul_run(const qmm_plan* plan, const void* w_blocks, const float* x, float* y,
                int64_t M, void* stream);

/*
 * Grouped run: y[i] = x . W[i]^T for count plans that share format, K and mode
 * and one activation matrix x (M x K), such as the q, k and v (or gate and up)
 * projections of one layer; each product is the one qmatmul_run computes
 * (page "同一个 GGUF，CPU 和 Metal 生成的文字不一样", section 出处).  plans,
 * w_blocks and y are host arrays of count entries (1 <= count <=
 * QMM_GROUP_MAX) holding each plan's device pointers, with qmatmul_run's
 * sizes and alignment; 0 <= M <= every plan's M_max.  At M == 1 for Q8_0 and
 * Q4_K (where the one-row decode kernel takes the rows), and at M <= 8 for
 * Q4_0, Q5_0 and Q6_K (where their activations fit in LDS), the plans' rows
 * go to one launch per four plans (the activations are loaded and quantized
 * once per workgroup for all of them), giving bit-for-bit the values
 * separate runs give; at M > 8 each plan takes the prefill kernel its own run
 * takes, the plans' output tiles going to one launch per four plans of that
 * kernel (the activations prepared once for the K-staged kernels; again the
 * separate runs' values bit for bit); otherwise the plans run one after
 * another as with qmatmul_run.  Errors: as
 * qmatmul_run for each plan, and QMM_EINVAL for null arrays, count out of
 * range or plans that differ in format, K or mode.
 */
#define QMM_GROUP_MAX 8
int qmatmul_run_group(const qmm_plan* const* plans, int count, const void* const* w_blocks, const float* x,
                      float* const* y, int64_t M, void* stream);

/*
 * For callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc.  Computes
 * what qmatmul_create(format, N, K, M, mode) followed by qmatmul_run(..., M,
 * stream) computes, with the same kernels and the same values, but without a
 * plan and without allocating: the workspace lives in a static device array
 * of QMM_NOALLOC_SCRATCH_BYTES that each GPU holds from the library's first
 * use on it until the process ends (qmatmul_workspace_bytes(format, N, K, M,
 * mode) says what a shape needs).  w_blocks, x, y: device, as in qmatmul_run.
 * Errors: those of qmatmul_create and qmatmul_run; QMM_EINVAL when the shape
 * needs more scratch than the array holds; QMM_EUNSUPPORTED for
 * QMM_MODE_DEQUANT (its product is a library GEMM that allocates).  Every call on a GPU uses that GPU's one
 * array: calls that overlap on one GPU (on two streams, or from two host
 * threads) race and must be serialized by the caller.  The first call on
 * each device looks up the array's address (no allocation); its kernels set
 * their launch attributes on first use, so capture a call in a HIP graph only
 * after one eager call of the same shape.
 */
#define QMM_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
int qmatmul_run_noalloc(int format, int64_t N, int64_t K, int64_t M, int mode, const void* w_blocks,
                        const float* x, float* y, void* stream);

/* Free a plan and its workspace (NULL is a no-op).  Synchronizes the device
 * before freeing, so pending runs of the plan finish first. */
int qmatmul_destroy(qmm_plan* plan);

/*
 * Dequantize-all form (page "同一个 GGUF，CPU 和 Metal 生成的文字不一样",
 * section 修法: CANDLE_DEQUANTIZE_ALL decodes every quantized weight to f32 at
 * load, then both devices run a plain f32 matmul).
 *
 * qmatmul_dequantize_weights: GGUF blocks (device, N * qmatmul_row_bytes(format,
 * K) bytes, 16-byte aligned) -> f32 [N x K] (device, 16-byte aligned, caller
 * owned).  Every value is the exact dequantized weight (Q8_0 d*q; Q4_K
 * d*sc_j*q - dmin*m_j; Q4_0 d*(q-8); Q5_0 d*(q-16); Q6_K d*sc*(q-32)) rounded
 * once to f32.
 *
 * qmatmul_run_dequantized (QMM_MODE_DEQUANT plans only): y = x . W^T with W
 * given as that f32 [N x K] matrix; x, y as in qmatmul_run.  The product is the
 * library f32 GEMM (rocBLAS), deterministic.  qmatmul_run on a QMM_MODE_DEQUANT
 * plan decodes w_blocks into the plan's workspace (N*K*4 bytes) first and then
 * does the same; load-once callers decode with qmatmul_dequantize_weights and
 * call qmatmul_run_dequantized.
 */
int qmatmul_dequantize_weights(int format, const void* w_blocks, int64_t N, int64_t K, float* out,
                               void* stream);
int qmatmul_run_dequantized(const qmm_plan* plan, const float* w_f32, const float* x, float* y,
                            int64_t M, void* stream);

/*
 * Quantize activation rows the way mode (b) does, writing canonical blocks:
 * act_format QMM_Q8_0 (34 B per 32) or QMM_Q8_K (292 B per 256).  Row-local:
 * each row depends only on itself (page "自己量化", section 动脑筋答案).
 * x: device f32 [M x K]; out_blocks: device, M * qmatmul_row_bytes(act_format, K)
 * bytes.  Bit-identical to the quantization inside qmatmul_run.
 */
int qmatmul_quantize_act(int act_format, const float* x, int64_t M, int64_t K,
                         void* out_blocks, void* stream);

/*
 * Quantize f32 weights [N x K] (device) into GGUF blocks (device, N *
 * qmatmul_row_bytes(format, K) bytes), the role of QTensor::quantize on the
 * page "自己量化" (section "3. 量化").  Q8_0: d = max|w|/127, q = round(w/d).
 * Q4_K: per 32-value sub-block an affine min/max fit, 6-bit scales and mins
 * against the super-block maximum / 63, 4-bit values re-quantized against the
 * stored f16 scales (no importance matrix).  Q4_0 / Q5_0: the signed value of
 * largest magnitude takes the most negative code, d = max/-8 (-16), q =
 * floor(w/d + 8.5) (+ 16.5) capped at 15 (31).  Q6_K: per 16 values s = (signed
 * max)/-32, d = (signed s of largest magnitude)/-128, scales round(s/d) capped
 * at 127, q = clamp(round(w/(d*sc)), -32, 31) + 32.  w and out_blocks
 * 16-byte aligned.
 */
int qmatmul_quantize_weights(int format, const float* w, int64_t N, int64_t K,
                             void* out_blocks, void* stream);

/*
 * Q4_K weight quantizer with a search (the page "自己量化", section "3. 量化",
 * names QTensor::quantize(&w, Q4K) without describing its search): per
 * 32-value sub-block, candidate codes for 22 scales around the min/max
 * rule's (that rule's own among them), each refitted by least squares to a
 * scale and a non-negative min, the smallest squared error kept; then the
 * super-block's 6-bit scales and mins and the 4-bit values as
 * qmatmul_quantize_weights(QMM_Q4_K, ...) forms them.  w: device f32 [N x K],
 * K % 256 == 0; out_blocks: device, N * qmatmul_row_bytes(QMM_Q4_K, K) bytes;
 * both 16-byte aligned.  One thread per super-block (an offline step).
 */
int qmatmul_quantize_q4_k_search(const float* w, int64_t N, int64_t K, void* out_blocks, void* stream);

/*
 * Traced run (mode (b) plans only): qmatmul_run's own kernels, with the same
 * launch configuration, compiled with a flag that also writes out the integer
 * parts the method fixes exactly (page "同一个 GGUF，CPU 和 Metal 生成的文字不一样",
 * section 出处: integer block dot products, then the scales).
 *   y: as qmatmul_run writes it, bit for bit (NULL: not written).
 *   sums: device int32 [M x N x qmatmul_block_sums_per_row(format, K)]:
 *     Q8_0, Q4_0, Q5_0: S[m][n][b] = sum over block b of qw*qx, qw the signed
 *       weight value (q, q - 8, q - 16);
 *     Q4_K: per super-block ten values S_0..S_7 (per 32 values), sumi =
 *       sum_j sc_j*S_j and summins = sum_j m_j*(bsums[2j]+bsums[2j+1]);
 *     Q6_K: per super-block 17 values S_0..S_15 (per 16, qw = q - 32) and
 *       sumi = sum_j sc_j*S_j.
 *     At M > 8 the K-staged Q4_K prefill kernel scales each S_j on its own
 *     and never forms sumi; there sumi is summed from the S_j it wrote (the
 *     short-row kernel forms it in int32 itself).  The Q6_K
 *     prefill kernel (M > 8) carries the scales in its weight operand and
 *     forms sumi exactly but no per-16 sums: there S_0..S_15 read INT32_MIN.
 *   act_blocks: device, M * qmatmul_row_bytes(Q8_0 or Q8_K, K) bytes, 4-byte
 *     aligned, or NULL: the canonical quantized activation blocks, written by
 *     the kernel that quantizes them in this run (a decode kernel's own
 *     prologue, the short-row prefill's, or the prefill's activation
 *     preparation).
 * Same preconditions and errors as qmatmul_run; sums must not be NULL.
 */
int qmatmul_run_traced(const qmm_plan* plan, const void* w_blocks, const float* x, float* y, int32_t* sums,
                       void* act_blocks, int64_t M, void* stream);

/* qmatmul_run_traced(plan, w_blocks, x, NULL, sums, NULL, M, stream). */
int qmatmul_run_block_sums(const qmm_plan* plan, const void* w_blocks, const float* x,
                           int32_t* sums, int64_t M, void* stream);

/*
 * Mixture-of-experts layers and 4-bit group weights, on activations of any of
 * three types, for one token or a long prompt.  These calls need no plan and
 * allocate nothing: where one needs scratch memory the caller passes it (ws,
 * ws_bytes >= the matching *_workspace_bytes, 16-byte aligned; NULL when that
 * is 0), so calls with scratch of their own may overlap on different streams
 * and be captured in graphs that run side by side.  Nothing has to be kept in
 * ws between calls, and only kernels are enqueued (no memset, no host copy, no
 * synchronization); run a shape once eagerly before capturing it, as with
 * qmatmul_run.
 */

/* activation and scale types */
#define QMM_F32 0
#define QMM_F16 1
#define QMM_BF16 2

/* scores of qmatmul_route_experts */
#define QMM_SCORE_SOFTMAX 0
#define QMM_SCORE_SIGMOID 1

/* activations of qmatmul_experts_glu */
#define QMM_ACT_SILU 0
#define QMM_ACT_GELU 1 /* 0.5 v (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3))) */

/* products of qmatmul_experts_workspace_bytes */
#define QMM_EXPERTS_RUN 0
#define QMM_EXPERTS_GLU 1
#define QMM_EXPERTS_COMBINE 2
#define QMM_EXPERTS_RUN_SLOTS 3 /* qmatmul_experts_run with per_slot = 1 */

/*
 * Choose experts: per row of logits [T x E] (type QMM_F32, QMM_F16 or
 * QMM_BF16; any alignment of that type), the top_k experts and their weights.
 *   s = softmax(logits) or sigmoid(logits); choice c = s + bias (bias: device
 *   f32 [E] or NULL).  An expert whose logit is NaN or -inf has no score (0,
 *   softmax's sum is without it); one whose c is NaN or -inf, by its logit or
 *   its bias, is masked: never chosen, and no part of a group's score.  A bias
 *   takes part in the choice alone: s is the same whatever it holds.
 *   groups > 1 (a divisor of E, at most 64): experts form that many groups of
 *   neighbours; a group's score is the sum of its group_top (1 or 2) largest
 *   c; only the top_groups best groups (ties: the lower index) stay.
 *   ids [T x top_k]: the remaining experts by descending c, ties to the lower
 *   index; -1 in the slots for which no expert is left.
 *   weights [T x top_k]: s of the chosen experts (without the bias), divided
 *   by their sum if renormalize (0 if that sum is 0), times scale; 0 where the
 *   id is -1.
 * Scores, sums and comparisons are carried in 64 bits; weights are rounded
 * once, to f32.  1 <= top_k <= 64, top_k <= E <= 1024, 0 <= T <= 2^24.  A +inf logit
 * gives softmax its limit: the +inf experts share the whole weight.  ids and
 * weights must not overlap the inputs or each other (QMM_EINVAL).
 */
int qmatmul_route_experts(const void* logits, int type, int64_t T, int64_t E, const float* bias, int score,
                          int top_k, int groups, int top_groups, int group_top, int renormalize, float scale,
                          int32_t* ids, float* weights, void* stream);

/*
 * Products with the weights of chosen experts.  w holds E matrices one after
 * another, each N x K in GGUF blocks as qmatmul_run takes them (E * N *
 * qmatmul_row_bytes(format, K) bytes, 16-byte aligned); ids: device int32
 * [T x top_k]; an id outside 0..E-1 means no expert; the same id may come
 * twice in a row.  x, h and y have the type `type`; x and h 16-byte aligned.
 * Activations are not quantized (mode (a)): f16 ones enter as they are, bf16
 * and f32 ones to 2^-22 of themselves, 2^-39 of the largest magnitude in their
 * row or 2^-151, whichever is most.  Products are summed in f32 and each output is
 * rounded once, to `type`.
 *
 * qmatmul_experts_run: y[t][s] = x[t] . W[ids[t][s]]^T, y [T x top_k x N];
 *   per_slot = 0: x [T x K], one row for a token's slots; per_slot = 1:
 *   x [T x top_k x K].  Slots without an expert give zeros.
 * qmatmul_experts_glu: h[t][s] = act(x[t] . Wg^T) * (x[t] . Wu^T) for the
 *   slot's expert, h [T x top_k x N]; no expert: zeros.
 * qmatmul_experts_combine: y[t] = sum_s weights[t][s] * (h[t][s] .
 *   W[ids[t][s]]^T), y [T x N], h [T x top_k x K], weights device f32
 *   [T x top_k]; slots without an expert add nothing, whatever their h and
 *   weight hold.
 *
 * A row of x with an infinity or NaN makes all the outputs computed from it
 * non-finite (infinite or NaN) and no others.
 * Limits: E <= 1024, top_k <= 64, T * top_k <= 2^24, N <= 2^24, and
 * qmatmul_create's limit on K; QMM_EINVAL ("shape too large") also where a
 * launch would need 2^32 threads (2^22 rows with K > 8192, or 2^23 tiles of
 * outputs).  T == 0 enqueues nothing.  Outputs and ws must not overlap inputs or
 * each other (QMM_EINVAL).
 */
int64_t qmatmul_experts_workspace_bytes(int product, int format, int64_t E, int64_t N, int64_t K, int64_t T,
                                        int64_t top_k, int type); /* -1 if invalid */
int qmatmul_experts_run(int format, int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, int type, int per_slot,
                        const void* w, const void* x, const int32_t* ids, void* y, void* ws, size_t ws_bytes,
                        void* stream);
int qmatmul_experts_glu(int format, int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, int type, int act,
                        const void* w_gate, const void* w_up, const void* x, const int32_t* ids, void* h, void* ws,
                        size_t ws_bytes, void* stream);
int qmatmul_experts_combine(int format, int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, int type,
                            const void* w, const void* h, const int32_t* ids, const float* weights, void* y, void* ws,
                            size_t ws_bytes, void* stream);

/*
 * y [M x N] = x [M x K] . W^T with W in 4-bit codes and one scale (and zero
 * point) per group of `group` values of a row:
 *   W[n][k] = scales[n][k / group] * (q[n][k] - z), z = zeros[n][k / group]
 *   or, zeros == NULL, 8.
 * q: device, N x K/2 bytes, element 2i in the low nibble of byte i and 2i + 1
 * in its high nibble, 16-byte aligned.  scales: device [N x K/group] of
 * scale_type (QMM_F32, QMM_F16 or QMM_BF16).  zeros: device uint8 [N x
 * K/group], 0..15 (other values are used as they are).  Scales may have any
 * finite size; those below 2^-83 enter to 2^-107.  group: a multiple of
 * 32 that divides K; N and M at most 2^24, K at most 2^20, N * K / 2 at most
 * 2^40.  x (16-byte aligned) and y have the type `type`.  M >= 0; M == 0
 * enqueues nothing.  Sums, rounding, non-finite rows, the limit on a launch and
 * overlaps as with qmatmul_experts_run.
 */
int64_t qmatmul_w4_workspace_bytes(int64_t N, int64_t K, int64_t M, int64_t group, int type); /* -1 if invalid */
int qmatmul_w4_run(int64_t N, int64_t K, int64_t M, int64_t group, int type, int scale_type, const void* q,
                   const void* scales, const uint8_t* zeros, const void* x, void* y, void* ws, size_t ws_bytes,
                   void* stream);

/*
 * Keys and values in a quantized paged cache, and attention over it: what lies
 * between a layer's q/k/v products and its output product in a server.  Like
 * the experts' calls these need no plan, allocate nothing and only enqueue
 * kernels.
 *
 * A cache is `pages` pages of page_size tokens; a page holds, for each of
 * `heads` heads, page_size rows of `dim` values in Q8_0 or Q4_0 blocks (32
 * values of a token and head): pages * heads * page_size *
 * qmatmul_row_bytes(format, dim) bytes for the keys (k, format_k) and as much
 * in format_v for the values (v).  Codes and scales are those that
 * qmatmul_quantize_act (Q8_0) and qmatmul_quantize_weights (Q4_0) give for the
 * row, with two exceptions: a block whose scale rounds to 0 has the codes of 0,
 * and a block that holds an infinity or a NaN, or whose scale is beyond f16,
 * reads back as NaN throughout.  Their order within a page is the one in which
 * the kernels read them; for 64 neighbouring tokens t (t = 32 s + 16 h + 4 g + i
 * = 16 u + r) of a head, together 64 * row bytes:
 *   keys: four tiles u of 64 lanes 16 c + r; a lane holds, for each block b, the
 *     codes of dimensions 32 b + 8 c + (0..7), cut into pieces of 16 bytes and a
 *     rest, each piece stored for the 64 lanes in turn;
 *   values: for each block b 64 lanes 16 g + n; a lane holds the codes of
 *     dimensions 32 b + n and 32 b + 16 + n (p = 0, 1) of 16 tokens in the order
 *     8 s + 4 h + i; Q8_0 [p][lane][16 bytes], Q4_0 [lane][p][8 bytes];
 *   codes: Q8_0 a byte q + 128; Q4_0 the 4 bits of q + 8, of eight in order
 *     number e in nibble e / 2 + 4 * (e % 2) of a 32-bit word;
 *   then f16 scales [dim / 32][64], token t at place 16 g + 8 s + 4 h + i.
 *
 * A batch names its sequences' tokens: sequence s has lengths[s] tokens in the
 * cache, the last starts[s + 1] - starts[s] of which are the call's; row
 * starts[s] + i of the call's tensors is its token at position lengths[s] -
 * (starts[s + 1] - starts[s]) + i.  starts must not decrease; rows before
 * starts[0] and from starts[batch] on belong to no sequence and are neither
 * read nor written, and neither are those of a sequence that has rows outside
 * 0..T - 1.  Position p lies in page table[s][p / page_size].  A
 * position without a page (negative, past the table, or where the entry is not
 * in 0..pages - 1) holds nothing: it is not stored, reads back as zeros, and
 * attention does not see it.
 */
typedef struct qmm_cache {
    int format_k, format_v;    /* QMM_Q8_0 or QMM_Q4_0 each */
    int64_t pages, page_size;  /* page_size: a multiple of 64, at most 8192 */
    int64_t heads, dim;        /* dim: 64, 96, 128 or 256 */
    void* k;                   /* device, 16-byte aligned; NULL is fine for 0 pages */
    void* v;
    int64_t batch, table_width; /* batch <= 2^20, batch * heads <= 2^21, table_width * page_size < 2^31 */
    const int32_t* table;      /* device [batch][table_width]; NULL is fine for 0 columns */
    const int32_t* starts;     /* device [batch + 1] */
    const int32_t* lengths;    /* device [batch] */
} qmm_cache;

/*
 * qmatmul_cache_store: the call's T rows of keys and values (device, `type`
 * QMM_F32, QMM_F16 or QMM_BF16, [T][heads][dim] with k_stride and v_stride
 * values from token to token) into the cache.  Bytes of other tokens keep their
 * values.  Where two sequences of a call write into the same 64 neighbouring
 * tokens of a page, each of those 64 holds codes of either or what it held.
 * qmatmul_cache_load: the rows read back, contiguous [T][heads][dim] of `type`,
 * each value rounded once; with lengths = starts[s + 1] - starts[s] these are
 * whole sequences.
 */
int qmatmul_cache_store(const qmm_cache* cache, int64_t T, int type, const void* k, int64_t k_stride, const void* v,
                        int64_t v_stride, void* stream);
int qmatmul_cache_load(const qmm_cache* cache, int64_t T, int type, void* k, void* v, void* stream);

/*
 * qmatmul_cache_attention: out[n][h] = sum_j p_j v_j, p = softmax over the
 * positions j that row n sees of c(scale * q[n][h] . k_j); query heads h to one
 * head of the cache: h / (q_heads / heads).  Row n at position p sees 0 <= j <
 * lengths[s]; causal: j <= p; window > 0 (causal only): j > p - window.  c is
 * the identity, or softcap * tanh(x / softcap) where softcap > 0 (to 2^-20 of x,
 * whatever the cap's size).  q: device
 * `type` [T][q_heads][dim], q_stride values from token to token; out: the same
 * type, contiguous.  lse: device f32 [T][q_heads] or NULL: ln of the sum of
 * exp(score), by which results over parts of a sequence can be joined.  A row
 * that sees nothing has out 0 and lse -inf.
 * Scores and sums are f32; q enters as f16 parts (f32 as two: 2^-22 of the
 * row's largest), and codes are exact.  Probabilities times value scales enter
 * as f16 (f32: as two parts), off by at most 2^-37 of the largest value in the
 * cache per position beside their rounding; where f16 or bf16 rows are many
 * (some hundred, with work for the whole card) values are rounded to f16 and
 * probabilities to f16 (f16 rows: as two parts), for bf16 rows also keys, and
 * that end of f16 lies at 2^-30.  Outputs of f16 rows are off by 2.6e-4 of their
 * size where rows are few and 2.2e-4 where they are many, 2.1e-4 of it their own
 * rounding; of bf16 rows by 1.67e-3 and 1.72e-3 (1.66e-3).  Which of both a call
 * takes and how its sums are cut depends on its sizes, so that a row's last bits
 * can differ between batches; the same call gives the same bits again.
 * A NaN or infinity in q, or a NaN in a key that a row sees, makes that row NaN;
 * a NaN in a value that a row sees makes the dimensions of its block NaN; what
 * a row does not see does not touch it.
 * max_length: at least the largest of lengths where the caller knows it (0:
 * table_width * page_size); it goes into how the work is split and the size of
 * the workspace; results are right also for longer sequences.  Work is split by
 * this bound and by the batch's average rows, not by each length: one token over
 * 4096 positions takes 13 us with the bound 4096 and 25 us with a table of 131072
 * and no bound, and a long sequence among many short ones, or a prompt among
 * single tokens, takes longer than in a call of its own.
 * Limits: q_heads a multiple of heads, at most 1024; T <= 2^24, T * q_heads <=
 * 2^25.  Outputs and ws must not overlap inputs or each other (QMM_EINVAL).
 */
int64_t qmatmul_cache_attention_workspace_bytes(const qmm_cache* cache, int64_t T, int64_t q_heads, int type, int causal,
                                                int64_t window, int64_t max_length); /* reads no pointer; -1 if invalid */
int qmatmul_cache_attention(const qmm_cache* cache, int64_t T, int64_t q_heads, int type, const void* q, int64_t q_stride,
                            float scale, int causal, int64_t window, float softcap, int64_t max_length, void* out,
                            float* lse, void* ws, size_t ws_bytes, void* stream);

/* Host-only helpers (no HIP calls; safe without a GPU). */
int qmatmul_check(int format, int64_t N, int64_t K, int64_t M_max, int mode); /* what create validates */
int64_t qmatmul_row_bytes(int format, int64_t K);           /* bytes of one row of blocks, -1 if invalid */
int64_t qmatmul_block_sums_per_row(int format, int64_t K);  /* int32 entries per (m, n), -1 if invalid */
int64_t qmatmul_workspace_bytes(int format, int64_t N, int64_t K, int64_t M_max, int mode); /* -1 if invalid */
const char* qmatmul_status_string(int status);
const char* qmatmul_last_error(void); /* message of the calling thread's last failure, "" if none */
int qmatmul_version(void);

#ifdef __cplusplus
}
#endif
#endif /* QMATMUL_H */
