/*
 * fo.h -- C ABI of the GB300 fused compressed-optimizer library (libfo.so).
 *
 * The library implements the optimizer step of "FlashOptim: Optimizers for
 * Memory Efficient Training" (Gonzalez Ortiz et al., arXiv 2602.23349v1):
 *
 *   - weight splitting (page section "权重复分裂", Eq. 1-2, Algorithm 1): the
 *     FP32 master weight theta is held as a BF16 weight theta' plus a b-bit
 *     integer correction rho, the rounding error normalised by ULP(theta')/2;
 *   - companded state quantization (section "带压缩扩展的优化器状态量化",
 *     Algorithms 2-3): momentum m as INT8 codes of phi_m(m) = 2m/(1+|m|),
 *     second moment v as UINT8 codes of phi_v(v) = sqrt(v), in groups of 32
 *     elements with one FP16 scale per group;
 *   - the fused step (section "融合优化器步骤", Algorithm 4): dequantize m
 *     and v, rebuild theta, apply the standard AdamW / SGD / Lion update,
 *     requantize m and v and re-split theta, in one pass over memory;
 *
 * the losses on a language model's logits whose gradients that step consumes,
 * and operators whose activations are kept for the backward pass in 8 bits (last
 * two sections, with rules of their own on accuracy and alignment).
 *
 * Exact arithmetic contract of the step and its codecs (bit for bit):
 *   theta' = BF16(theta), round to nearest even.
 *   h      = half the BF16 gap between theta' and its neighbour on theta's
 *            side (the usual ULP/2, halved again just below a power of two).
 *   rho    = rint(((theta - theta') / h) * Q), Q = 127 (8-bit) or 32767
 *            (16-bit); FP32 product, round half to even.
 *   theta^ = fma(rho * kappa, h, theta'), kappa = 1/Q rounded to FP32.
 *   group scale s = FP16(max |phi(x)|) (round to nearest even, capped at
 *            65504); code = clamp(rint(phi(x) * (L / s)), ...), L = 127 for m
 *            (codes -127..127) and 255 for v (codes 0..255); s = 0 gives codes 0.
 *   decode: m = z / (2 - |z|), z = code * (s / 127);  v = r * r, r = code * (s / 255).
 *   AdamW:  theta *= (1 - lr*wd); m = fma(b1, m, (1-b1)*g);
 *           v = fma(b2, v, ((1-b2)*g)*g);
 *           theta = fma(-lr/bc1, m / fma(sqrt(v), 1/sqrt(bc2), eps), theta),
 *           bc_i = 1 - b_i^t (t >= 1), b^t by repeated squaring in double.
 *   SGD:    m = fma(mu, m, fma(wd, theta, g)); theta = fma(-lr, m, theta).
 *   Lion:   c = fma(b1, m, (1-b1)*g); theta = fma(-lr, sign(c), theta*(1-lr*wd));
 *           m = fma(b2, m, (1-b2)*g).
 *   g is the row's gradient as FP32 (a BF16 gradient widened exactly).
 *   All arithmetic is IEEE binary32 round-to-nearest-even without flush to
 *   zero. Hyper-parameters are doubles; each per-element scalar is the
 *   hyper-parameter, or a quantity formed from them in double, rounded to FP32.
 *   The contract holds for finite inputs with |theta| below the largest BF16;
 *   NaN and infinity propagate into unspecified codes without a trap.
 *
 * Memory and ownership: every array argument is DEVICE memory owned by the
 * caller (for example torch tensors' data pointers). The library allocates no
 * device memory. Tables and hyper-parameter structs are HOST memory, read
 * only during the call (the table is copied into kernel parameters before the
 * call returns). To check a table for overlapping arrays, a step call sorts
 * the table's address ranges in a per-thread host array (16 bytes per array
 * of the largest table seen), kept until the thread exits; nothing else
 * persists between calls.
 *
 * Layout of the step and its codecs: element arrays are contiguous, one element
 * per entry; each array must start on a 16-byte boundary. Scale arrays hold ceil(numel/32) FP16
 * values (any 2-byte alignment); group k covers elements [32k, 32k+32) of its
 * tensor and the last group of a tensor may be partial.
 *
 * Streams and errors: all work is enqueued on `stream` (a cudaStream_t; NULL
 * is the legacy default stream) of the CURRENT device, and the calls return
 * without synchronizing. Argument errors are detected on the host before
 * anything is launched and return a non-zero fo_status_t. A CUDA error left
 * pending by earlier, unrelated work is read (and so cleared) before the
 * first launch and returned as FO_ERR_CUDA with nothing launched; a launch
 * that fails returns FO_ERR_CUDA (fo_last_cuda_error gives the cudaError_t).
 * A step table can need several launches (one per correction width and
 * gradient type, and per 384 rows): if one of them fails, the launches
 * before it stay enqueued, so the rows they cover are stepped and the others
 * are not -- do not simply retry such a call. Faults that happen later
 * surface at the caller's next synchronization. Nothing is thrown across the
 * ABI. Calls on distinct streams over disjoint buffers are independent and
 * thread-safe. State buffers are updated in place: an array that a call
 * writes may share no byte with any other array of the call (FO_ERR_ALIAS),
 * in the same table row or another; gradients are only read, so rows may
 * share one gradient array.
 */
#ifndef FO_H
#define FO_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. FO_OK is 0; every error is non-zero. */
typedef enum fo_status {
    FO_OK = 0,
    FO_ERR_NULL = 1,             /* a required pointer is NULL                  */
    FO_ERR_MISALIGNED = 2,       /* an element array is not 16-byte aligned     */
    FO_ERR_SIZE = 3,             /* a count is negative or too large            */
    FO_ERR_BAD_ARG = 4,          /* a flag or hyper-parameter is out of range   */
    FO_ERR_TOO_MANY_TENSORS = 5, /* ntensors exceeds FO_MAX_TENSORS             */
    FO_ERR_CUDA = 6,             /* a CUDA call failed (see fo_last_cuda_error) */
    FO_ERR_ALIAS = 7             /* a written array overlaps another array      */
} fo_status_t;

/* Kind of optimizer state coded by fo_quant_state / fo_dequant_state. */
typedef enum fo_state_kind {
    FO_STATE_MOMENTUM = 0,        /* INT8 codes (int8_t), phi_m companding   */
    FO_STATE_VARIANCE = 1,        /* UINT8 codes (uint8_t), phi_v companding */
    /* The same group quantization with phi the identity: the plain linear
     * quantizer that section "实验结果分析" (Fig. 4, Fig. 5) compares the
     * companded codecs against. For quality studies; the step never uses it. */
    FO_STATE_MOMENTUM_LINEAR = 2, /* INT8 codes of m itself                  */
    FO_STATE_VARIANCE_LINEAR = 3, /* UINT8 codes of v itself                 */
    /* FO_STATE_VARIANCE with an opt-in safety rule that the page does not
     * have (its Algorithm 3 "numerical stability" step is unprinted): in a
     * group with a non-zero scale s the codes are max(rint(.), 1), so every
     * decoded v there is at least (s/255)^2 and none is 0. A group whose
     * largest sqrt(v) rounds to an FP16 scale of 0 still stores codes 0.
     * Decoding is FO_STATE_VARIANCE's. */
    FO_STATE_VARIANCE_NONZERO = 5
} fo_state_kind_t;

#define FO_GROUP 32               /* elements per quantization group            */
#define FO_MAX_TENSORS (1 << 20)  /* rows per step call (split into launches)   */

/* A cudaStream_t passed through the ABI without CUDA headers. */
typedef void *fo_stream_t;

/*
 * Element type of a row's gradient. BF16 is the page's setting (the fused
 * step reads 2 bytes of gradient per parameter). FP32 serves callers whose
 * gradients are FP32 (for example accumulated in FP32): the FP32 value enters
 * the FP32 update as it is, with no rounding to BF16 first, at 2 more bytes
 * of reads per parameter.
 */
typedef enum fo_grad_dtype {
    FO_GRAD_BF16 = 0, /* grad holds uint16_t BF16 bit patterns */
    FO_GRAD_F32 = 1   /* grad holds float                      */
} fo_grad_dtype_t;

/*
 * One row of the multi-tensor parameter table: the compressed state of one
 * tensor of numel elements. All pointers are device memory.
 */
typedef struct fo_tensor {
    uint16_t *theta;       /* theta': BF16 bit patterns, numel, in/out                 */
    void *rho;             /* rho: int8_t (rho_bits 8) or int16_t (16), numel, in/out  */
    int8_t *m_q;           /* momentum codes, numel, in/out                            */
    uint16_t *m_scale;     /* FP16 momentum scales, ceil(numel/32), in/out             */
    uint8_t *v_q;          /* second-moment codes, numel, in/out (AdamW; else NULL)     */
    uint16_t *v_scale;     /* FP16 second-moment scales (AdamW; else NULL)              */
    const void *grad;      /* gradient, numel, read only; element type per grad_dtype  */
    int64_t numel;         /* elements; 0 skips the row                                */
    double weight_decay;   /* this tensor's weight decay (0 disables it)               */
    int32_t rho_bits;      /* 8 or 16                                                  */
    int32_t grad_dtype;    /* fo_grad_dtype_t: FO_GRAD_BF16 (0) or FO_GRAD_F32 (1)     */
} fo_tensor_t;

/* AdamW: lr > 0 finite, 0 <= beta < 1, eps > 0 (weight decay is per row).
 * flags: 0, or FO_ADAMW_V_NONZERO to requantize v with the rule of
 * FO_STATE_VARIANCE_NONZERO. Without it, an element whose sqrt(v) falls below
 * 1/510 of its group's scale decodes to v = 0, and the next step divides its
 * momentum by little more than its newest gradient's share of v (or by eps).
 * reserved must be 0. */
#define FO_ADAMW_V_NONZERO 1u
typedef struct fo_adamw_hparams {
    double lr, beta1, beta2, eps;
    uint32_t flags;
    uint32_t reserved;
} fo_adamw_hparams_t;
/* SGD with momentum, dampening 0, no Nesterov, L2 weight decay added to grad. */
typedef struct fo_sgd_hparams { double lr, momentum; } fo_sgd_hparams_t;
/* Lion (Chen et al. 2023) with decoupled weight decay. */
typedef struct fo_lion_hparams { double lr, beta1, beta2; } fo_lion_hparams_t;

/*
 * fo_split -- weight splitting, section "权重复分裂" (Eq. 1-2): from FP32
 * weights theta_f32[n] write theta'[n] (BF16) and rho[n] (int8_t or int16_t
 * per rho_bits). Used to initialise the compressed weights.
 * Errors: FO_ERR_NULL, FO_ERR_MISALIGNED, FO_ERR_SIZE (n < 0 or n > 2^46),
 * FO_ERR_BAD_ARG (rho_bits not 8 or 16), FO_ERR_ALIAS (an output overlaps
 * another array), FO_ERR_CUDA. n = 0 is a no-op.
 */
fo_status_t fo_split(const float *theta_f32, uint16_t *theta_bf16, void *rho, int64_t n,
                     int32_t rho_bits, fo_stream_t stream);

/*
 * fo_merge -- the inverse of fo_split, section "权重复分裂": rebuild
 * theta^[n] (FP32) from theta'[n] and rho[n]. Used to export FP32 weights.
 * Errors as fo_split.
 */
fo_status_t fo_merge(const uint16_t *theta_bf16, const void *rho, float *theta_f32, int64_t n,
                     int32_t rho_bits, fo_stream_t stream);

/*
 * fo_quant_state -- companded group quantization, section
 * "带压缩扩展的优化器状态量化" (Algorithm 2 for m, Algorithm 3 for v):
 * x[n] (FP32; v must be >= 0) -> codes q[n] (int8_t for the momentum kinds,
 * uint8_t for the variance kinds) and scales[ceil(n/32)] (FP16).
 * Errors: FO_ERR_NULL, FO_ERR_MISALIGNED, FO_ERR_SIZE (n < 0 or n > 2^46),
 * FO_ERR_BAD_ARG (kind), FO_ERR_ALIAS (an output overlaps another array),
 * FO_ERR_CUDA. n = 0 is a no-op.
 */
fo_status_t fo_quant_state(const float *x, void *q, uint16_t *scales, int64_t n,
                           fo_state_kind_t kind, fo_stream_t stream);

/*
 * fo_dequant_state -- the inverse of fo_quant_state (same section): codes and
 * scales -> x[n] (FP32). Errors as fo_quant_state.
 */
fo_status_t fo_dequant_state(const void *q, const uint16_t *scales, float *x, int64_t n,
                             fo_state_kind_t kind, fo_stream_t stream);

/*
 * fo_adamw_step -- one fused FlashAdamW step, section "融合优化器步骤"
 * (Algorithm 4), over `ntensors` rows of `table` (host array), step counter
 * `step` = t >= 1 (owned by the caller; it is the only state outside the
 * buffers, so a checkpoint is the buffers plus t). Every row needs theta, rho,
 * m_q, m_scale, v_q, v_scale and grad. Each byte of the state crosses device
 * memory once per call.
 * Errors: FO_ERR_NULL, FO_ERR_MISALIGNED, FO_ERR_SIZE (numel < 0, step < 1,
 * ntensors < 0), FO_ERR_TOO_MANY_TENSORS, FO_ERR_BAD_ARG (rho_bits,
 * grad_dtype, non-finite or out-of-range hyper-parameters), FO_ERR_ALIAS,
 * FO_ERR_CUDA. ntensors = 0 is a no-op. Rows of both correction widths and
 * both gradient types may be mixed in one table (one launch per combination
 * present).
 */
fo_status_t fo_adamw_step(const fo_tensor_t *table, int32_t ntensors,
                          const fo_adamw_hparams_t *hp, int64_t step, fo_stream_t stream);

/*
 * fo_adamw_step_dev -- fo_adamw_step with the step counter t read from
 * DEVICE memory when the kernel runs: step_dev points to one int64_t
 * (8-byte aligned, caller-owned) on the current device. The bias corrections
 * and the other step-dependent scalars are then derived on the device, with
 * the same double-precision expressions as fo_adamw_step, so the two calls
 * give identical results for the same t. This serves steps captured in a
 * CUDA graph: a replay reads the counter's value at that moment, where
 * fo_adamw_step would repeat the t it was captured with. The call does not
 * advance the counter; the caller does (for example with an increment
 * enqueued, or captured, before the call). If the counter holds a value below
 * 1 when the kernel runs, the launch updates nothing.
 * Errors: those of fo_adamw_step (without the step check), FO_ERR_NULL
 * (step_dev), FO_ERR_MISALIGNED (step_dev not 8-byte aligned).
 */
fo_status_t fo_adamw_step_dev(const fo_tensor_t *table, int32_t ntensors,
                              const fo_adamw_hparams_t *hp, const int64_t *step_dev,
                              fo_stream_t stream);

/*
 * fo_sgd_step -- one fused FlashSGD step (SGD with momentum and the same
 * compression; pages' sections "论文背景和研究动机" and "融合优化器步骤").
 * Rows need theta, rho, m_q, m_scale, grad; v_q and v_scale are ignored.
 * Errors as fo_adamw_step (without the step counter).
 */
fo_status_t fo_sgd_step(const fo_tensor_t *table, int32_t ntensors, const fo_sgd_hparams_t *hp,
                        fo_stream_t stream);

/*
 * fo_lion_step -- one fused FlashLion step (Lion with the same compression;
 * same sections). Rows need theta, rho, m_q, m_scale, grad; v_q and v_scale
 * are ignored. Errors as fo_sgd_step.
 */
fo_status_t fo_lion_step(const fo_tensor_t *table, int32_t ntensors,
                         const fo_lion_hparams_t *hp, fo_stream_t stream);

/*
 * fo_verify_fast_arithmetic -- the fused step (section "融合优化器步骤")
 * must leave exactly the state the IEEE operations of the contract above
 * give. Its fast path builds division and square root from the GPU's
 * reciprocal and reciprocal-square-root approximations, whose exact results
 * the instruction set leaves open; each sequence is exact on a one-variable
 * or finite operand domain given the approximation's behaviour. This call
 * enumerates every such domain on the CURRENT device, running the step's own
 * device functions, and counts the operands whose result differs from the
 * IEEE operation (both signs where the domain is signed):
 *   counts[0]  refined reciprocal vs RN(1/b), every b in [2^-100, 2^100]
 *   counts[1]  square root vs RN(sqrt(v)), every v in [2^-100, 2^126] and 0
 *   counts[2]  phi_m division of AdamW (m scaled by 2^32), every |m'| in
 *              [2^-62, 2^85]
 *   counts[3]  phi_m division of SGD and Lion, every |m| in [2^-100, 2^100]
 *   counts[4]  momentum decoding phi_m^-1(code * s/127), every code byte
 *              under every FP16 scale below 127/64
 *   counts[5]  127/s, 255/s, s/127 and s/255, every positive finite FP16 s
 * All are 0 where the fast path is exact. `counts`: DEVICE memory of
 * FO_VERIFY_COUNTS uint64 entries (8-byte aligned) owned by the caller,
 * overwritten; the work (about 7e9 evaluations) is enqueued on `stream`.
 * Errors: FO_ERR_NULL, FO_ERR_MISALIGNED, FO_ERR_CUDA.
 */
#define FO_VERIFY_COUNTS 6
fo_status_t fo_verify_fast_arithmetic(uint64_t *counts, fo_stream_t stream);

/* --- losses on the logits of a language model ---------------------------------
 *
 * The step above consumes gradients; these calls stand at the other end of the
 * backward pass. All work on rows of logits x[vocab] at a temperature T:
 * s = x / T, m = max s, Z = sum exp(s - m), p = exp(s - m) / Z.
 *   - fo_token_logprobs: log p of given tokens, the entropy, the top
 *     alternatives (what a distillation teacher writes down), and
 *     fo_token_logprobs_grad, their gradient;
 *   - fo_distill: KL(q || p) for a teacher distribution q known by its top
 *     logits, optionally with its gradient in the same pass, and
 *     fo_distill_grad, the gradient alone;
 *   - fo_policy_loss: the clipped loss of policy training on sampled tokens,
 *     with a KL term, optionally with its gradient in the same pass, and
 *     fo_policy_loss_grad, the gradient alone.
 * Arrays need the alignment of their element type only, stats that of 16
 * bytes. Nothing here needs a workspace.
 * Accuracy: statistics and sums are FP32. An exponential of (x - m) / T is
 * within 2^-22 plus 3 roundings of its argument, relatively, and a row's sum is
 * of short chains of them; a gradient is rounded once, to the logits' type.
 * A teacher's q is within (3 |d| + 3 E|d| + 19) 2^-24, relatively, with d its
 * logit less its largest, over its temperature, and E the mean under q: where
 * its logits lie does not matter. With a tail, ln q is within two roundings of
 * its own size.
 * Every result is the same bit for bit on every run with the same arrays at
 * the same addresses modulo 16: no atomics join partial sums.
 * Rules for masked and special values, in every call:
 *   - a logit of -inf has probability 0, as has one of the type's lowest value
 *     beside ordinary ones; a row whose every logit is -inf has no
 *     distribution: log probabilities -inf, entropy 0, gradient 0 (its KL is
 *     +inf where the teacher's is not 0);
 *   - NaN, or a logit of +inf, makes the row's results NaN (top_ids are still
 *     valid: NaN counts as the largest value);
 *   - a negative token or teacher id is no entry: it adds nothing, and a
 *     negative token's log probability is 0; an id of vocab or more makes the
 *     row's results NaN;
 *   - a row whose incoming gradients (or row weight) are all 0 gets an exactly
 *     zero gradient (and loss), whatever it holds.
 */

/* Element type of logits, of their gradient and of a teacher's logits. */
typedef enum fo_logit_dtype {
    FO_LOGITS_BF16 = 0,
    FO_LOGITS_F32 = 1,
    FO_LOGITS_F16 = 2
} fo_logit_dtype_t;

#define FO_MAX_TOP_K 128              /* top alternatives and teacher ids by row        */
#define FO_MAX_ROW_BYTES (1600 * 1024) /* vocab * element size                           */
#define FO_MAX_LOGIT_ROWS (1 << 27)
#define FO_LOSS_STATS 4               /* floats of saved statistics by row              */

/*
 * Logits: `rows` rows of `vocab` contiguous elements. Row r = o * inner_rows + i
 * starts at element o * outer_stride + i * row_stride (a plain matrix has
 * inner_rows = rows; logits[:, :-1] of a [batch, time, vocab] tensor has
 * inner_rows = time - 1 and outer_stride = time * vocab). `data` needs the
 * alignment of its element type only. Strides are not negative.
 */
typedef struct fo_logits {
    const void *data;
    int64_t rows, vocab;
    int64_t row_stride;     /* elements                                   */
    int64_t inner_rows;     /* >= 1; rows is a multiple of it             */
    int64_t outer_stride;   /* elements; ignored where inner_rows == rows */
    double temperature;     /* T, in [2^-20, 2^20]                        */
    int32_t dtype;          /* fo_logit_dtype_t                           */
    int32_t reserved;       /* 0                                          */
} fo_logits_t;

/* A gradient of the logits: same rows, vocab, inner_rows and element type.
 * Its rows may not overlap one another. `data` and the strides may be those of
 * the logits themselves (the gradient then replaces them); any other overlap
 * of the two address ranges is refused. */
typedef struct fo_logits_grad {
    void *data;
    int64_t row_stride, outer_stride;
} fo_logits_grad_t;

/* A teacher's top logits: k ids and logits by row, [rows, k] contiguous. q is
 * softmax(logits / temperature) over the row's ids; with tail = 1 it is
 * q_k = exp(logits_k / temperature - lse) and the rest of the mass,
 * max(0, 1 - sum q), is one more outcome, compared with the student's
 * probability of all tokens that are not listed. Where that probability is 0
 * (below e^-746), a rest of at most 2^-16 is none: roundings leave that much
 * beside a list that holds all tokens a mask allows. A larger one counts as it
 * is, and makes KL infinite where all unlisted logits are -inf. An id listed
 * twice counts twice in q. */
typedef struct fo_teacher {
    const int32_t *ids;
    const void *logits;
    const float *lse;       /* [rows], tail only: log-sum-exp of the teacher's logits / temperature
                             * over its whole vocabulary; NULL: 0 (logits are log probabilities) */
    double temperature;     /* in [2^-20, 2^20]          */
    int32_t k;              /* 1 .. FO_MAX_TOP_K         */
    int32_t dtype;          /* fo_logit_dtype_t          */
    int32_t tail;           /* 0 or 1                    */
    int32_t reserved;       /* 0                         */
} fo_teacher_t;

/*
 * fo_token_logprobs -- by row: logp[rows] = log p[token], entropy[rows] =
 * -sum p log p, and the top_k largest logits, top_ids[rows, top_k] and
 * top_logp[rows, top_k], in descending order, equal ones by ascending id.
 * Outputs that are NULL are not computed (tokens may be NULL where logp is;
 * top_ids and top_logp are both given where top_k > 0). stats[rows,
 * FO_LOSS_STATS], optional, is what fo_token_logprobs_grad needs.
 * Errors: FO_ERR_NULL, FO_ERR_MISALIGNED (an array not aligned to its element
 * type, stats not to 16 bytes), FO_ERR_SIZE (a count is negative or above its
 * limit, vocab < 1, top_k > vocab), FO_ERR_BAD_ARG (temperature, dtype,
 * strides, reserved), FO_ERR_ALIAS, FO_ERR_CUDA. rows = 0 is a no-op.
 */
fo_status_t fo_token_logprobs(const fo_logits_t *logits, const int64_t *tokens, int32_t top_k, float *logp,
                              float *entropy, int32_t *top_ids, float *top_logp, float *stats,
                              fo_stream_t stream);

/*
 * fo_token_logprobs_grad -- the gradient of
 *   sum_r g_logp[r] logp[r] + g_entropy[r] entropy[r] + sum_k g_top[r, k] top_logp[r, k]
 * with respect to the logits, from the stats that fo_token_logprobs wrote for
 * them (the top ids count as constants). A NULL g_* is 0; tokens are needed
 * with g_logp, top_ids with g_top. Errors as fo_token_logprobs.
 */
fo_status_t fo_token_logprobs_grad(const fo_logits_t *logits, const int64_t *tokens, int32_t top_k,
                                   const int32_t *top_ids, const float *stats, const float *g_logp,
                                   const float *g_entropy, const float *g_top, const fo_logits_grad_t *grad,
                                   fo_stream_t stream);

/*
 * fo_distill -- loss[r] = w[r] KL(q_r || p_r), w = row_weight or 1 where that
 * is NULL. With `grad`, also the gradient of sum_r loss[r] with respect to the
 * logits, in the same call: the logits come from device memory once (a second
 * time from the L2 cache) and the gradient goes there once. stats
 * [rows, FO_LOSS_STATS], optional, is what fo_distill_grad needs (of rows with
 * weight 0 it is not written). `loss` and `grad` may each be NULL.
 * Errors as fo_token_logprobs.
 */
fo_status_t fo_distill(const fo_logits_t *logits, const fo_teacher_t *teacher, const float *row_weight,
                       float *loss, float *stats, const fo_logits_grad_t *grad, fo_stream_t stream);

/*
 * fo_distill_grad -- the gradient of sum_r g_loss[r] KL(q_r || p_r) with
 * respect to the logits, from the stats that fo_distill wrote for them with
 * the same teacher. Errors as fo_token_logprobs.
 */
fo_status_t fo_distill_grad(const fo_logits_t *logits, const fo_teacher_t *teacher, const float *stats,
                            const float *g_loss, const fo_logits_grad_t *grad, fo_stream_t stream);

/* Tokens that an earlier state of the policy sampled, one by row, and how the
 * loss of a row is formed. With l = log p[token], q = exp(l - old_logp), A the
 * advantage:
 *   loss = -min(q A, clip(q, 1 - clip_low, 1 + clip_high) A)
 *          + kl_weight (exp(ref_logp - l) - (ref_logp - l) - 1),
 *   dloss/dl = -A q where the minimum is taken by q A (at the border too), else 0,
 *              + kl_weight (1 - exp(ref_logp - l)).
 * A negative token is no position (padding): loss, log probability and gradient
 * are 0, and the row is not read. An advantage of 0 has no policy term, whatever
 * q is; ref_logp is read where kl_weight is not 0. A row whose dloss/dl is NaN or
 * beyond FP32 gets a gradient of NaN (of 0 where the row has no distribution). */
typedef struct fo_policy {
    const int64_t *tokens;      /* [rows]                                   */
    const float *old_logp;      /* [rows]: of the policy that sampled       */
    const float *advantages;    /* [rows]                                   */
    const float *ref_logp;      /* [rows], of a reference; may be NULL where kl_weight is 0 */
    double clip_low, clip_high; /* in [0, 1]; in [0, 2^100]                 */
    double kl_weight;           /* in [0, 2^100]                            */
} fo_policy_t;

/*
 * fo_policy_loss -- loss[r] = w[r] (the loss above), w = row_weight or 1 where
 * that is NULL, and logp[r] = log p[token]. With `grad`, also the gradient of
 * sum_r loss[r] with respect to the logits, in the same call: the logits come
 * from device memory once and the gradient goes there once. A row of weight 0 is
 * not read: its loss, logp and gradient are 0. stats[rows, FO_LOSS_STATS],
 * optional, is what fo_policy_loss_grad needs (of the unweighted loss). loss,
 * logp and grad may each be NULL. Errors as fo_token_logprobs.
 */
fo_status_t fo_policy_loss(const fo_logits_t *logits, const fo_policy_t *policy, const float *row_weight, float *loss,
                           float *logp, float *stats, const fo_logits_grad_t *grad, fo_stream_t stream);

/*
 * fo_policy_loss_grad -- the gradient of sum_r g_loss[r] loss[r] with respect to
 * the logits, from the stats that fo_policy_loss wrote for them (with no
 * row_weight, or of rows whose weight was not 0). Errors as fo_token_logprobs.
 */
fo_status_t fo_policy_loss_grad(const fo_logits_t *logits, const int64_t *tokens, const float *stats,
                                const float *g_loss, const fo_logits_grad_t *grad, fo_stream_t stream);

/* --- activations kept in 8 bits ------------------------------------------------
 *
 * What a training step keeps for its backward pass, in the manner of the
 * optimizer state: int8 codes with one BF16 step for every 32 elements of a row
 * (FO_GROUP; the last group of a row may be partial).
 *   a    = max |x| of the group
 *   step = the smallest BF16 number that is at least max(a / 127, 2^-126)
 *   code = rint(x r), half to even, r = 1 / step rounded to FP32; the product is
 *          not rounded before
 *   x^   = code * step, exact in FP32
 * so |x^ - x| is at most (1 + 2^-15) step / 2. A NaN or an infinity in a group
 * makes its step NaN, and with it all that the group stands for. As the step is
 * rounded up, x^ of a number near the largest of a 16-bit type may lie beyond that:
 * fo_expand gives the largest number then, and infinity only for an x^ more than a
 * step beyond, which stands for no number of the type.
 *
 * Matrices are rows of contiguous elements of BF16, FP16 or FP32 (fo_rows_t), all
 * of one call of one type, aligned to it. Rows that are only read may overlap;
 * rows that are written may not, and what is written shares no byte with another
 * array: from a matrix's first byte to its last, whatever lies between its rows (but
 * grad_x and grad_up below may be side by side in the rows of one matrix). For a
 * matrix of `width` columns and G = ceil(width / 32), codes is [rows, 32 G] (0
 * beyond the width, beside a step that is a number), aligned to 16 bytes, and
 * steps [rows, G]. No byte beside the rows is read or written. All arithmetic is
 * FP32, results are rounded once, to the matrices' type. Every result is the
 * same bit for bit on every run of the same call on the same kind of device.
 * What one row holds has no effect on another's results (grad_weight sums them all).
 */
typedef struct fo_rows {
    void *data;             /* only read where the call names the matrix in, up or grad_y */
    int64_t rows, width;    /* width <= FO_MAX_ACT_WIDTH, rows * ceil(width / 32) <=
                             * FO_MAX_ACT_GROUPS                                      */
    int64_t row_stride;     /* elements, not negative                                  */
    int32_t dtype;          /* fo_logit_dtype_t                                        */
    int32_t reserved;       /* 0                                                       */
} fo_rows_t;

#define FO_MAX_ACT_GROUPS (1 << 29)
#define FO_MAX_ACT_WIDTH (1 << 30)

/* Activation functions. */
typedef enum fo_act {
    FO_ACT_SILU = 0,        /* x / (1 + e^-x)                               */
    FO_ACT_GELU = 1         /* x Phi(x), Phi the normal distribution's      */
} fo_act_t;

/*
 * fo_compress -- codes and steps of x. fo_expand -- x^, rounded to x's type (that
 * of the compressed matrix or another), into x.
 * Errors of every call of this section: FO_ERR_NULL, FO_ERR_MISALIGNED,
 * FO_ERR_SIZE (rows < 0, width < 1, too many groups, a span beyond 2^58 elements), FO_ERR_BAD_ARG (dtype,
 * stride, reserved, matrices of unlike sizes or types, eps), FO_ERR_ALIAS,
 * FO_ERR_CUDA. rows = 0 is a no-op.
 */
fo_status_t fo_compress(const fo_rows_t *in, int8_t *codes, uint16_t *steps, fo_stream_t stream);
fo_status_t fo_expand(const int8_t *codes, const uint16_t *steps, const fo_rows_t *x, fo_stream_t stream);

/*
 * fo_activation -- y = f(x), or y = f(x) up where `up` is not NULL (a gated MLP:
 * x the gate), and, where codes is not NULL, the codes of x and of up. The
 * function is taken of x itself, not of its code.
 * fo_activation_grad -- from the codes: grad_x = grad_y f'(x^) (times up^), and
 * grad_up = grad_y f(x^). grad_up, up_codes and up_steps are NULL without `up`.
 * x and up may be the halves of one matrix, and so may grad_x and grad_up.
 */
fo_status_t fo_activation(fo_act_t kind, const fo_rows_t *in, const fo_rows_t *up, const fo_rows_t *y, int8_t *codes,
                          uint16_t *steps, int8_t *up_codes, uint16_t *up_steps, fo_stream_t stream);
fo_status_t fo_activation_grad(fo_act_t kind, const int8_t *codes, const uint16_t *steps, const int8_t *up_codes,
                               const uint16_t *up_steps, const fo_rows_t *grad_y, const fo_rows_t *grad_x,
                               const fo_rows_t *grad_up, fo_stream_t stream);

/*
 * fo_rms_norm -- y = x r weight, r = 1 / sqrt(mean x^2 + eps) over a row; weight
 * [width] of weight_dtype (fo_logit_dtype_t), NULL: 1. eps in [2^-80, 2^20].
 * Where codes is not NULL: the codes of x and inv_rms[rows] = r. A row with a NaN
 * or an infinity gives NaN.
 * fo_rms_norm_grad -- from the codes, with h = x^ r (r as it was):
 *   grad_x = r (grad_y w - h mean(grad_y w h)),  grad_weight = sum over rows of grad_y h.
 * grad_x or grad_weight may be NULL. workspace: FP32, aligned to 16 bytes,
 * fo_rms_norm_workspace(rows, width) elements (NULL without grad_weight); its
 * contents are of no use after the call. Calls that may run at the same time need
 * one each. With rows = 0, grad_weight is 0.
 */
fo_status_t fo_rms_norm(const fo_rows_t *in, const void *weight, int32_t weight_dtype, double eps, const fo_rows_t *y,
                        float *inv_rms, int8_t *codes, uint16_t *steps, fo_stream_t stream);
int64_t fo_rms_norm_workspace(int64_t rows, int64_t width);
fo_status_t fo_rms_norm_grad(const int8_t *codes, const uint16_t *steps, const float *inv_rms, const void *weight,
                             int32_t weight_dtype, const fo_rows_t *grad_y, const fo_rows_t *grad_x, void *grad_weight,
                             float *workspace, fo_stream_t stream);

/* A static, human-readable name for a status code (never NULL). */
const char *fo_status_string(fo_status_t status);

/* The cudaError_t (as int) behind the last FO_ERR_CUDA on this thread, or 0. */
int fo_last_cuda_error(void);

/*
 * Launch accounting for measurements: the number of kernels this library has
 * launched in the calling process so far (all threads).
 */
uint64_t fo_kernel_launch_count(void);

#ifdef __cplusplus
}
#endif
#endif /* FO_H */
