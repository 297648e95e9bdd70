/*
 * loco.h - C ABI of the MI355X (gfx950) library for LoCo's per-GPU gradient path.
 *
 * Sources of the operations (page title, section and equation):
 *   "LoCo: Low-Bit Communication Adaptor for Large-scale Model Training"
 *   (arXiv 2407.04480): Sec. 3.1 Eqns. (1)-(3) compensate and compress,
 *   Sec. 3.2 Eqns. (4)-(5) the moving-average compression error,
 *   Sec. 3.3 Eqn. (8) the all2all partitions and their high-precision average,
 *   Sec. 4 Eqn. (9) the Adam-family step that consumes the average.
 *   "Communication Efficient LLM Pre-training with SparseLoCo" (summary and
 *   abstract): Top-k sparsification, 2-bit codes and error feedback, and the sparse
 *   aggregation of the nodes' sparse updates.
 *
 * The pages hand the method a flattened gradient (the FSDP communication hook) and
 * keep the error local to each node; the exchange between nodes is not part of this
 * library.  A rank calls loco_compensate_quantize on its flat gradient, split into
 * one segment per destination partition, sends each partition's payload
 * (codes + absmax) to its owner, and calls loco_dequant_reduce on the payloads it
 * receives.  loco_topk_quantize is the SparseLoCo-style mode and loco_sparse_aggregate
 * its receiving side.
 *
 * Conventions shared by every entry point
 *   - Device pointers are caller-owned device memory (e.g. PyTorch tensors) and must
 *     be 16-byte aligned; host arrays (segs, peers) are read during the call only.
 *   - The library allocates nothing and keeps no state between calls, apart from the
 *     compute-unit count of each device, read once and cached.  Every call is
 *     asynchronous on `stream` (a hipStream_t; NULL is the default stream) and runs on
 *     the calling thread's current device; buffers must stay alive until the stream has
 *     consumed them.
 *   - Arguments are validated on the host before anything is launched: a validation
 *     status (LOCO_ERR_INVALID, LOCO_ERR_ALIGN, LOCO_ERR_UNSUPPORTED) means nothing was
 *     launched and nothing was written.  LOCO_ERR_HIP means a kernel launch failed; a
 *     call that takes several launches (more than 32 segments, a short last Top-k
 *     chunk, or more chunks than one grid holds) may have enqueued the launches before
 *     it.  Device faults surface at the caller's next synchronisation, as for any HIP
 *     call.
 *   - Arithmetic: IEEE binary32, round to nearest even, no fused multiply-add, in
 *     the order stated below; bf16 stores round to nearest even.
 *   - Stateless and reentrant across host threads and streams.
 */
#ifndef LOCO_H
#define LOCO_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of gradients, errors and outputs.  LOCO_I8 is only an error type of
 * loco_compensate_quantize_ex: the paper's 8-bit error codes of a fixed scale s_e. */
typedef enum { LOCO_F32 = 0, LOCO_BF16 = 1, LOCO_I8 = 2 } loco_dtype_t;

/* Status codes: 0 ok, < 0 error (nothing launched, except as LOCO_ERR_HIP below). */
#define LOCO_OK 0
#define LOCO_ERR_INVALID (-1)     /* bad size, bits, block, k, chunk, beta, scale, dtype,
                                     peer count < 1, null pointer, or overlapping buffers */
#define LOCO_ERR_ALIGN (-2)       /* a device pointer is not aligned, to 16 bytes unless its call says otherwise */
#define LOCO_ERR_UNSUPPORTED (-3) /* valid but not built: bits not in {2,4,8}, block not
                                     in {64,128,256,512}, chunk not in
                                     {256,512,1024,2048,4096}, more than LOCO_MAX_PEERS
                                     peers */
#define LOCO_ERR_HIP (-4)         /* the HIP launch failed */

/* Largest number of peers one dequant-reduce call accepts. */
#define LOCO_MAX_PEERS 128

/*
 * One segment of a compensate-quantize call: a contiguous gradient range with its
 * own error buffer and payload.  Scale blocks restart at element 0 of every
 * segment, so each segment's payload is self-contained (one all2all partition,
 * LoCo Sec. 3.3).
 *   grad    device, n elements of grad_dtype (read)
 *   err     device, n elements of err_dtype (4, 2 or 1 bytes each), read and
 *           updated in place
 *   codes   device, ceil(n*bits/8) bytes (written); codes are two's complement,
 *           packed little end first (4 bits: element 2j in the low nibble of byte j;
 *           2 bits: element 4j+t at bits 2t of byte j); unused high bits of the last
 *           byte are 0
 *   absmax  device, ceil(n/block) floats (written): the block's max |h|; unused and
 *           may be NULL when fixed_scale > 0
 *   n       elements (>= 0; 0 is a no-op)
 * No buffer a call writes (the err, codes and absmax of any of its segments) may
 * overlap another buffer of the call; gradients are only read and may overlap each
 * other (LOCO_ERR_INVALID otherwise).
 */
typedef struct {
    const void* grad;
    void* err;
    uint8_t* codes;
    float* absmax;
    int64_t n;
} loco_cq_segment_t;

/*
 * loco_compensate_quantize - LoCo Sec. 3.1-3.2, Eqns. (1)-(5), fused in one pass.
 *
 * For every segment and every block of `block` elements (the last may be partial):
 *   h      = g + e                                  Eqn. (2), g and e widened to f32
 *   absmax = max |h| over the block
 *   step   = absmax / qmax,  inv = 1 / step         qmax = 2^(bits-1) - 1; both 0
 *                                                   when absmax == 0
 *   q      = clamp(rint(h * inv), -2^(bits-1), qmax) Eqns. (1),(3); ties to even
 *   r      = h - q * step                           Eqn. (4)
 *   e     <- beta * e + (1 - beta) * r              Eqn. (5); 1 - beta rounded to f32
 * and stores the packed q, the block absmax and the new e (bf16: round to nearest
 * even).  fixed_scale = s > 0 is Eqn. (1) as printed: inv = s and step = 1/s for
 * every element, and no absmax is written.
 *   segs        host array of nseg segments (nseg >= 0)
 *   grad_dtype  LOCO_F32 or LOCO_BF16 (all segments); err_dtype likewise
 *   bits        2, 4 or 8
 *   block       64, 128, 256 or 512 (ignored when fixed_scale > 0)
 *   beta        in [0, 1]
 *   fixed_scale 0 for per-block absmax scales, or a finite s > 0
 * g and e must be finite, and so must h = g + e; for NaN or infinite values the codes,
 * scales and error are unspecified (no fault).
 * Any number of segments is accepted (they are launched 32 at a time, in order).
 * err_dtype LOCO_I8 is refused here (LOCO_ERR_INVALID): it needs the error scale of
 * loco_compensate_quantize_ex.
 * Returns LOCO_OK or an error status.
 */
int loco_compensate_quantize(const loco_cq_segment_t* segs, int nseg,
                             loco_dtype_t grad_dtype, loco_dtype_t err_dtype,
                             int bits, int block, float beta, float fixed_scale,
                             void* stream);

/* Options of loco_compensate_quantize_ex (a host struct, read during the call). */
typedef struct {
    int bits;          /* 2, 4 or 8 */
    int block;         /* 64, 128, 256 or 512 (ignored when fixed_scale > 0) */
    float beta;        /* in [0, 1] */
    float fixed_scale; /* 0, or a finite s > 0 */
    float err_scale;   /* s_e of an 8-bit error (err_dtype LOCO_I8); ignored otherwise */
    int reset_error;   /* nonzero: this step stores e = 0 */
} loco_cq_options_t;

/*
 * loco_compensate_quantize_ex - loco_compensate_quantize plus LoCo Sec. 3.2, Eqn. (7):
 * the compensation error kept in 8 bits, and its periodic reset.
 *
 * Same segments, arithmetic and outputs as loco_compensate_quantize, with:
 *   err_dtype LOCO_I8: err holds n int8 codes e8 of the scale s_e = err_scale, which
 *     must be finite, > 0, with 256 / s_e finite.  On load e = e8 * fl(1 / s_e) (the
 *     decompressor of Eqn. (1) with the error's own scale); on store
 *     e8 <- clamp(rint(e * s_e), -128, 127), ties to even (Eqn. (7)).
 *   reset_error != 0: the codes and absmax are those of h = g + e as usual, but the
 *     stored error is 0 (Eqn. (7) resets the error every T_c steps; the caller
 *     passes reset_error on those steps).  Any err_dtype.
 * Returns LOCO_OK or an error status (LOCO_ERR_INVALID for a NULL opt).
 */
int loco_compensate_quantize_ex(const loco_cq_segment_t* segs, int nseg,
                                loco_dtype_t grad_dtype, loco_dtype_t err_dtype,
                                const loco_cq_options_t* opt, void* stream);

/* One peer's payload for a partition: what loco_compensate_quantize wrote. */
typedef struct {
    const uint8_t* codes;  /* device, ceil(n*bits/8) bytes */
    const float* absmax;   /* device, ceil(n/block) floats; may be NULL when fixed_scale > 0 */
} loco_payload_t;

/*
 * loco_dequant_reduce - LoCo Sec. 3.3, Eqn. (8): decompress and average the N peers'
 * low-bit payloads of one partition, in high precision.
 *
 * For every element i:
 *   acc = 0;  for p = 0 .. npeers-1 in order:  acc = acc + q_p[i] * step_p
 *   out[i] = acc * out_scale                      (out_scale = 1/N for the average)
 * with step_p = absmax_p[block of i] / qmax (0 for an all-zero block), or 1/s in
 * fixed-scale mode.  The accumulator lives in registers; bf16 output rounds to
 * nearest even.  Every product and sum is the IEEE fp32 result for any absmax value,
 * up to FLT_MAX and including inf and NaN (a tile whose step is 2^100 or more, or not
 * finite, takes a slower element-wise path).
 *   peers      host array of npeers payloads, 1 <= npeers <= LOCO_MAX_PEERS
 *   n          elements of the partition (>= 0; 0 is a no-op)
 *   bits       2, 4 or 8;  block  64, 128, 256 or 512 (ignored when fixed_scale > 0)
 *   fixed_scale 0, or the s the payloads were made with
 *   out_scale  finite
 *   out        device, n elements of out_dtype (written); must not overlap a payload
 *   out_dtype  LOCO_F32 or LOCO_BF16
 */
int loco_dequant_reduce(const loco_payload_t* peers, int npeers, int64_t n,
                        int bits, int block, float fixed_scale, float out_scale,
                        void* out, loco_dtype_t out_dtype, void* stream);

/* Hyper-parameters of the LoCo-Adam step (host struct, read during the call). */
typedef struct {
    float lr;     /* learning rate eta, finite */
    float beta1;  /* weight of the new gradient in m, in [0, 1] (the page's typical 0.1) */
    float beta2;  /* weight of the new squared gradient in v, in [0, 1] (typical 0.001-0.05) */
    float delta;  /* finite, > 0: added to v under the square root */
} loco_adam_t;

/*
 * loco_dequant_reduce_adam - LoCo Sec. 3.3 Eqn. (8) fused with Sec. 4 Eqn. (9): the
 * peers' payloads are averaged exactly as loco_dequant_reduce does (fp32, peer order,
 * times out_scale; never rounded to bf16), and the average g drives one Adam-family
 * step on the partition's fp32 weights and moments, in one pass:
 *   m     <- (1 - beta1) * m + beta1 * g              (1 - beta rounded to f32 first)
 *   v     <- (1 - beta2) * v + beta2 * (g * g)
 *   u      = 1 / sqrt(v + delta)                      (correctly rounded sqrt and divide)
 *   param <- param - lr * (m * u)
 * in that order of roundings, with no bias correction or weight decay (the page names
 * neither); m and v start at 0 (the caller zeroes them).  The reduced gradient is not
 * written anywhere.
 *   peers, npeers, n, bits, block, fixed_scale, out_scale: as loco_dequant_reduce
 *   adam        host pointer to the hyper-parameters
 *   param, m, v device f32[n] each, read and updated in place
 *   param_bf16  device u16[n] (written: the RNE bf16 copy of the new param), or NULL
 * None of param, m, v, param_bf16 may overlap each other or a payload.
 */
int loco_dequant_reduce_adam(const loco_payload_t* peers, int npeers, int64_t n,
                             int bits, int block, float fixed_scale, float out_scale,
                             const loco_adam_t* adam, float* param, float* m, float* v,
                             uint16_t* param_bf16, void* stream);

/*
 * loco_topk_quantize - SparseLoCo-style per-chunk Top-k with low-bit codes and error
 * feedback ("Communication Efficient LLM Pre-training with SparseLoCo").
 *
 * For every chunk c of `chunk` elements (the last may be short; it keeps
 * keff = min(k, its length)):
 *   h  = g + ef_decay * e
 *   keep the keff elements with the largest |h| (compared as the bit pattern of
 *   |h|), ties to the lower index
 *   absmax = max |h| over the kept values; step = absmax / qmax; inv = 1 / step
 *   (both 0 if absmax == 0); q = clamp(rint(h * inv), -2^(bits-1), qmax)
 *   e <- h - q * step on the kept elements, e <- h elsewhere
 *   grad     device f32[n] (read);  err  device f32[n] (read and updated in place)
 *   n        elements (>= 0; 0 is a no-op)
 *   chunk    256, 512, 1024, 2048 or 4096;  1 <= k <= chunk
 *   bits     2, 4 or 8;  ef_decay in [0, 1]
 *   idx      device u16[chunks * k]: chunk-local indices of the kept elements,
 *            ascending; unused slots 0xFFFF
 *   codes    device u8[chunks * ceil(k*bits/8)]: the kept codes in index order,
 *            packed as in loco_cq_segment_t; unused slots 0
 *   absmax   device f32[chunks]
 * where chunks = ceil(n / chunk).  No two buffers may overlap.
 */
int loco_topk_quantize(const float* grad, float* err, int64_t n, int chunk, int k,
                       int bits, float ef_decay, uint16_t* idx, uint8_t* codes,
                       float* absmax, void* stream);

/* One peer's Top-k payload of a shard: what loco_topk_quantize wrote. */
typedef struct {
    const uint16_t* idx;   /* device u16[chunks * k] */
    const uint8_t* codes;  /* device u8[chunks * ceil(k*bits/8)] */
    const float* absmax;   /* device f32[chunks] */
} loco_sparse_payload_t;

/*
 * loco_sparse_aggregate - SparseLoCo's sparse aggregation ("Communication Efficient LLM
 * Pre-training with SparseLoCo", summary and abstract) of the peers' Top-k payloads of
 * one shard into a dense output, computed as the high-precision average of LoCo
 * Sec. 3.3, Eqn. (8) over sparse vectors.
 *
 * For every element i:
 *   acc = 0;  for p = 0 .. npeers-1 in order: if peer p's chunk c = i / chunk has a
 *   used slot j with idx_p[c*k + j] == i - c*chunk:  acc = acc + q_p[c, j] * step_p[c]
 *   out[i] = acc * out_scale                      (out_scale = 1/N for the average)
 * with step_p[c] = absmax_p[c] / qmax (0 for an all-zero chunk).  A slot is used when
 * its index lies inside its chunk (the last chunk may be short); other slots, such as
 * the 0xFFFF that loco_topk_quantize writes in unused slots, are skipped.  Elements no
 * peer names are 0.  The slots of one peer's chunk must name distinct elements (as
 * loco_topk_quantize writes them); repeated ones give an unspecified sum of their
 * values but never touch memory outside the output.  The accumulator is fp32; bf16
 * output rounds to nearest even.
 *   peers      host array of npeers payloads, 1 <= npeers <= LOCO_MAX_PEERS
 *   n          elements of the shard (>= 0; 0 is a no-op)
 *   chunk      256, 512, 1024, 2048 or 4096;  1 <= k <= chunk;  bits 2, 4 or 8
 *   out_scale  finite
 *   out        device, n elements of out_dtype (written); must not overlap a payload
 *   out_dtype  LOCO_F32 or LOCO_BF16
 * where chunks = ceil(n / chunk).
 */
int loco_sparse_aggregate(const loco_sparse_payload_t* peers, int npeers, int64_t n,
                          int chunk, int k, int bits, float out_scale, void* out,
                          loco_dtype_t out_dtype, void* stream);

/* ---------------------------------------------------------------------------------
 * Layer operators: the products, norms and activation checkpoints of the layer whose
 * backward pass writes the gradient that loco_compensate_quantize takes.
 *
 * Matrices are row-major and contiguous; rows are tokens.  A call that needs scratch
 * memory takes `workspace`, device memory of at least the bytes that the matching
 * loco_*_workspace function returns for the same sizes (0: none, and workspace may be
 * NULL); its contents before and after are unspecified.  Sums, statistics and
 * accumulators are fp32 (the matrix cores' products of bf16 are exact in it); fused
 * multiply-adds are used, and sums run in an order of the library's own that depends on
 * the sizes (and, up to 16 rows of loco_linear, on whether a checkpoint is written), so the
 * same call gives the same bits.  Infinities and NaNs in the inputs follow IEEE arithmetic
 * into the outputs they reach.
 * ------------------------------------------------------------------------------ */

/* Activations a(z). */
typedef enum {
    LOCO_ACT_NONE = 0, /* z */
    LOCO_ACT_RELU = 1, /* max(z, 0) */
    LOCO_ACT_GELU = 2, /* z * sigmoid(2 sqrt(2/pi) (z + 0.044715 z^3)), the tanh form */
    LOCO_ACT_SILU = 3  /* z * sigmoid(z) */
} loco_act_t;

/*
 * An 8-bit activation checkpoint of a matrix [rows, cols].  Blocks of `block` elements
 * run along each row and restart with it (the last of a row may be short).
 *   codes  device i8[rows * cols]
 *   exps   device u8[rows * ceil(cols / block)]: the block's step is 2^(exps - 127)
 *   block  32 or 64
 * A value is codes * step.  Written, the step is the least power of two >= 2^-126 with
 * max|x| < 127.5 * step and the code is rint(x / step), ties to even: one rounding, of at
 * most half a step.  A code times a power of two has at most 7 significant bits, so
 * every value is a bf16 number and the matrix cores read it exactly.  A block that holds
 * an infinity or a NaN is written with exps 255 and codes 0; exps 255 reads as NaN where the
 * code is 0 and as an infinity elsewhere, exps 0 as 0.
 */
typedef struct {
    int8_t* codes;
    uint8_t* exps;
    int block;
} loco_checkpoint_t;

/*
 * loco_layer_norm - y = (x - mean) * rstd * weight + bias per row, with
 * mean = sum(x)/cols and rstd = 1/sqrt(sum((x - mean)^2)/cols + eps).
 *   x, y          device [rows, cols] of `dtype` (LOCO_F32 or LOCO_BF16)
 *   weight, bias  device [cols] of `param_dtype`; NULL: ones, zeros
 *   eps           finite, >= 0
 *   mean, rstd    device f32[rows] (written), for the backward pass
 *   ckpt          NULL, or the 8-bit checkpoint of y to write (of the fp32 y, before its
 *                 rounding to dtype)
 *   cols          1 .. 16384 (LOCO_ERR_UNSUPPORTED beyond); rows 0 is a no-op
 */
int loco_layer_norm(const void* x, loco_dtype_t dtype, const void* weight, const void* bias,
                    loco_dtype_t param_dtype, int64_t rows, int64_t cols, float eps, void* y,
                    float* mean, float* rstd, const loco_checkpoint_t* ckpt, void* stream);

/*
 * loco_layer_norm_backward - with xh = (x - mean) * rstd and g = dy * weight:
 *   dx      = rstd * (g - sum(g)/cols - xh * sum(g * xh)/cols) [+ residual]
 *   dweight = sum over the rows of dy * xh,  dbias = sum over the rows of dy
 *   dy, x, residual, dx  device [rows, cols] of `dtype`; residual may be NULL
 *   weight               device [cols] of `param_dtype`; NULL: ones
 *   mean, rstd           device f32[rows], as loco_layer_norm wrote them
 *   dweight, dbias       device [cols] of `grad_dtype` (written), each may be NULL;
 *                        with rows 0 they are written as zeros
 *   workspace            loco_layer_norm_backward_workspace(rows, cols) bytes; may be NULL
 *                        if dweight and dbias are
 */
int loco_layer_norm_backward(const void* dy, const void* x, loco_dtype_t dtype, const void* weight,
                             loco_dtype_t param_dtype, const float* mean, const float* rstd,
                             const void* residual, int64_t rows, int64_t cols, void* dx,
                             void* dweight, void* dbias, loco_dtype_t grad_dtype,
                             void* workspace, int64_t workspace_bytes, void* stream);
int64_t loco_layer_norm_backward_workspace(int64_t rows, int64_t cols);

/*
 * loco_checkpoint_write - the 8-bit checkpoint of x [rows, cols] of `dtype`.
 * loco_checkpoint_read  - out = act(value), [rows, cols] of `out_dtype`.
 */
int loco_checkpoint_write(const void* x, loco_dtype_t dtype, int64_t rows, int64_t cols,
                          const loco_checkpoint_t* ckpt, void* stream);
int loco_checkpoint_read(const loco_checkpoint_t* ckpt, int64_t rows, int64_t cols, loco_act_t act,
                         void* out, loco_dtype_t out_dtype, void* stream);

/*
 * loco_linear - z = x weight^T + bias; out = act(z) + residual.
 *   x         device bf16[rows, in];  weight  device bf16[out_features, in]
 *   bias      device bf16[out_features], or NULL;  residual  device bf16[rows, out_features],
 *             or NULL
 *   ckpt      NULL, or the 8-bit checkpoint of z to write (of the fp32 z)
 *   out       device [rows, out_features] of `out_dtype`
 *   rows >= 0; in and out_features 0 .. 2^20 (LOCO_ERR_UNSUPPORTED beyond)
 *   workspace loco_linear_workspace(rows, out_features, in) bytes, which is what a call that
 *             writes a checkpoint needs; without one, up to 16 rows of at most 4096 in and
 *             out_features need none, and others need the same
 */
int loco_linear(const uint16_t* x, const uint16_t* weight, const uint16_t* bias, const uint16_t* residual,
                int64_t rows, int64_t out_features, int64_t in_features, loco_act_t act, void* out,
                loco_dtype_t out_dtype, const loco_checkpoint_t* ckpt, void* workspace,
                int64_t workspace_bytes, void* stream);
int64_t loco_linear_workspace(int64_t rows, int64_t out_features, int64_t in_features);

/*
 * loco_linear_input_grad - dx = (dy weight) * act'(z) + residual, where z is read from the
 * 8-bit checkpoint of the activation's input [rows, in].
 *   dy        device bf16[rows, out_features];  weight  device bf16[out_features, in]
 *   ckpt      the checkpoint; NULL: act must be LOCO_ACT_NONE
 *   residual  device bf16[rows, in], or NULL
 *   dx        device [rows, in] of `out_dtype`
 */
int loco_linear_input_grad(const uint16_t* dy, const uint16_t* weight, const uint16_t* residual,
                           int64_t rows, int64_t out_features, int64_t in_features, loco_act_t act,
                           const loco_checkpoint_t* ckpt, void* dx, loco_dtype_t out_dtype,
                           void* workspace, int64_t workspace_bytes, void* stream);
int64_t loco_linear_input_grad_workspace(int64_t rows, int64_t out_features, int64_t in_features);

/*
 * loco_linear_weight_grad - dweight = dy^T a, dbias = sum over the rows of dy, with
 * a = act(value of the 8-bit checkpoint [rows, in]).  LOCO_ACT_NONE and LOCO_ACT_RELU take the
 * checkpoint's values as they are, which are bf16 numbers.  A value of LOCO_ACT_GELU or
 * LOCO_ACT_SILU is rounded to bf16 for the product if grad_dtype is LOCO_BF16; for LOCO_F32 it
 * enters as the sum of two bf16 numbers, in two products, which take twice the time.
 *   dy          device bf16[rows, out_features]
 *   dweight     device [out_features, in] of `grad_dtype`
 *   dbias       device [out_features] of `grad_dtype`, or NULL
 *   accumulate  nonzero: added to what dweight and dbias hold (in fp32, rounded once per
 *               product)
 * With rows 0 the gradients are zero.
 */
int loco_linear_weight_grad(const uint16_t* dy, const loco_checkpoint_t* ckpt, int64_t rows,
                            int64_t out_features, int64_t in_features, loco_act_t act, int accumulate,
                            void* dweight, void* dbias, loco_dtype_t grad_dtype, void* workspace,
                            int64_t workspace_bytes, void* stream);
int64_t loco_linear_weight_grad_workspace(int64_t rows, int64_t out_features, int64_t in_features,
                                          loco_act_t act);

/* ---------------------------------------------------------------------------------
 * The norms around a transformer block: the RMS norm of its output, its gate, the residual
 * stream, and the RMS norm before the next block, in one pass.  The conventions are the layer
 * operators'.
 * ------------------------------------------------------------------------------ */

/* What multiplies a block's output beside the scale. */
typedef enum {
    LOCO_GATE_NONE = 0,
    LOCO_GATE_COLUMN = 1,  /* device [cols] of param_dtype */
    LOCO_GATE_ELEMENT = 2  /* device [rows, cols] of dtype */
} loco_gate_t;

/*
 * loco_residual_norm - per row:
 *   u   = y * post_rstd * post_weight,  post_rstd = 1/sqrt(sum(y^2)/cols + eps)
 *         (post_rstd NULL: u = y, and post_weight must be NULL)
 *   h   = residual + scale * gate * u   (residual NULL: without it)
 *   out = h * rstd * weight,  rstd = 1/sqrt(sum(h^2)/cols + eps)
 *   y, residual          device [rows, cols] of `dtype`; one may be NULL.  y NULL: h = residual, the
 *                        norm alone (gate and post-norm must be absent)
 *   gate                 as gate_kind says; NULL with LOCO_GATE_NONE
 *   weight, post_weight  device [cols] of `param_dtype`; NULL: ones
 *   scale, eps           finite; eps >= 0
 *   h                    device [rows, cols] of `dtype` (written), or NULL.  out is formed from the
 *                        fp32 h, before its rounding
 *   out, rstd            device [rows, cols] of `dtype`, f32[rows] (written); NULL both (then weight
 *                        and ckpt too): h alone
 *   post_rstd            device f32[rows] (written), for the backward pass
 *   ckpt                 NULL, or the 8-bit checkpoint of out to write (of its fp32 values)
 *   cols                 1 .. 16384 (LOCO_ERR_UNSUPPORTED beyond); rows 0 is a no-op
 * A sum of squares past FLT_MAX (values around 1e19) gives rstd 0.
 */
int loco_residual_norm(const void* y, const void* residual, loco_dtype_t dtype, const void* gate,
                       loco_gate_t gate_kind, const void* post_weight, const void* weight,
                       loco_dtype_t param_dtype, int64_t rows, int64_t cols, float scale, float eps,
                       void* h, void* out, float* post_rstd, float* rstd,
                       const loco_checkpoint_t* ckpt, void* stream);

/*
 * loco_residual_norm_backward - from the gradients dout of out and dh of h (either may be NULL: 0),
 * with xh = h * rstd and yh = y * post_rstd (post_rstd NULL: yh = y, post_weight ones):
 *   dresidual = dh + rstd * (dout * weight - xh * sum(dout * weight * xh)/cols)
 *   dweight   = sum over the rows of dout * xh
 *   t         = scale * gate * dresidual * post_weight
 *   dy        = post_rstd * (t - yh * sum(t * yh)/cols)     (post_rstd NULL: dy = t)
 *   dpost_weight = sum over the rows of scale * gate * dresidual * yh
 *   dgate     = scale * dresidual * yh * post_weight, summed over the rows for LOCO_GATE_COLUMN
 * all formed from the fp32 dresidual, before its rounding.
 *   dout, dh, h, y       device [rows, cols] of `dtype`; h (as stored) is needed with dout, y with
 *                        post_rstd or a gate
 *   dresidual, dy        device [rows, cols] of `dtype` (written), each may be NULL
 *   dgate                device [cols] of `grad_dtype`, or [rows, cols] of `dtype` (written); may be NULL
 *   dweight, dpost_weight  device [cols] of `grad_dtype` (written), each may be NULL
 *   workspace            loco_residual_norm_backward_workspace(rows, cols) bytes; may be NULL without
 *                        sums over the rows
 * With rows 0 the sums are written as zeros.
 */
int loco_residual_norm_backward(const void* dout, const void* dh, const void* h, const void* y,
                                loco_dtype_t dtype, const void* gate, loco_gate_t gate_kind,
                                const void* post_weight, const void* weight, loco_dtype_t param_dtype,
                                const float* post_rstd, const float* rstd, int64_t rows, int64_t cols,
                                float scale, void* dresidual, void* dy, void* dgate, void* dpost_weight,
                                void* dweight, loco_dtype_t grad_dtype, void* workspace,
                                int64_t workspace_bytes, void* stream);
int64_t loco_residual_norm_backward_workspace(int64_t rows, int64_t cols);

/* ---------------------------------------------------------------------------------
 * Log probabilities of given tokens under the logits of a head, with the entropy of each row's
 * distribution and its best alternatives; and the gradient that starts a backward pass.  The
 * conventions are the layer operators', but the rows of logits and dlogits may be any number of
 * elements >= vocab apart (ld, dld); what lies between them is neither read nor written.
 *
 * A row that holds a NaN or plus infinity has no distribution: its outputs are NaN (top_ids -1), and so
 * is its gradient.  A row of minus infinities only has the log probability minus infinity, the entropy 0
 * and the gradient 0; with a target past the vocabulary both are NaN, as in any row.  Minus infinity
 * elsewhere (a masked token) has the probability 0.
 *
 * The same call has the same bits.  The order of a row's sums depends on the number of rows of the call, so between
 * calls of other numbers of rows the last bits of its log probabilities, entropy and stats may differ.
 * ------------------------------------------------------------------------------ */

/* Largest number of alternatives. */
#define LOCO_MAX_TOP 32

/*
 * loco_token_logprobs - per row, with m = max x, S = sum exp(scale (x - m)), p = exp(scale (x - m)) / S:
 *   logprob = scale (x[target] - m) - ln S       0 for target < 0 (a token that is not scored),
 *                                                NaN for target >= vocab
 *   entropy = - sum p ln p
 *   top_ids, top_logprobs: the `top` largest logits in order, ties to the lower index, and their log
 *             probabilities; past vocab the id -1 and minus infinity
 *   logits   device [rows, vocab] of `dtype`, rows `ld` elements apart
 *   targets  device i64[rows]; may be NULL without logprob
 *   scale    1e-6 .. 1e6: an inverse temperature
 *   logprob, entropy  device f32[rows] (written), each may be NULL
 *   stats    device f32[rows][2] (written: m and S, for the backward pass), or NULL; ln sum exp(scale x) is
 *            scale m + ln S
 *   top      0 .. LOCO_MAX_TOP (LOCO_ERR_UNSUPPORTED beyond); top_ids i32, top_logprobs f32 [rows, top]
 *   workspace  loco_token_logprobs_workspace(rows, vocab, top) bytes
 *   vocab    1 .. 2^24 (LOCO_ERR_UNSUPPORTED beyond); rows 0 is a no-op
 */
int loco_token_logprobs(const void* logits, loco_dtype_t dtype, int64_t rows, int64_t vocab, int64_t ld,
                        const int64_t* targets, float scale, float* logprob, float* entropy,
                        float* stats, int top, int32_t* top_ids, float* top_logprobs,
                        void* workspace, int64_t workspace_bytes, void* stream);
int64_t loco_token_logprobs_workspace(int64_t rows, int64_t vocab, int top);

/*
 * loco_token_logprobs_backward - the gradient of sum(dlogprob * logprob + dentropy * entropy):
 *   dlogits[j] = scale * (dlogprob * ((j == target) - p[j]) - dentropy * p[j] * (ln p[j] + entropy))
 * A target < 0 takes its row's dlogprob for 0, one >= vocab makes its row's gradient NaN.  Rows without
 * anything to differentiate (no dentropy, target < 0) are written as zeros and not read.
 *   stats, entropy      as loco_token_logprobs wrote them; entropy with dentropy only
 *   dlogprob, dentropy  device f32[rows]; one may be NULL: 0.  targets go with dlogprob
 *   dlogits             device [rows, vocab] of `dtype` (written), rows dld elements apart.  It may be
 *                       logits itself (with dld = ld): in place; else, from first to last element, it may
 *                       not overlap them
 */
int loco_token_logprobs_backward(const void* logits, loco_dtype_t dtype, int64_t rows, int64_t vocab,
                                 int64_t ld, const int64_t* targets, float scale, const float* stats,
                                 const float* entropy, const float* dlogprob, const float* dentropy,
                                 void* dlogits, int64_t dld, void* stream);

/*
 * loco_token_logprobs_ex, loco_token_logprobs_backward_ex - the same of seqs sequences of `rows` rows each, where the
 * last rows of a sequence, or other elements, lie between it and the next: logits[:, :-1] with targets ids[:, 1:].
 *   seq_ld, dseq_ld  elements from one sequence's first row of logits, of dlogits, to the next one's: at least
 *                    (rows - 1) * ld + vocab
 *   target_ld        the same of targets: at least rows.  All other buffers hold seqs * rows rows without gaps
 *   dlogits          may be logits itself with dld = ld and dseq_ld = seq_ld
 * With one sequence these steps are ignored; more may have 2^32 - 1 rows in all (LOCO_ERR_UNSUPPORTED beyond).  The
 * workspace is that of seqs * rows rows, and the only buffer to be 16-byte aligned: the others need their elements'
 * alignment (8 bytes for targets, 4 for stats), so that each may start anywhere in a tensor.
 */
int loco_token_logprobs_ex(const void* logits, loco_dtype_t dtype, int64_t seqs, int64_t rows, int64_t vocab,
                           int64_t ld, int64_t seq_ld, const int64_t* targets, int64_t target_ld,
                           float scale, float* logprob, float* entropy, float* stats, int top,
                           int32_t* top_ids, float* top_logprobs, void* workspace,
                           int64_t workspace_bytes, void* stream);
int loco_token_logprobs_backward_ex(const void* logits, loco_dtype_t dtype, int64_t seqs, int64_t rows,
                                    int64_t vocab, int64_t ld, int64_t seq_ld, const int64_t* targets,
                                    int64_t target_ld, float scale, const float* stats,
                                    const float* entropy, const float* dlogprob, const float* dentropy,
                                    void* dlogits, int64_t dld, int64_t dseq_ld, void* stream);

/* ---------------------------------------------------------------------------------
 * AdamW over many tensors at once, with states in fp32 or in 8 bits: the step of the parameters
 * whose gradient does not arrive as payloads of loco_dequant_reduce_adam, or whose states
 * should take 2 bytes and not 8.
 *
 * An 8-bit state of n elements has blocks of `block` elements from element 0 (the last may be
 * partial), each with one exponent byte.
 *   first moment   codes u8[n]: float8 of 4 exponent and 3 mantissa bits (bias 7, largest 448,
 *                  torch.float8_e4m3fn) times 2^(exps - 127), the least power of two
 *                  (>= 2^-117) that keeps the block's largest magnitude within 448
 *   second moment  codes u8[n]: 0 is 0; a code c > 0 is (1 + (c & 7)/8) * 2^((c >> 3) - 31 + exps -
 *                  127), with exps (>= 32; read as 32 below) the biased exponent of the block's
 *                  largest value rounded to 4 significant bits.  Values that are not 0 are
 *                  never stored as 0, but as the code 1 at least; values < 0 are stored as 0
 *   exps   u8[ceil(n/block)]
 * Each value is rounded once, to four significant bits (fewer where a first moment is below 2^-14 of
 * its block's range): by loco_adamw and loco_adamw_state_write to nearest, ties to even; by loco_adamw_ex at
 * random.  A block that holds an infinity or a NaN (or a second moment that rounds to 2^128) is stored with
 * exps 255 and codes 0 and reads as NaN.  A state whose codes are 0 is 0, whatever its exps below 255.
 *
 * Steps of a training run need random rounding.  To nearest, what changes a state by less than half a step is
 * lost, at every step again: a second moment stays where it is for good wherever 1 - beta2 is below 1/18, and is
 * off its average at any beta2 above 0.9; a first moment from beta1 of about 0.945 on, and at any beta1 where it
 * is below 2^-14 of its block's range, so that a parameter without a gradient goes on moving.
 * ------------------------------------------------------------------------------ */

/* One tensor (host struct, read while planning and at each step). */
typedef struct {
    void* param;          /* device, n elements of param_dtype, updated in place */
    const void* grad;     /* device, n elements of grad_dtype */
    void* m;              /* device, f32[n] or codes u8[n], updated in place */
    void* v;              /* the same */
    uint8_t* m_exps;      /* device u8[ceil(n/block)], updated; unused with states in fp32 */
    uint8_t* v_exps;
    uint16_t* param_bf16; /* device (written: the RNE bf16 copy of the new param), or NULL; LOCO_F32 only */
    int64_t n;            /* elements (>= 0; 0 is a no-op) */
    double weight_decay;  /* finite */
} loco_adamw_tensor_t;

/* Hyper-parameters (host struct, read during the call: a captured graph repeats them). */
typedef struct {
    double lr;           /* finite */
    double beta1, beta2; /* in [0, 1): the weights of the OLD moments (unlike loco_adam_t) */
    double eps;          /* > 0, and as a float too */
    int64_t step;        /* >= 1: this step's number t */
} loco_adamw_t;

/*
 * A plan describes the tensors of many calls once: their addresses lie in a table in device memory, so
 * that a step of any number of tensors is one launch that reads nothing but its arguments from the
 * host.  The caller keeps this struct, the table and the host array of tensors as they are, and the tensors
 * where they are, for as long as calls use the plan; its fields are the library's.
 */
typedef struct {
    int kind, ntensors;
    int64_t live, tiles;
    const void* table;
    const loco_adamw_tensor_t* tensors;
    int param_dtype, grad_dtype, state_bits, block;
} loco_adamw_plan_t;

/* Bytes of the table of n tensors, or of n states. */
int64_t loco_adamw_table_bytes(int n);

/*
 * loco_adamw_plan - checks ntensors (>= 0) tensors, fills their table on `stream` (calls on other
 * streams have to wait for it) and *plan.
 *   state_bits  32 or 8;  block  64, 128, 256 or 512 (ignored with 32)
 *   table       device memory of table_bytes >= loco_adamw_table_bytes(ntensors)
 * No buffer that a step writes may overlap another of its buffers, or the table.
 */
int loco_adamw_plan(const loco_adamw_tensor_t* tensors, int ntensors, loco_dtype_t param_dtype,
                    loco_dtype_t grad_dtype, int state_bits, int block, void* table,
                    int64_t table_bytes, loco_adamw_plan_t* plan, void* stream);

/*
 * loco_adamw - one step of a plan's tensors: for every element, in IEEE fp32 operations in this order:
 *   g     = grad * grad_scale[0]                      (grad_scale NULL: g = grad)
 *   m     = beta1 * m + (1 - beta1) * g
 *   v     = beta2 * v + (1 - beta2) * (g * g)
 *   param = param * (1 - lr * weight_decay)
 *           - lr / (1 - beta1^t) * (m / (sqrt(v) * (1 / sqrt(1 - beta2^t)) + eps))
 * with each factor of the hyper-parameters formed in 64 bits and rounded to fp32 once.  With 8-bit states
 * the parameter's update takes m and v before they are rounded into their codes.
 *   grad_scale  device f32[1] (read), such as a clipping factor, or NULL; it must not lie in a buffer
 *               that the step writes
 * 8-bit states are rounded to nearest: for single steps (see above).
 */
int loco_adamw(const loco_adamw_plan_t* plan, const loco_adamw_t* options, const float* grad_scale,
               void* stream);

/* The random bits of a step (host struct, read during the call). */
typedef struct {
    uint64_t seed;
    const int64_t* counter; /* device i64[1] (read by the step), or NULL: 0.  A captured graph repeats seed and
                               options->step: give it a counter that another kernel of the graph raises */
} loco_adamw_rounding_t;

/*
 * loco_adamw_ex - loco_adamw with the 8-bit states rounded at random, up or down to the nearest codes in the
 * proportion of the distances: with other bits at every step, m and v are their averages in the mean.
 *   rounding  NULL: to nearest, as loco_adamw; of no effect on states in fp32.  counter must not lie in a buffer
 *             that the step writes
 * The bits are a hash of seed, options->step, *counter and the element's place among the plan's elements, in
 * which each tensor takes a multiple of 512: the same call has the same results.  A value goes up
 * if the part of the step that it has over the lower code, in 2^-20 of a step, and 20 bits come to 2^20 or
 * more; what is a code's value stays.  exps of a second moment are those of the block's largest value rounded up
 * to 4 significant bits (255 past 15/8 2^127); a value > 0 below the code 1 is still stored as 1.
 */
int loco_adamw_ex(const loco_adamw_plan_t* plan, const loco_adamw_t* options, const float* grad_scale,
                  const loco_adamw_rounding_t* rounding, void* stream);

/* One 8-bit state and its values (host struct, read while planning). */
typedef struct {
    uint8_t* codes; /* device u8[n] */
    uint8_t* exps;  /* device u8[ceil(n/block)] */
    void* values;   /* device, n elements of `dtype` */
    int64_t n;
    int moment;     /* 1 or 2 */
} loco_adamw_state_t;

/*
 * loco_adamw_state_plan  - as loco_adamw_plan, for states and their values, LOCO_F32 or LOCO_BF16; no buffer may
 *                          overlap another.  The array of states is read during the call only.
 * loco_adamw_state_read  - values = what the plan's states stand for (exact in either type).
 * loco_adamw_state_write - the states of the plan's values, as loco_adamw stores them.
 */
int loco_adamw_state_plan(const loco_adamw_state_t* states, int nstates, int block, loco_dtype_t dtype,
                          void* table, int64_t table_bytes, loco_adamw_plan_t* plan, void* stream);
int loco_adamw_state_read(const loco_adamw_plan_t* plan, void* stream);
int loco_adamw_state_write(const loco_adamw_plan_t* plan, void* stream);

/* A static, human-readable name for a status code. */
const char* loco_status_string(int status);

/* Library ABI version (major * 10000 + minor * 100 + patch). */
int loco_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LOCO_H */
