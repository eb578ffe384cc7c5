/*
 * qlora_train.h -- C ABI of the operators around the quantized linear in a
 * fine-tuning step (gfx950 / MI355X; same library as qlora_nf4.h): token
 * embedding and its gradient, the residual norm of a block and its gradient,
 * the global gradient norm and the AdamW step over many tensors.
 *
 * Conventions are those of qlora_nf4.h: device pointers owned by the caller,
 * nothing allocated, freed or synchronized (qlora_adamw_init excepted), work
 * enqueued on `stream`, every argument checked before the first HIP call,
 * positive QLORA_ERR_* statuses (qlora_strerror), deterministic results (the
 * same inputs give the same bits).  Nothing that a result depends on is kept between calls;
 * qlora_grad_norm alone writes to memory of the plan while it runs, so that two of
 * its calls on one plan must not overlap.
 * Dtypes are QLORA_F32, QLORA_BF16 and QLORA_F16.  Matrices are row-major
 * with unit column stride; ld* is the row stride in elements (>= the row
 * width).  Tensors need the alignment of one element only; rows that start on
 * 16 bytes are read and written fastest.  Sums, means and optimizer moments
 * are formed in binary32; every output is rounded once, to nearest even.  Inside,
 * the norms' reciprocal roots and the root and reciprocal of the AdamW update are those of
 * the instructions, good to one unit in the last place of binary32 (the update's are
 * rounded to nearest where eps is below 2^-39 / sqrt(1 - beta2^t)).
 */
#ifndef QLORA_TRAIN_H
#define QLORA_TRAIN_H

#include <stddef.h>
#include <stdint.h>

#include "qlora_nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------ embedding */

#define QLORA_EMBED_MAX_M 16777216LL  /* tokens of one embedding call (2^24) */
#define QLORA_EMBED_MAX_V 4194304LL   /* table rows (2^22) */
#define QLORA_EMBED_MAX_D 65536LL     /* row width */

/*
 * out[t][:] = scale * E[ids[t]][:], t < m.  A row whose id lies outside
 * [0, vocab) (a padding marker such as -1) is all zeros.
 * E [vocab x d] in e_dtype; ids: m token ids of id_bits (32 or 64) bits,
 * signed; out [m x d] in out_dtype: e_dtype, QLORA_F32, or for an fp32 table
 * any dtype.  m == 0 enqueues nothing.  out must not overlap E or ids.
 * QLORA_ERR_SHAPE: m < 0 or above QLORA_EMBED_MAX_M, vocab or d < 1 or above
 * their limits, a row stride below d; QLORA_ERR_DTYPE; QLORA_ERR_ARG for
 * another id_bits; QLORA_ERR_ALIGN for a pointer not aligned to its elements.
 */
int qlora_embed_fwd(const void *E, int e_dtype, int64_t vocab, int64_t d, int64_t lde,
                    const void *ids, int id_bits, int64_t m, float scale, void *out, int out_dtype,
                    int64_t ldo, void *stream);

/*
 * Host.  Workspace bytes of qlora_embed_bwd (0 on a shape it refuses).
 */
size_t qlora_embed_workspace_bytes(int64_t m, int64_t vocab, int64_t d);

/*
 * dE[v][:] = scale * sum over {t : ids[t] == v} of dY[t][:], the tokens of a
 * row added in a fixed order (a stable sort of the ids; fp32 partial sums over
 * runs of consecutive sorted tokens, joined in order).  Ids outside
 * [0, vocab) contribute nothing.
 * accumulate == 0 writes all vocab rows (zeros where no token points);
 * accumulate != 0 adds to dE instead, touching only rows with a token.
 * dY [m x d] in dy_dtype; dE [vocab x d] in de_dtype: QLORA_F32 or dy_dtype.
 * dE must not overlap dY or ids.  Errors as qlora_embed_fwd, and
 * QLORA_ERR_WORKSPACE when `workspace` (16-byte aligned) is missing or too
 * small.  m == 0 writes zeros, or nothing when accumulating.
 */
int qlora_embed_bwd(const void *dY, int dy_dtype, int64_t m, int64_t d, int64_t lddy,
                    const void *ids, int id_bits, int64_t vocab, float scale, void *dE,
                    int de_dtype, int64_t ldde, int accumulate, void *workspace,
                    size_t workspace_bytes, void *stream);

/* -------------------------------------------------------- residual norm */

#define QLORA_RESNORM_MAX_D 65536   /* widest row */

/* gate of the residual norm (gate_kind) */
enum {
  QLORA_GATE_NONE = 0,
  QLORA_GATE_CHANNEL = 1, /* gate[d], one value a column */
  QLORA_GATE_TOKEN = 2,   /* gate[m], one value a row */
  QLORA_GATE_FULL = 3     /* gate[m x d], row stride ldg */
};

/*
 * The residual path at the end of a block and the start of the next:
 *   rms(u) = u / sqrt(mean(u^2) + eps)                        over a row of d
 *   p = post ? rms(y) * (w_offset + w_post) : y
 *   h = x + scale * gate * p                                  (new residual)
 *   z = rms(h) * (w_offset + w_pre)      when pre             (next block's input)
 * z uses h before its rounding to res_dtype.  A row's squares are summed in binary32: one
 * whose sum passes its range counts as infinitely large (rms(u) = 0), and with eps == 0 a
 * row of zeros divides by zero (NaN).  With y == NULL there is no
 * branch: z = rms(x) * (w_offset + w_pre); post, gate_kind, h are then ignored and
 * pre must be set.  A NULL w_post / w_pre stands for w_offset + w = 1.
 * x, h in res_dtype (QLORA_F32 or act_dtype); y, z and a full gate in
 * act_dtype; w_post, w_pre, channel and token gates in param_dtype (QLORA_F32
 * or act_dtype).  h may be x itself and z may be y itself (same pointer and
 * row stride); other overlaps are not allowed.  m == 0 enqueues nothing.
 * QLORA_ERR_SHAPE: m < 0 or above QLORA_MAX_M, d outside
 * [1, QLORA_RESNORM_MAX_D], a row stride below d; QLORA_ERR_NULL for a missing
 * x, h (with y), z (with pre) or gate; QLORA_ERR_ARG: unknown gate_kind, eps
 * negative or not finite, neither y nor pre; QLORA_ERR_DTYPE; QLORA_ERR_ALIGN.
 */
typedef struct {
  int64_t m, d;
  int32_t act_dtype, res_dtype, param_dtype;
  int32_t post, pre, gate_kind;
  float scale, eps, w_offset;
  const void *x, *y, *gate, *w_post, *w_pre;
  int64_t ldx, ldy, ldg;
  void *h, *z;
  int64_t ldh, ldz;
} qlora_resnorm;

int qlora_resnorm_fwd(const qlora_resnorm *a, void *stream);

/* Host.  Workspace bytes of qlora_resnorm_bwd for any gate and outputs (0 on a bad shape). */
size_t qlora_resnorm_workspace_bytes(int64_t m, int64_t d);

/*
 * Gradients of the above from dz (the gradient of z, with pre) and dh (the
 * gradient that reaches h from later blocks; NULL: none), given h as stored by the
 * forward (x for a call without y), y, the gate and the weights:
 *   D = dh + d(z)/d(h)^T dz                                    -> dx
 *   dw_pre[c]  = sum_t dz * rms(h)
 *   q = scale * gate * D;   dy = post ? d(rms(y) (w_offset + w_post))/d(y)^T q : q
 *   dw_post[c] = sum_t q * rms(y)
 *   dgate = scale * D * p, summed over the rows (channel), over the columns (token), or
 *           not at all (full)
 * dz, dy and a full dgate in act_dtype; dh, dx in res_dtype; dw_pre, dw_post
 * [d], channel dgate [d] and token dgate [m] fp32.  A NULL dy, dgate, dw_post
 * or dw_pre is not computed.  dx may be dh itself and dy may be dz itself (same pointer
 * and row stride).  Without y: dx and dw_pre only.  m == 0 writes zeros to
 * dw_post, dw_pre and a channel dgate.
 * The workspace (16-byte aligned) is needed when dw_post, dw_pre or a channel
 * dgate is asked for.
 * Errors as qlora_resnorm_fwd, QLORA_ERR_NULL when neither dz (with pre) nor
 * dh is given, and QLORA_ERR_WORKSPACE.
 */
typedef struct {
  int64_t m, d;
  int32_t act_dtype, res_dtype, param_dtype;
  int32_t post, pre, gate_kind;
  float scale, eps, w_offset;
  const void *dz, *dh, *h, *y, *gate, *w_post, *w_pre;
  int64_t lddz, lddh, ldh, ldy, ldg;
  void *dx, *dy, *dgate;
  int64_t lddx, lddy, lddg;
  float *dw_post, *dw_pre;
} qlora_resnorm_grad;

int qlora_resnorm_bwd(const qlora_resnorm_grad *a, void *workspace, size_t workspace_bytes,
                      void *stream);

/* ---------------------------------------------------------------- AdamW */

#define QLORA_ADAMW_BLOCK 256          /* values a section is padded to, and that share 8-bit scales */
#define QLORA_ADAMW_MAX_TENSORS 1048576

/*
 * One tensor of a plan: n values at p (read), written to p_out (p itself for
 * an update in place), gradient g, optional copy of the new fp32 values in 16
 * bits (for a model whose forward reads bf16 or fp16 weights).  lr_mul and wd_mul
 * multiply the step's learning rate and weight decay for this tensor.
 */
typedef struct {
  const void *p, *g;
  void *p_out, *copy;
  int64_t n;
  float lr_mul, wd_mul;
} qlora_opt_tensor;

/* Plain-data handle filled by qlora_adamw_init; `table` is the caller's device buffer. */
typedef struct {
  void *table;
  int32_t count, p_dtype, g_dtype, copy_dtype, state_bits;
  int64_t blocks, chunks;
} qlora_adamw;

/*
 * The moments of all tensors of a plan, in the order of the plan: tensor i
 * owns the blocks [b_i, b_i + ceil(n_i / 256)) of QLORA_ADAMW_BLOCK values, b_0 = 0,
 * sections back to back (plan.blocks in all); values past n_i in a last
 * block are zero.
 *   state_bits 32: m, v fp32 [blocks x 256]; m_scale, v_scale unused.
 *   state_bits 8:  m codes in OCP e4m3 and v codes in OCP e5m2, one byte a
 *     value, with fp32 scales m_scale, v_scale [blocks]: the moment is
 *     code * scale.  A block's scale is its largest magnitude / 448 (m) or
 *     / 57344 (v), 0 with all codes 0 when that magnitude is below 2^-110.
 * Zero bytes everywhere are the state before the first step.
 */
typedef struct {
  void *m, *v;
  float *m_scale, *v_scale;
} qlora_opt_state;

/* Step settings.  step counts from 1. */
typedef struct {
  int64_t step;
  double lr, beta1, beta2, eps, weight_decay;
  uint32_t seed;                       /* of the 8-bit states' rounding */
} qlora_adamw_hyper;

/* Host.  Device bytes of the table for tensors of n[0..count) values (0 on a bad size). */
size_t qlora_adamw_table_bytes(const int64_t *n, int count);

/*
 * Host, setup time.  Checks the tensors and writes the device table (16-byte
 * aligned, >= qlora_adamw_table_bytes) with a blocking copy: this call
 * synchronizes, but only with that copy: earlier work on the table's memory must have
 * ended.  All tensors share p_dtype, g_dtype (any dtype each) and, where copies are
 * given, copy_dtype (QLORA_BF16 or QLORA_F16, with p_dtype QLORA_F32).  The plan holds the
 * buffers' addresses: they must stay valid while it is used, each step reads its gradients from
 * them, and gradients at other addresses need another plan.  n == 0 tensors are allowed.
 * QLORA_ERR_NULL; QLORA_ERR_SHAPE: n < 0, or 2^31 blocks or more in all;
 * QLORA_ERR_ARG: count outside [1, QLORA_ADAMW_MAX_TENSORS], state_bits not 8
 * or 32, a non-finite multiplier; QLORA_ERR_DTYPE; QLORA_ERR_ALIGN; QLORA_ERR_WORKSPACE: table_bytes too
 * small; QLORA_ERR_HIP.
 */
int qlora_adamw_init(qlora_adamw *plan, const qlora_opt_tensor *tensors, int count, int p_dtype,
                     int g_dtype, int copy_dtype, int state_bits, void *table, size_t table_bytes);

/* Host.  Workspace bytes of qlora_grad_norm. */
size_t qlora_grad_norm_workspace_bytes(const qlora_adamw *plan);

/*
 * out[0] = sqrt(sum of g^2 over all tensors of the plan), out[1] = the factor
 * that brings it to max_norm: min(1, max_norm / (out[0] + 1e-6)), 1 when max_norm <= 0,
 * NaN when out[0] is not finite (a step given that factor is
 * skipped).  out: 2 floats on the device.  The call counts its workgroups in the plan's
 * table, zero again when it ends: two calls on one plan must not overlap, whatever
 * streams, workspaces and outputs they have (their results would be undefined; later
 * calls are not affected).  The step only reads the table.
 */
int qlora_grad_norm(const qlora_adamw *plan, float max_norm, float *out, void *workspace,
                    size_t workspace_bytes, void *stream);

/*
 * One AdamW step over all tensors of the plan (decoupled weight decay), with
 * c = *grad_scale (device; NULL: 1), t = step, lr = h->lr * lr_mul,
 * wd = h->weight_decay * wd_mul:
 *   g' = c g;  m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) g'^2
 *   p  = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
 * The moments are read from `in` and written to `out` (the same buffers for a
 * step in place).  If c is not finite the step is skipped: p_out = p (and
 * copy = p rounded), out = in.  A gradient that is not finite otherwise
 * reaches p.  With eps == 0 a second moment of 0 (a square below binary32's smallest number
 * among them) is divided by, as the formula says.
 * 8-bit moments: p is updated from the fp32 moments of this step, which are
 * then rounded stochastically: a magnitude x goes to the grid with random
 * bits added below the kept mantissa bits, so that its expectation is x; a
 * positive second moment never becomes 0.  A moment that is not finite (a
 * gradient's infinity or NaN, or a square above binary32's range) is left out of its
 * block's scale and gets the largest code with its sign, so that the block's other values
 * are held as if it were 0.  For value j of block b of the
 * state, mod 2^32:
 *   mix(x): x ^= x >> 16; x *= 0x6A09E667; x ^= x >> 15; x *= 0xBB67AE85; x ^= x >> 16
 *   bits = mix(mix(mix(seed + 0x9E3779B9 step) + 0x510E527F b) + 0x9E3779B9 (j + 1))
 * m takes the low and v the high 16 bits.
 * The settings in `h` are read when the call is made: a captured step repeats them, its
 * step count among them, on every replay.  Only *grad_scale, the gradients, the parameters and
 * the state are read on the device.
 * QLORA_ERR_ARG: step < 1, beta1 or beta2 outside [0, 1), lr, eps or weight_decay negative
 * or not finite, a handle not filled by qlora_adamw_init.
 */
int qlora_adamw_step(const qlora_adamw *plan, const qlora_opt_state *in, const qlora_opt_state *out,
                     const qlora_adamw_hyper *h, const float *grad_scale, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* QLORA_TRAIN_H */
