/*
 * lora_train.h -- training adapters of a paged pool: losses on logits, and the
 * optimizer step.
 *
 * lora_sgmv_backward (lora_sgmv.h) turns dL/dy into dA_i and dB_i, added into an
 * fp32 gradient array laid out like the pool's pages.  This part is what stands
 * on either side of it in a training step:
 *   - lora_token_logprobs, lora_preference_loss, lora_policy_loss: from the
 *     logits of a batch to its loss and dL/dlogits;
 *   - lora_grad_sumsq, lora_adamw_step: from the gradient array to new weights
 *     in the pool, for the adapters listed in a call, each with its own step
 *     count, learning rate and clipping norm (tenants train at their own pace);
 *   - lora_adamw_init: the state of adapters that enter the pool.
 *
 * Conventions are those of lora_sgmv.h: the caller owns every buffer, calls are
 * asynchronous on `stream`, allocate nothing and keep nothing between calls,
 * argument errors found on the host are returned before anything is launched,
 * and what only the device can see is OR-ed into *dev_err (may be NULL).
 * Calls can be captured in CUDA graphs.  Results do not depend on timing: every
 * sum has a fixed order (a row's depends on the call, on T and V and on where its
 * 16-byte boundaries lie).
 * A bounded wait inside a kernel that ran out sets LORA_DERR_TIMEOUT; the rows it
 * concerned are left as they were.
 */
#ifndef LORA_TRAIN_H
#define LORA_TRAIN_H

#include "lora_sgmv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further bits of the device error word. */
#define LORA_DERR_BAD_LABEL 16 /* a label >= V: its row does not count */
#define LORA_DERR_BAD_SEQ 32   /* sequence offsets not ascending within [0, T] */
#define LORA_DERR_NONFINITE 64 /* an adapter's gradient norm is not finite: it was not stepped */

/* ------------------------------------------------------------ loss on logits --
 *
 * logits: device [T, ld] rows of V entries (ld >= V; columns past V are neither
 * read nor written), bf16 or fp32; rows need no alignment beyond the element's.
 * labels: device int32 [T]: row t's next token; a negative label marks a row
 * that does not count (prompt, padding): its per-row outputs are 0 and its
 * gradient row is zero.  Entries may be -inf (masked); a row with nothing else
 * has logp = -inf and a zero gradient row.  NaN and +inf propagate to the
 * row's outputs.  Exponentials and sums are fp32; each gradient entry is
 * rounded once to the logits' type.
 *
 * dlogits: device [T, ldd >= V], the logits' type, written only; it may be the
 * logits themselves (same pointer, ldd = ld), else it must not overlap them.
 * NULL: the loss without its gradient.
 */
#define LORA_LOGITS_BF16 0
#define LORA_LOGITS_F32 1

/**
 * logp[t] = logits[t, labels[t]] - lse[t], lse[t] = log sum_v exp(logits[t, v]).
 * logp, lse: device fp32 [T]; lse may be NULL.  V >= 1, T >= 0 (T = 0: nothing
 * to do).
 */
lora_status_t lora_token_logprobs(const void* logits, int64_t ld, int32_t dtype, const int32_t* labels,
                                  int32_t T, int32_t V, float* logp, float* lse, int32_t* dev_err,
                                  lora_stream_t stream);

/* Kinds of lora_preference_loss. */
#define LORA_PREF_SIGMOID 0
#define LORA_PREF_HINGE 1
#define LORA_PREF_IPO 2
/* Flags of lora_preference_loss. */
#define LORA_PREF_AVERAGE 1 /* log ratios are means over the counted tokens, not sums */

typedef struct {
  int32_t kind;          /* LORA_PREF_* */
  uint32_t flags;        /* LORA_PREF_AVERAGE or 0 */
  float beta;            /* > 0 */
  float label_smoothing; /* 0 .. 1, of LORA_PREF_SIGMOID */
  float margin;          /* subtracted from beta * (difference), of sigmoid and hinge */
  float grad_scale;      /* multiplies the gradient (1 / n_pairs for a mean loss) */
} lora_pref_opts_t;

/** Bytes of the workspace of lora_preference_loss (16-byte aligned; contents do not matter). */
size_t lora_preference_workspace_bytes(int32_t T, int32_t n_pairs);

/**
 * Paired preference loss.  Sequence s covers rows seq_indptr[s] ..
 * seq_indptr[s + 1] (device int32 [2 n_pairs + 1], ascending, within [0, T]);
 * pair p is sequence 2p (chosen) and 2p + 1 (rejected).  With
 *     R_s = sum over the sequence's counted rows of logp[t] - ref_logp[t]
 * (the mean with LORA_PREF_AVERAGE; 0 for a sequence without counted rows),
 * D = R_chosen - R_rejected and z = beta D - margin:
 *     sigmoid: -(1 - e) log s(z) - e log s(-z)   (e = label_smoothing)
 *     hinge:   max(0, 1 - z)
 *     ipo:     (D - 1 / (2 beta))^2
 * loss[p] (device fp32 [n_pairs]) is the pair's loss, seq_logp[s] (device fp32
 * [2 n_pairs], may be NULL) the plain sum of its counted logp, and
 *     dlogits[t, v] = +- dloss/dD * share * grad_scale
 *                     * (1[v = label] - softmax(logits[t])[v]),
 * share = 1, or 1 / counted rows with LORA_PREF_AVERAGE.  Rows of no sequence
 * get a zero gradient.  ref_logp: device fp32 [T], read at counted rows; NULL
 * stands for zeros.  Offsets that are not ascending within [0, T] set
 * LORA_DERR_BAD_SEQ; every loss, seq_logp and gradient is then 0.
 */
lora_status_t lora_preference_loss(const void* logits, int64_t ld, int32_t dtype, const int32_t* labels,
                                   const float* ref_logp, const int32_t* seq_indptr, int32_t n_pairs,
                                   int32_t T, int32_t V, const lora_pref_opts_t* opts, float* loss,
                                   float* seq_logp, void* dlogits, int64_t ldd, void* workspace,
                                   size_t workspace_bytes, int32_t* dev_err, lora_stream_t stream);

typedef struct {
  float clip_low;   /* 0 .. 1: the ratio's lower bound is 1 - clip_low */
  float clip_high;  /* >= 0: its upper bound is 1 + clip_high */
  float kl_coef;    /* >= 0; 0: ref_logp is not read and kl is 0 */
  float grad_scale; /* multiplies the gradient */
} lora_policy_opts_t;

/**
 * Clipped policy loss with a KL term, per row: q = exp(logp - old_logp),
 * d = ref_logp - logp, kl = exp(d) - 1 - d,
 *     loss[t] = weight[t] * (kl_coef * kl - min(q A, clip(q) A)),
 *     dlogits[t, v] = grad_scale * weight[t] * (kl_coef (1 - exp(d)) - [q A <= clip(q) A] q A)
 *                     * (1[v = label] - softmax(logits[t])[v]).
 * old_logp, advantage: device fp32 [T]; ref_logp (NULL only if kl_coef = 0) and
 * weight (NULL: 1) likewise.  A row of weight 0 has loss 0 and a zero gradient
 * row, whatever its ratio.  logp, loss: device fp32 [T]; kl: fp32 [T] or NULL.
 * logp is lora_token_logprobs's but for the order of the row's sum (the same bits
 * up to V = 128 vectors of 16 bytes), so the first step on a policy's own samples
 * has ratios of 1 within its rounding.
 */
lora_status_t lora_policy_loss(const void* logits, int64_t ld, int32_t dtype, const int32_t* labels,
                               const float* old_logp, const float* ref_logp, const float* advantage,
                               const float* weight, int32_t T, int32_t V, const lora_policy_opts_t* opts,
                               float* logp, float* loss, float* kl, void* dlogits, int64_t ldd,
                               int32_t* dev_err, lora_stream_t stream);

/* ------------------------------------------------------------ optimizer step --
 *
 * A projection's training state.  Every array is laid out like the pool: the
 * element at pool[i] has its gradient at grad[i] and its moments at m[i], v[i].
 * State belongs to pages, not to adapter ids: pin an adapter (lora_pool_pin)
 * while it trains, and run lora_adamw_init after a load.
 *
 * Moments: LORA_STATE_F32 holds the first moment in m and the second in v, as
 * fp32.  LORA_STATE_E4M3 holds one byte each, e4m3 codes with one bf16 scale for
 * each LORA_ADAMW_BLOCK consecutive elements (m_scale[i / 64], v_scale[i / 64]):
 * m's code times its scale is the first moment; v's code times its scale is the
 * square ROOT of the second (which halves the range that the codes must span).
 * A scale is bf16(largest magnitude of the block / 448); codes are rounded to
 * nearest, ties to even; a root above zero never takes code 0, so that no
 * element divides by eps alone; a block whose largest value is below 2^-100
 * holds zeros, and second moments below 2^-126 count as zero.
 */
#define LORA_STATE_F32 0
#define LORA_STATE_E4M3 1
#define LORA_ADAMW_BLOCK 64

typedef struct {
  lora_pool_view_t view; /* the pool; lora_adamw_step writes it, though the view declares it const */
  float* grad;           /* device fp32 [n_pages * page_elems], as lora_sgmv_backward fills it */
  float* master;         /* device fp32 weights, or NULL: the bf16 pool is the only copy */
  void* m;               /* first moments */
  void* v;               /* second moments, or their roots */
  void* m_scale;         /* bf16 [n_pages * page_elems / 64]; NULL with LORA_STATE_F32 */
  void* v_scale;
} lora_train_proj_t; /* 16-byte aligned (the scales: 2), no two overlapping */

/** One adapter's settings (32 bytes, device array of n_adapters, indexed by adapter id). */
typedef struct {
  int32_t step;       /* t of this step, from 1; below 1: the adapter is not stepped */
  float lr;
  float beta1;
  float beta2;
  float eps;
  float weight_decay; /* decoupled: w is multiplied by 1 - lr * weight_decay */
  float max_norm;     /* gradient norm to clip to, where a call has sumsq; <= 0: no clipping */
  float grad_scale;   /* multiplies the gradient (1 / accumulated batches, say) */
} lora_adamw_hyper_t;

/**
 * Prepare the listed adapters' state: grad, m and v (and their scales) to zero,
 * master to the pool's weights.
 *
 * This and the next two calls share: projs (host array of n_proj, every view
 * with the same n_adapters); ids (device int32 [n_ids], the adapters, at most
 * LORA_MAX_ADAPTERS).  An id outside [0, n_adapters) or listed before sets
 * LORA_DERR_BAD_ADAPTER, one whose rank in a projection is outside
 * [1, max_rank] LORA_DERR_BAD_RANK, and the call passes over it (for a rank: in
 * that projection).  Elements whose page-list slot or page is outside the pool
 * set LORA_DERR_BAD_PAGE and stay as they were; the others are processed.
 * Elements of no listed adapter are never written.  n_ids = 0: nothing to do.
 */
lora_status_t lora_adamw_init(const lora_train_proj_t* projs, int32_t n_proj, int32_t state,
                              const int32_t* ids, int32_t n_ids, int32_t* dev_err, lora_stream_t stream);

/**
 * Bytes of lora_grad_sumsq's workspace (16-byte aligned; contents do not matter); 0 on bad arguments.
 * One made for n_ids adapters serves any shorter list over the same projections.
 */
size_t lora_grad_sumsq_workspace_bytes(const lora_train_proj_t* projs, int32_t n_proj, int32_t n_ids);

/**
 * sumsq[i] = sum of grad^2 over adapter i's elements in all the projections,
 * for the listed ids (device fp32 [n_adapters]; others are not written); with
 * accumulate != 0 it is added to what sumsq[i] holds, so that a norm can span
 * several calls.  Squares are fp32, summed in an order that the projections fix:
 * an adapter's sum does not depend on what is listed beside it.
 */
lora_status_t lora_grad_sumsq(const lora_train_proj_t* projs, int32_t n_proj, const int32_t* ids,
                              int32_t n_ids, int32_t accumulate, float* sumsq, void* workspace,
                              size_t workspace_bytes, int32_t* dev_err, lora_stream_t stream);

/* Flags of lora_adamw_step. */
#define LORA_ADAMW_ZERO_GRAD 1 /* clear the gradient of what was stepped, in the same pass */

/**
 * One AdamW step of the listed adapters, in place: with h = hyper[i],
 *     c = min(1, max_norm / (|grad_scale| sqrt(sumsq[i]) + 1e-6)),  1 without sumsq
 *     g = grad_scale * c * grad
 *     m = beta1 m + (1 - beta1) g;    v = beta2 v + (1 - beta2) g^2
 *     w = w (1 - lr wd) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * in fp32, the update taking m and v before they are rounded to codes.  w is
 * master (and the pool takes bf16(w)), or without master the pool's bf16,
 * rounded to nearest.  sumsq: device fp32 [n_adapters] or NULL; an adapter whose
 * sumsq is not finite keeps its weights, state and gradient and sets
 * LORA_DERR_NONFINITE.  (Without sumsq a gradient that is not finite spoils its
 * element, and with LORA_STATE_E4M3 an infinite one its block of 64.)
 */
lora_status_t lora_adamw_step(const lora_train_proj_t* projs, int32_t n_proj, int32_t state,
                              const int32_t* ids, int32_t n_ids, const lora_adamw_hyper_t* hyper,
                              const float* sumsq, uint32_t flags, int32_t* dev_err, lora_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_TRAIN_H */
