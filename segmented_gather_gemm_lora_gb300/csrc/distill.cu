// The distillation loss (lora_train.h).
//
// With d = log p - log q of an outcome, a term of a divergence is
//     KL(p | q): p log(p / q) - p + q = p h(-d),   h(x) = e^x - 1 - x,
// which is never negative (outcomes of p and of q both add up to 1).  The gradient of kd
// with respect to a logit of an outcome is q / temperature (e - C):
//     forward: e = 1 - p / q,            C = 0
//     reverse: e = -d,                   C = sum of q e over the outcomes
//     jsd:     e = -(1 - mix) log(m / q), C likewise
// where q is the logit's own share and e its outcome's.
#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "lora_train.h"
#include "rows.cuh"

namespace lora {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// ----------------------------------------------------------------- divergence --

// p log(p / m) - p + m with x = log(m / p): p h(x).
__device__ __forceinline__ float term(float p, float m, float x) {
  if (p == 0.f) return m;
  if (fabsf(x) < 0.35f) {  // e^x - 1 - x by its series: the next term is 1e-7 of the sum
    const float s = fmaf(x, fmaf(x, fmaf(x, fmaf(x, fmaf(x, 1.f / 5040.f, 1.f / 720.f), 1.f / 120.f), 1.f / 24.f), 1.f / 6.f), 0.5f);
    return p * (x * x) * s;
  }
  if (fabsf(x) < 4.f) return p * (expm1f(x) - x);
  return m - p - p * x;
}

// One outcome of probabilities e^lp (teacher) and e^lq (student).
struct Outcome {
  float kd;     // its term
  float slope;  // e
  float mass;   // q e, of C
  float share;  // q (e - C) without C: for forward exact where p and q are close
};
__device__ __forceinline__ Outcome outcome(int kind, float mix, float lp, float lq) {
  const float p = expf(lp), q = expf(lq), d = lp - lq;
  if (p == 0.f && q == 0.f) return Outcome{0.f, 0.f, 0.f, 0.f};
  Outcome o;
  if (kind == LORA_DISTILL_FORWARD) {
    o.kd = p == 0.f ? q : q == 0.f ? INF_F : term(p, q, -d);
    o.slope = -expm1f(d);
    o.mass = 0.f;
    o.share = d < 1.f ? q * o.slope : q - p;
  } else if (kind == LORA_DISTILL_REVERSE) {
    o.kd = q == 0.f ? p : p == 0.f ? INF_F : term(q, p, d);
    o.slope = -d;
    o.mass = o.share = q == 0.f ? 0.f : q * -d;
  } else {
    // u = log(m / q), v = log(m / p)
    float u, v;
    if (d > 0.f) {
      v = log1pf((1.f - mix) * expm1f(-d));
      u = d + v;
    } else {
      u = log1pf(mix * expm1f(d));
      v = u - d;
    }
    const float m = mix * p + (1.f - mix) * q;
    o.kd = mix * term(p, m, v) + (1.f - mix) * term(q, m, u);
    o.slope = -(1.f - mix) * u;
    o.mass = o.share = q == 0.f ? 0.f : q * o.slope;
  }
  return o;
}

// ---------------------------------------------------------------------- rows --

struct DistillArgs {
  const void* logits;
  long long ld;
  const int32_t* ids;
  const float* values;
  const float* tail;
  const int32_t* labels;
  const float* weight;
  int T, V, k;
  lora_distill_opts_t opt;
  float* loss;
  float* kd;
  float* ce;
  void* dlogits;
  long long ldd;
  int32_t* err;
};

__device__ __forceinline__ float block_max(float x, float* sh) {
  x = warp_max(x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
  __syncthreads();
  x = sh[0];
  for (int i = 1; i < kWarps; ++i) x = fmaxf(x, sh[i]);
  return x;
}
__device__ __forceinline__ float block_add(float x, float* sh) {
  x = warp_add(x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
  __syncthreads();
  x = sh[0];
  for (int i = 1; i < kWarps; ++i) x += sh[i];
  return x;
}

// A CTA a row; a bit a logit says whether it is listed.
template <typename E>
__global__ void __launch_bounds__(kThreads) distill_kernel(const __grid_constant__ DistillArgs a) {
  extern __shared__ uint32_t bits[];
  __shared__ float sh[kWarps];
  __shared__ int bad;
  pdl_wait_then_release();
  const int t = blockIdx.x, tid = threadIdx.x, V = a.V;
  const E* row = static_cast<const E*>(a.logits) + (long long)t * a.ld;
  E* out = a.dlogits == nullptr ? nullptr : static_cast<E*>(a.dlogits) + (long long)t * a.ldd;
  for (int i = tid; i < (V + 31) / 32; i += kThreads) bits[i] = 0;
  if (tid == 0) bad = 0;
  __syncthreads();
  int id = tid < a.k ? a.ids[(long long)t * a.k + tid] : -1;
  float value = id >= 0 ? a.values[(long long)t * a.k + tid] : -INF_F;
  if (value == -INF_F) id = -1;
  const int label = a.labels == nullptr ? -1 : a.labels[t];
  const bool counts = a.labels == nullptr || label >= 0;
  if (counts) {
    if (id >= V || (a.labels != nullptr && label >= V)) bad = 1;
    else if (id >= 0 && (atomicOr(&bits[id >> 5], 1u << (id & 31)) >> (id & 31) & 1)) bad = 1;
  }
  __syncthreads();
  const float w = a.weight == nullptr ? 1.f : a.weight[t];
  if (!counts || bad) {
    if (tid == 0 && bad) report(a.err, LORA_DERR_BAD_LABEL);
    if (out != nullptr)
      for (int v = tid; v < V; v += kThreads) out[v] = Elem<E>::put(0.f);
    if (tid == 0) {
      a.loss[t] = 0.f;
      if (a.kd != nullptr) a.kd[t] = 0.f;
      if (a.ce != nullptr) a.ce[t] = 0.f;
    }
    return;
  }
  const float inv = 1.f / a.opt.temperature;
  // the student
  float top = -INF_F;
  for (int v = tid; v < V; v += kThreads) top = fmaxf(top, Elem<E>::get(row[v]));
  top = base_of(block_max(top, sh));
  float rest = 0.f, all = 0.f;
  for (int v = tid; v < V; v += kThreads) {
    const float x = Elem<E>::get(row[v]) - top;
    if (!(bits[v >> 5] >> (v & 31) & 1)) rest += expf(x * inv);
    if (a.opt.ce_weight > 0.f) all += expf(x);
  }
  rest = block_add(rest, sh);
  if (a.opt.ce_weight > 0.f) all = block_add(all, sh);
  const float x = id >= 0 ? Elem<E>::get(row[id]) - top : 0.f, xl = label >= 0 ? Elem<E>::get(row[label]) - top : 0.f;
  const float total = rest + block_add(id >= 0 ? expf(x * inv) : 0.f, sh), lt = logf(total);
  // the teacher
  const float tail = a.tail == nullptr ? -INF_F : a.tail[t];
  const float high = base_of(fmaxf(block_max(value * inv, sh), tail));
  const float mass = block_add(id >= 0 ? expf(value * inv - high) : 0.f, sh) + expf(tail - high), lm = logf(mass);
  Outcome o{0.f, 0.f, 0.f, 0.f}, r = o;
  if (mass != 0.f && total != 0.f) {
    if (id >= 0) o = outcome(a.opt.kind, a.opt.mix, value * inv - high - lm, x * inv - lt);
    r = outcome(a.opt.kind, a.opt.mix, tail - high - lm, logf(rest) - lt);
  }
  const float kd = block_add(o.kd, sh) + r.kd, C = block_add(o.mass, sh) + r.mass;
  bool none = total == 0.f;  // nothing is visible
  const float ce = a.opt.ce_weight > 0.f ? (none ? INF_F : logf(all) - xl) : 0.f;
  if (tid == 0) {
    const float kdv = none && mass > 0.f ? INF_F : kd;
    a.loss[t] = w == 0.f ? 0.f : w * ((a.opt.kd_weight > 0.f ? a.opt.kd_weight * kdv : 0.f) + (a.opt.ce_weight > 0.f ? a.opt.ce_weight * ce : 0.f));
    if (a.kd != nullptr) a.kd[t] = kdv;
    if (a.ce != nullptr) a.ce[t] = ce;
  }
  if (out == nullptr) return;
  __syncthreads();
  none = none || w == 0.f;
  const bool zero = fabsf(C) == INF_F;
  const float gs = a.opt.grad_scale * w, kw = gs * a.opt.kd_weight * inv, cw = a.opt.ce_weight > 0.f ? gs * a.opt.ce_weight : 0.f;
  const float slope = rest > 0.f ? r.slope - C : 0.f;
  const float mine = id >= 0 ? o.share - (a.opt.kind == LORA_DISTILL_FORWARD ? 0.f : expf(x * inv - lt) * C) : 0.f;
  for (int v = tid; v < V; v += kThreads) {
    const float y = Elem<E>::get(row[v]) - top;
    float g = zero ? 0.f : kw * slope * expf(y * inv - lt);
    if (cw != 0.f && !none) g += cw * (expf(y) / all - (v == label ? 1.f : 0.f));
    out[v] = Elem<E>::put(none ? 0.f : g);
  }
  __syncthreads();
  if (id >= 0 && !none) {
    float g = zero ? 0.f : kw * mine;
    if (cw != 0.f) g += cw * (expf(x) / all - (id == label ? 1.f : 0.f));
    out[id] = Elem<E>::put(g);
  }
}

}  // namespace

}  // namespace lora

using namespace lora;

extern "C" {

lora_status_t lora_distill_loss(const void* logits, int64_t ld, int32_t dtype, const int32_t* ids, const float* values,
                                const float* tail, int32_t k, const int32_t* labels, const float* weight, int32_t T,
                                int32_t V, const lora_distill_opts_t* opts, float* loss, float* kd, float* ce,
                                void* dlogits, int64_t ldd, int32_t* dev_err, lora_stream_t stream) {
  lora_status_t st = check_logits(logits, ld, dtype, labels != nullptr ? labels : ids, T, V);
  if (st != LORA_OK) return st;
  if (opts == nullptr || k < 1) return LORA_ERR_INVALID_ARG;
  if (k > LORA_TOPK_MAX) return LORA_ERR_UNSUPPORTED;
  if (opts->kind != LORA_DISTILL_FORWARD && opts->kind != LORA_DISTILL_REVERSE && opts->kind != LORA_DISTILL_JSD)
    return LORA_ERR_INVALID_ARG;
  if (!(opts->temperature > 0.f) || opts->temperature == INFINITY) return LORA_ERR_INVALID_ARG;
  if (opts->kind == LORA_DISTILL_JSD && !(opts->mix > 0.f && opts->mix < 1.f)) return LORA_ERR_INVALID_ARG;
  if (!(opts->kd_weight >= 0.f) || !(opts->ce_weight >= 0.f)) return LORA_ERR_INVALID_ARG;
  if ((st = check_grad(logits, ld, dtype, dlogits, ldd, T, V)) != LORA_OK || T == 0) return st;
  if (!f32_ok(ids) || !f32_ok(values) || !f32_ok(loss)) return LORA_ERR_INVALID_ARG;
  if (!aligned_to(tail, 4) || !aligned_to(weight, 4) || !aligned_to(kd, 4) || !aligned_to(ce, 4)) return LORA_ERR_INVALID_ARG;
  if (opts->kind == LORA_DISTILL_REVERSE && tail == nullptr) return LORA_ERR_INVALID_ARG;
  if (opts->ce_weight > 0.f && labels == nullptr) return LORA_ERR_INVALID_ARG;
  DistillArgs a;
  memset(&a, 0, sizeof(a));
  a.logits = logits;
  a.ld = ld;
  a.ids = ids;
  a.values = values;
  a.tail = tail;
  a.labels = labels;
  a.weight = weight;
  a.T = T;
  a.V = V;
  a.k = k;
  a.opt = *opts;
  a.loss = loss;
  a.kd = kd;
  a.ce = ce;
  a.dlogits = dlogits;
  a.ldd = ldd;
  a.err = dev_err;
  const void* f = dtype == LORA_LOGITS_BF16 ? (const void*)distill_kernel<uint16_t> : (const void*)distill_kernel<float>;
  const size_t smem = ((size_t)V + 31) / 32 * 4;
  if (smem > 200000) return LORA_ERR_UNSUPPORTED;
  if (ensure_smem_attr(f, smem) != cudaSuccess) return LORA_ERR_CUDA;
  return launch_pdl(f, dim3((unsigned)T), dim3(kThreads), smem, (cudaStream_t)stream, 0, &a) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

}  // extern "C"
