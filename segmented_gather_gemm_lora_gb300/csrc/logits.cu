// Losses on logits (lora_train.h): per-token log-probabilities, the paired
// preference loss and the clipped policy loss, with the gradient of the logits.
//
// A row of V logits belongs to a cluster of 1, 2, 4 or 8 CTAs, each taking a
// share of its 16-byte vectors.  A row's sum of exponentials is kept as its
// maximum m and s = sum of exp(x - m): lse = m + log s, logp = (x - m) - log s,
// and a softmax entry is 2^((x - m) log2 e - log2 s).  The difference x - m comes
// first, so nothing is lost where logits are large (rows masked with -1e30 or
// the type's lowest value included).
#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "lora_train.h"

namespace lora {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;      // vectors in flight a thread
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;
#define INF_F __int_as_float(0x7f800000)

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One element and a 16-byte vector of a row's type.
template <typename E>
struct Elem;
template <>
struct Elem<uint16_t> {
  static constexpr int kN = 8;
  static constexpr uint32_t kMinusInf = 0xff80ff80u;
  static __device__ __forceinline__ float get(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ uint16_t put(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) { unpack8(v, f); }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Elem<float> {
  static constexpr int kN = 4;
  static constexpr uint32_t kMinusInf = 0xff800000u;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// A running sum of exponentials: its maximum m, and s = sum of exp(x - base(m)).
struct Sum {
  float m, s;
};
__device__ __forceinline__ float base_of(float m) { return fabsf(m) == INF_F ? 0.f : m; }
// The sum of two.  An empty one is {-inf, 0}.
__device__ __forceinline__ Sum join(const Sum& x, const Sum& y) {
  Sum r;
  r.m = fmaxf(x.m, y.m);
  const float base = base_of(r.m);
  r.s = x.s * ex2((x.m - base) * kLog2e) + y.s * ex2((y.m - base) * kLog2e);
  return r;
}

// A row cut for this CTA: vectors [v0, v1) of its 16-byte-aligned middle; the
// elements before it go to the first CTA of the cluster, those after to the last.
template <typename E>
struct Cut {
  const E* row;
  int head, nvec, tail0;  // elements before the middle; its vectors; first element after it
  int v0, v1;
  bool first, last;
};
template <typename E>
__device__ __forceinline__ Cut<E> cut_row(const E* row, int V, int rank, int n) {
  constexpr int kN = Elem<E>::kN;
  Cut<E> c;
  c.row = row;
  c.head = min(V, (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(E)));
  c.nvec = (V - c.head) / kN;
  c.tail0 = c.head + c.nvec * kN;
  const int per = (c.nvec + n - 1) / n;
  c.v0 = min(c.nvec, rank * per);
  c.v1 = min(c.nvec, c.v0 + per);
  c.first = rank == 0;
  c.last = rank == n - 1;
  return c;
}

// The edge element of this thread: its index in the row, or -1.
template <typename E>
__device__ __forceinline__ int edge_of(const Cut<E>& c, int V) {
  const int t = threadIdx.x;
  if (c.first && t < c.head) return t;
  if (c.last && t >= 32 && t - 32 < V - c.tail0) return c.tail0 + t - 32;
  return -1;
}

// This thread's part of the row's sum.
template <typename E>
__device__ __forceinline__ Sum thread_sum(const Cut<E>& c, int V) {
  constexpr int kN = Elem<E>::kN;
  const uint4* mid = reinterpret_cast<const uint4*>(c.row + c.head);
  Sum t{-INF_F, 0.f};
  for (int i = c.v0 + (int)threadIdx.x; i < c.v1; i += kUnroll * kThreads) {
    uint4 r[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int k = i + u * kThreads;
      r[u] = k < c.v1 ? mid[k] : make_uint4(Elem<E>::kMinusInf, Elem<E>::kMinusInf, Elem<E>::kMinusInf, Elem<E>::kMinusInf);
    }
    float top = -INF_F;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float f[kN];
      Elem<E>::unpack(r[u], f);
#pragma unroll
      for (int k = 0; k < kN; ++k) top = fmaxf(top, f[k]);
    }
    const float m = fmaxf(t.m, top), base = base_of(m);
    float part = 0.f;  // a sum of its own: the running sum takes one addition a round
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float f[kN];
      Elem<E>::unpack(r[u], f);
#pragma unroll
      for (int k = 0; k < kN; ++k) part += ex2((f[k] - base) * kLog2e);
    }
    t.s = t.s * ex2((t.m - base) * kLog2e) + part;
    t.m = m;
  }
  const int e = edge_of(c, V);
  if (e >= 0) {
    const float x = Elem<E>::get(c.row[e]);
    t = join(t, Sum{x, x == x ? (x == -INF_F ? 0.f : x == INF_F ? x : 1.f) : x});
  }
  return t;
}

struct RowShared {
  Sum warp[kThreads / 32];
  Sum cta[kMaxCluster];
  float coef;
};

// A peer's shared memory may be written once that CTA runs: each arrives when it
// starts on the row and waits before its first store to a peer.
__device__ __forceinline__ void cluster_started(int n) {
  if (n > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}

// The row's sum over the CTA, then the cluster (which has arrived by
// cluster_started).
__device__ __forceinline__ Sum row_sum(Sum t, RowShared* sh, int rank, int n) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const Sum o{__shfl_xor_sync(0xffffffffu, t.m, d), __shfl_xor_sync(0xffffffffu, t.s, d)};
    t = join(t, o);
  }
  if ((threadIdx.x & 31) == 0) sh->warp[threadIdx.x >> 5] = t;
  __syncthreads();
  t = sh->warp[0];
#pragma unroll
  for (int k = 1; k < kThreads / 32; ++k) t = join(t, sh->warp[k]);
  if (n > 1) {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (threadIdx.x < (unsigned)n) {
      const uint32_t at = mapa(smem_u32(&sh->cta[rank]), threadIdx.x);
      st_dsmem_u32(at, __float_as_uint(t.m));
      st_dsmem_u32(at + 4, __float_as_uint(t.s));
    }
    cluster_sync();
    t = sh->cta[0];
    for (int k = 1; k < n; ++k) t = join(t, sh->cta[k]);
  }
  return t;
}

// Gradient entries coef * ([v = label] - 2^((x - base) log2 e - l2)) of this CTA's
// share (l2: log2 of the row's sum);
// zeros when `zero` (the logits are not read).
template <typename E>
__device__ __forceinline__ void write_grad(const Cut<E>& c, E* out, int V, int label, float base, float l2, float coef, bool zero) {
  constexpr int kN = Elem<E>::kN;
  const uint4* mid = reinterpret_cast<const uint4*>(c.row + c.head);
  E* const dst = out + c.head;
  // vectors where the output row sits on the boundary of the logits row, else
  // element by element
  const bool wide = (reinterpret_cast<uintptr_t>(dst) & 15) == 0;
  for (int i = c.v0 + (int)threadIdx.x; i < c.v1; i += kUnroll * kThreads) {
    uint4 r[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int k = i + u * kThreads;
      r[u] = !zero && k < c.v1 ? mid[k] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int k = i + u * kThreads;
      if (k >= c.v1) break;
      if (!zero) {
        float f[kN];
        Elem<E>::unpack(r[u], f);
#pragma unroll
        for (int j = 0; j < kN; ++j) f[j] = -coef * ex2(fmaf(f[j] - base, kLog2e, -l2));
        const int at = label - c.head - k * kN;
        if ((unsigned)at < (unsigned)kN) {
#pragma unroll
          for (int j = 0; j < kN; ++j)
            if (j == at) f[j] += coef;
        }
        r[u] = Elem<E>::pack(f);
      }
      if (wide) {
        reinterpret_cast<uint4*>(dst)[k] = r[u];
      } else {
        float f[kN];
        Elem<E>::unpack(r[u], f);
#pragma unroll
        for (int j = 0; j < kN; ++j) dst[k * kN + j] = Elem<E>::put(f[j]);
      }
    }
  }
  const int e = edge_of(c, V);
  if (e >= 0) {
    float g = 0.f;
    if (!zero) g = (e == label ? coef : 0.f) - coef * ex2(fmaf(Elem<E>::get(c.row[e]) - base, kLog2e, -l2));
    out[e] = Elem<E>::put(g);
  }
}

struct RowArgs {
  const void* logits;
  long long ld;
  const int32_t* labels;
  int V;
  float* logp;
  float* lse;   // or NULL
  float* top;   // for the gradient pass, or NULL: the sum's base (-inf: nothing visible),
  float* log2s;  // log2 of its sum
  float* coef;  // and its gradient coefficient (the sum's pass sets it to 0)
  void* dlogits;
  long long ldd;
  // policy loss
  const float* old_logp;
  const float* ref_logp;
  const float* advantage;
  const float* weight;
  float* loss;
  float* kl;
  lora_policy_opts_t opt;
  int32_t* err;
};

// The label of the row, -1 if the row does not count.
__device__ __forceinline__ int row_label(const RowArgs& a, int t, bool lead) {
  const int label = a.labels[t];
  if (label >= a.V) {
    if (lead) report(a.err, LORA_DERR_BAD_LABEL);
    return -1;
  }
  return label < 0 ? -1 : label;
}

// Nothing of the row is visible (a NaN among the masked entries is).
__device__ __forceinline__ bool empty(const Sum& t) { return t.m == -INF_F && t.s == 0.f; }

__device__ __forceinline__ float label_logp(float x, const Sum& t) {
  return empty(t) ? -INF_F : (x - base_of(t.m)) - logf(t.s);
}

// logp and lse of each row: one read of the logits.
template <typename E>
__global__ void __launch_bounds__(kThreads) row_sum_kernel(const __grid_constant__ RowArgs a) {
  __shared__ RowShared sh;
  const int n = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  pdl_wait_then_release();
  const int t = (int)cluster_id_x();
  const bool lead = rank == 0 && threadIdx.x == 0;
  const int label = row_label(a, t, lead);
  if (lead && a.coef != nullptr) a.coef[t] = 0.f;
  if (label < 0) {
    if (lead) {
      a.logp[t] = 0.f;
      if (a.lse != nullptr) a.lse[t] = 0.f;
    }
    return;
  }
  const E* row = static_cast<const E*>(a.logits) + (long long)t * a.ld;
  const Cut<E> c = cut_row(row, a.V, rank, n);
  cluster_started(n);
  const Sum r = row_sum(thread_sum(c, a.V), &sh, rank, n);
  if (lead) {
    a.logp[t] = label_logp(Elem<E>::get(row[label]), r);
    if (a.lse != nullptr) a.lse[t] = base_of(r.m) + logf(r.s);
    if (a.top != nullptr) {
      a.top[t] = empty(r) ? r.m : base_of(r.m);
      a.log2s[t] = log2f(r.s);
    }
  }
}

// The gradient rows from the rows' L and coefficients.
template <typename E>
__global__ void __launch_bounds__(kThreads) row_grad_kernel(const __grid_constant__ RowArgs a) {
  const int n = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  pdl_wait_then_release();
  const int t = (int)cluster_id_x();
  const int label = row_label(a, t, false);
  const float coef = a.coef[t];
  const bool zero = label < 0 || coef == 0.f || a.top[t] == -INF_F;
  const Cut<E> c = cut_row(static_cast<const E*>(a.logits) + (long long)t * a.ld, a.V, rank, n);
  write_grad(c, static_cast<E*>(a.dlogits) + (long long)t * a.ldd, a.V, label,
             zero ? 0.f : a.top[t], zero ? 0.f : a.log2s[t], coef, zero);
}

// The policy loss of each row and its gradient row: the coefficient depends on
// the row alone, so one kernel reads the row, sums it and writes its gradient.
template <typename E>
__global__ void __launch_bounds__(kThreads) policy_kernel(const __grid_constant__ RowArgs a) {
  __shared__ RowShared sh;
  const int n = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  pdl_wait_then_release();
  const int t = (int)cluster_id_x();
  const bool lead = rank == 0 && threadIdx.x == 0;
  const int label = row_label(a, t, lead);
  const E* row = static_cast<const E*>(a.logits) + (long long)t * a.ld;
  E* out = a.dlogits == nullptr ? nullptr : static_cast<E*>(a.dlogits) + (long long)t * a.ldd;
  const Cut<E> c = cut_row(row, a.V, rank, n);
  if (label < 0) {
    if (lead) {
      a.logp[t] = a.loss[t] = 0.f;
      if (a.kl != nullptr) a.kl[t] = 0.f;
    }
    if (out != nullptr) write_grad(c, out, a.V, -1, 0.f, 0.f, 0.f, true);
    return;
  }
  // before anyone writes the gradient, which may take the logits' place
  const float x = threadIdx.x == 0 ? Elem<E>::get(row[label]) : 0.f;
  cluster_started(n);
  const Sum r = row_sum(thread_sum(c, a.V), &sh, rank, n);
  if (threadIdx.x == 0) {
    const float lp = label_logp(x, r);
    const float w = a.weight == nullptr ? 1.f : a.weight[t];
    const float adv = a.advantage[t], q = expf(lp - a.old_logp[t]);
    const float free_ = q * adv, held = fminf(fmaxf(q, 1.f - a.opt.clip_low), 1.f + a.opt.clip_high) * adv;
    float kl = 0.f, slope = 0.f;
    if (a.opt.kl_coef > 0.f) {
      const float d = a.ref_logp[t] - lp, g = expm1f(d);
      kl = d == INF_F ? d : g - d;
      slope = a.opt.kl_coef * g;
    }
    const bool open = free_ <= held;
    float coef = 0.f, loss = 0.f;
    if (w != 0.f) {
      loss = w * (a.opt.kl_coef * kl - (open ? free_ : held));
      coef = -a.opt.grad_scale * w * (slope + (open ? free_ : 0.f));
    }
    sh.coef = coef;
    if (rank == 0) {
      a.logp[t] = lp;
      a.loss[t] = loss;
      if (a.kl != nullptr) a.kl[t] = kl;
    }
  }
  if (out == nullptr) return;
  __syncthreads();
  const float coef = sh.coef;
  write_grad(c, out, a.V, label, base_of(r.m), log2f(r.s), coef, coef == 0.f || empty(r));
}

struct PairArgs {
  const int32_t* labels;
  const float* logp;
  const float* ref;
  const int32_t* indptr;
  int n_pairs, T, V;
  lora_pref_opts_t opt;
  float* loss;
  float* seq_logp;
  float* coef;
  int32_t* err;
};

__device__ __forceinline__ double cta_sum(double x, double* sh) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
  __syncthreads();
  double t = 0;
#pragma unroll
  for (int k = 0; k < kThreads / 32; ++k) t += sh[k];
  return t;
}

__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }
__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

// One CTA a pair: the two sequences' sums (in double, threads and warps in a
// fixed order), the loss, and its coefficient for every counted row.
__global__ void __launch_bounds__(kThreads) pair_kernel(const __grid_constant__ PairArgs a) {
  __shared__ double sh[kThreads / 32];
  pdl_wait_then_release();
  const int p = blockIdx.x, tid = threadIdx.x;
  int bad = 0;
  for (int k = tid; k <= 2 * a.n_pairs; k += kThreads) {
    const int hi = a.indptr[k], lo = k > 0 ? a.indptr[k - 1] : 0;
    bad |= hi < lo || hi > a.T;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      if (p == 0) report(a.err, LORA_DERR_BAD_SEQ);
      a.loss[p] = 0.f;
      if (a.seq_logp != nullptr) a.seq_logp[2 * p] = a.seq_logp[2 * p + 1] = 0.f;
    }
    return;
  }
  double ratio[2];
  float share[2];
  for (int s = 0; s < 2; ++s) {
    const int t0 = a.indptr[2 * p + s], t1 = a.indptr[2 * p + s + 1];
    double lp = 0, d = 0, cnt = 0;
    for (int t = t0 + tid; t < t1; t += kThreads) {
      const int label = a.labels[t];
      if (label < 0 || label >= a.V) continue;
      const float x = a.logp[t];
      lp += x;
      d += a.ref == nullptr ? x : (double)x - a.ref[t];
      cnt += 1;
    }
    lp = cta_sum(lp, sh);
    d = cta_sum(d, sh);
    cnt = cta_sum(cnt, sh);
    const bool mean = a.opt.flags & LORA_PREF_AVERAGE;
    ratio[s] = mean && cnt > 0 ? d / cnt : d;
    share[s] = mean && cnt > 0 ? (float)(1.0 / cnt) : 1.f;
    if (tid == 0 && a.seq_logp != nullptr) a.seq_logp[2 * p + s] = (float)lp;
  }
  const double D = ratio[0] - ratio[1];
  const float z = (float)(a.opt.beta * D - a.opt.margin);
  float loss, slope;  // slope: dloss / dD
  if (a.opt.kind == LORA_PREF_SIGMOID) {
    const float e = a.opt.label_smoothing;
    loss = slope = 0.f;  // a term of weight 0 is left out: its logarithm may be infinite
    if (e < 1.f) {
      loss = (1.f - e) * softplus(-z);
      slope = (e - 1.f) * sigmoid(-z);
    }
    if (e > 0.f) {
      loss += e * softplus(z);
      slope += e * sigmoid(z);
    }
    slope *= a.opt.beta;
  } else if (a.opt.kind == LORA_PREF_HINGE) {
    loss = z < 1.f || z != z ? 1.f - z : 0.f;
    slope = z < 1.f ? -a.opt.beta : z != z ? z : 0.f;
  } else {
    const float off = (float)(D - 0.5 / a.opt.beta);
    loss = off * off;
    slope = 2.f * off;
  }
  if (tid == 0) a.loss[p] = loss;
  if (a.coef == nullptr) return;
  for (int s = 0; s < 2; ++s) {
    const float coef = (s == 0 ? slope : -slope) * share[s] * a.opt.grad_scale;
    const int t0 = a.indptr[2 * p + s], t1 = a.indptr[2 * p + s + 1];
    for (int t = t0 + tid; t < t1; t += kThreads) a.coef[t] = coef;
  }
}

// ------------------------------------------------------------------- host --

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool f32_ok(const void* p) { return p != nullptr && aligned_to(p, 4); }

bool overlap(const void* a, long long abytes, const void* b, long long bbytes) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + (uintptr_t)bbytes && b0 < a0 + (uintptr_t)abytes;
}

lora_status_t check_logits(const void* logits, long long ld, int dtype, const int32_t* labels, int T, int V) {
  if (T < 0 || V < 1) return LORA_ERR_INVALID_ARG;
  if (dtype != LORA_LOGITS_BF16 && dtype != LORA_LOGITS_F32) return LORA_ERR_INVALID_ARG;
  if (T == 0) return LORA_OK;
  if (ld < V || ld > (1LL << 40) / T) return LORA_ERR_INVALID_ARG;
  const size_t b = dtype == LORA_LOGITS_BF16 ? 2 : 4;
  if (logits == nullptr || !aligned_to(logits, b) || !f32_ok(labels)) return LORA_ERR_INVALID_ARG;
  return LORA_OK;
}

// The gradient's place: the logits' own (same rows), or apart from them.
lora_status_t check_grad(const void* logits, long long ld, int dtype, const void* d, long long ldd, int T, int V) {
  if (d == nullptr || T == 0) return LORA_OK;
  const long long b = dtype == LORA_LOGITS_BF16 ? 2 : 4;
  if (ldd < V || ldd > (1LL << 40) / T || !aligned_to(d, b)) return LORA_ERR_INVALID_ARG;
  if (d == logits && ldd == ld) return LORA_OK;
  const long long rows = T - 1;
  return overlap(logits, (rows * ld + V) * b, d, (rows * ldd + V) * b) ? LORA_ERR_INVALID_ARG : LORA_OK;
}

// CTAs a row: more while the rows alone leave SMs idle and each CTA still has a
// vector for every thread.
int row_ctas(int T, int V, int dtype) {
  const int per = kThreads * (dtype == LORA_LOGITS_BF16 ? 8 : 4);
  int n = 1;
  while (n < kMaxCluster && (long long)T * n < 2LL * sm_count() && V / (2 * n) >= per) n *= 2;
  return n;
}

enum RowKind { kRowSum, kRowGrad, kRowPolicy };

lora_status_t launch_rows(int kind, int dtype, RowArgs* a, int T, cudaStream_t s) {
  const bool h = dtype == LORA_LOGITS_BF16;
  const void* f = kind == kRowSum    ? (h ? (const void*)row_sum_kernel<uint16_t> : (const void*)row_sum_kernel<float>)
                  : kind == kRowGrad ? (h ? (const void*)row_grad_kernel<uint16_t> : (const void*)row_grad_kernel<float>)
                                     : (h ? (const void*)policy_kernel<uint16_t> : (const void*)policy_kernel<float>);
  const int n = row_ctas(T, a->V, dtype);
  if ((long long)T * n > 0x7fffffffLL) return LORA_ERR_UNSUPPORTED;
  return launch_pdl(f, dim3((unsigned)(T * n)), dim3(kThreads), 0, s, n, a) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

size_t pref_floats(int T) { return ((size_t)T + 3) / 4 * 4; }

}  // namespace

}  // namespace lora

using namespace lora;

extern "C" {

lora_status_t lora_token_logprobs(const void* logits, int64_t ld, int32_t dtype, const int32_t* labels, int32_t T,
                                  int32_t V, float* logp, float* lse, int32_t* dev_err, lora_stream_t stream) {
  const lora_status_t st = check_logits(logits, ld, dtype, labels, T, V);
  if (st != LORA_OK || T == 0) return st;
  if (!f32_ok(logp) || !aligned_to(lse, 4)) return LORA_ERR_INVALID_ARG;
  RowArgs a;
  memset(&a, 0, sizeof(a));
  a.logits = logits;
  a.ld = ld;
  a.labels = labels;
  a.V = V;
  a.logp = logp;
  a.lse = lse;
  a.err = dev_err;
  return launch_rows(kRowSum, dtype, &a, T, (cudaStream_t)stream);
}

size_t lora_preference_workspace_bytes(int32_t T, int32_t n_pairs) {
  if (T < 0 || n_pairs < 0) return 0;
  return 4 * pref_floats(T) * sizeof(float) + 16;
}

lora_status_t lora_preference_loss(const void* logits, int64_t ld, int32_t dtype, const int32_t* labels,
                                   const float* ref_logp, const int32_t* seq_indptr, int32_t n_pairs, int32_t T,
                                   int32_t V, const lora_pref_opts_t* opts, float* loss, float* seq_logp, void* dlogits,
                                   int64_t ldd, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                   lora_stream_t stream) {
  lora_status_t st = check_logits(logits, ld, dtype, labels, T, V);
  if (st != LORA_OK) return st;
  if (n_pairs < 0 || opts == nullptr) return LORA_ERR_INVALID_ARG;
  if (opts->kind != LORA_PREF_SIGMOID && opts->kind != LORA_PREF_HINGE && opts->kind != LORA_PREF_IPO)
    return LORA_ERR_INVALID_ARG;
  if (opts->flags & ~(uint32_t)LORA_PREF_AVERAGE) return LORA_ERR_INVALID_ARG;
  if (!(opts->beta > 0.f) || !(opts->label_smoothing >= 0.f && opts->label_smoothing <= 1.f)) return LORA_ERR_INVALID_ARG;
  if (n_pairs > 0 && (!f32_ok(seq_indptr) || !f32_ok(loss))) return LORA_ERR_INVALID_ARG;
  if (n_pairs > 0x3fffffff) return LORA_ERR_UNSUPPORTED;
  if (!aligned_to(ref_logp, 4) || !aligned_to(seq_logp, 4)) return LORA_ERR_INVALID_ARG;
  if ((st = check_grad(logits, ld, dtype, dlogits, ldd, T, V)) != LORA_OK) return st;
  if (T == 0 && n_pairs == 0) return LORA_OK;
  if (workspace == nullptr || !aligned_to(workspace, 16)) return LORA_ERR_INVALID_ARG;
  if (workspace_bytes < lora_preference_workspace_bytes(T, n_pairs)) return LORA_ERR_WORKSPACE;
  const cudaStream_t s = (cudaStream_t)stream;
  RowArgs a;
  memset(&a, 0, sizeof(a));
  a.logits = logits;
  a.ld = ld;
  a.labels = labels;
  a.V = V;
  a.logp = static_cast<float*>(workspace);
  a.top = a.logp + pref_floats(T);
  a.log2s = a.top + pref_floats(T);
  a.coef = a.log2s + pref_floats(T);
  a.dlogits = dlogits;
  a.ldd = ldd;
  a.err = dev_err;
  if (T > 0 && (st = launch_rows(kRowSum, dtype, &a, T, s)) != LORA_OK) return st;
  if (n_pairs > 0) {
    PairArgs p;
    memset(&p, 0, sizeof(p));
    p.labels = labels;
    p.logp = a.logp;
    p.ref = ref_logp;
    p.indptr = seq_indptr;
    p.n_pairs = n_pairs;
    p.T = T;
    p.V = V;
    p.opt = *opts;
    p.loss = loss;
    p.seq_logp = seq_logp;
    p.coef = dlogits == nullptr ? nullptr : a.coef;
    p.err = dev_err;
    if (launch_pdl((const void*)pair_kernel, dim3((unsigned)n_pairs), dim3(kThreads), 0, s, 0, &p) != cudaSuccess)
      return LORA_ERR_CUDA;
  }
  if (T == 0 || dlogits == nullptr) return LORA_OK;
  return launch_rows(kRowGrad, dtype, &a, T, s);
}

lora_status_t lora_policy_loss(const void* logits, int64_t ld, int32_t dtype, const int32_t* labels,
                               const float* old_logp, const float* ref_logp, const float* advantage,
                               const float* weight, int32_t T, int32_t V, const lora_policy_opts_t* opts, float* logp,
                               float* loss, float* kl, void* dlogits, int64_t ldd, int32_t* dev_err,
                               lora_stream_t stream) {
  lora_status_t st = check_logits(logits, ld, dtype, labels, T, V);
  if (st != LORA_OK) return st;
  if (opts == nullptr || !(opts->clip_low >= 0.f && opts->clip_low <= 1.f) || !(opts->clip_high >= 0.f) ||
      !(opts->kl_coef >= 0.f))
    return LORA_ERR_INVALID_ARG;
  if ((st = check_grad(logits, ld, dtype, dlogits, ldd, T, V)) != LORA_OK || T == 0) return st;
  if (!f32_ok(old_logp) || !f32_ok(advantage) || !f32_ok(logp) || !f32_ok(loss)) return LORA_ERR_INVALID_ARG;
  if (!aligned_to(ref_logp, 4) || !aligned_to(weight, 4) || !aligned_to(kl, 4)) return LORA_ERR_INVALID_ARG;
  if (opts->kl_coef > 0.f && ref_logp == nullptr) return LORA_ERR_INVALID_ARG;
  RowArgs a;
  memset(&a, 0, sizeof(a));
  a.logits = logits;
  a.ld = ld;
  a.labels = labels;
  a.V = V;
  a.logp = logp;
  a.dlogits = dlogits;
  a.ldd = ldd;
  a.old_logp = old_logp;
  a.ref_logp = ref_logp;
  a.advantage = advantage;
  a.weight = weight;
  a.loss = loss;
  a.kl = kl;
  a.opt = *opts;
  a.err = dev_err;
  return launch_rows(kRowPolicy, dtype, &a, T, (cudaStream_t)stream);
}

}  // extern "C"
