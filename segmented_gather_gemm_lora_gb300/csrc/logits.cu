// Losses on logits (lora_train.h): per-token log-probabilities, the paired
// preference loss and the clipped policy loss, with the gradient of the logits.
//
// A row's sum of exponentials is kept as its maximum m and s = sum of
// exp(x - m): lse = m + log s, logp = (x - m) - log s, and a softmax entry is
// 2^((x - m) log2 e - log2 s).  The difference x - m comes first, so nothing is
// lost where logits are large (rows masked with -1e30 or the type's lowest value
// included).
//
// Two forms of the row kernels, chosen by row_plan() below:
//  - streamed: a row is a cluster of 1, 2, 4 or 8 CTAs of 256 threads that read
//    it from global memory, again for its gradient where one is written;
//  - held: a row stays in the registers of a warp, a CTA or a cluster from its sum
//    to its gradient, so it is read once.  (Read twice, the rows in flight on the
//    GPU exceed its L2: of 2048 x 128256 bf16 the second read missed L2
//    throughout.)  The CTAs are persistent: starting one costs a microsecond or
//    two, the time of a row.
#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "lora_train.h"
#include "pairs.cuh"
#include "rows.cuh"

namespace lora {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;    // vectors a thread takes at once
constexpr int kMaxCluster = 8;

struct RowShared {
  uint64_t probe_bar;
  Sum part[kMaxCluster * kWarps];
};

// This thread's part of the row's sum.
template <typename E>
__device__ __forceinline__ Sum thread_sum(const Cut<E>& c, int V) {
  const uint4* mid = reinterpret_cast<const uint4*>(c.row + c.head);
  Sum t{-INF_F, 0.f};
  for (int i = c.v0 + (int)threadIdx.x; i < c.v1; i += kUnroll * kThreads) {
    uint4 r[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) r[u] = i + u * kThreads < c.v1 ? mid[i + u * kThreads] : low_vector<E>();
    t = add_vectors<E>(t, r);
  }
  const int e = edge_of(c, V, threadIdx.x);
  return e >= 0 ? add_one(t, Elem<E>::get(c.row[e])) : t;
}

// A peer's shared memory may be written once that CTA runs: each arrives when it
// starts on the row and waits before its first store to a peer.
__device__ __forceinline__ void cluster_started(int n) {
  if (n > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

// The row's sum over the cluster (which has arrived by cluster_started): each
// warp leaves its sum with every CTA, one barrier, and every warp joins them all.
__device__ __forceinline__ Sum row_sum(Sum t, RowShared* sh, int rank, int n) {
  t = warp_sum(t);
  const int lane = threadIdx.x & 31, slot = rank * kWarps + (threadIdx.x >> 5);
  if (n > 1) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (lane < n) {
      const uint32_t at = mapa(smem_u32(&sh->part[slot]), lane);
      st_dsmem_u32(at, __float_as_uint(t.m));
      st_dsmem_u32(at + 4, __float_as_uint(t.s));
    }
    cluster_sync();
  } else {
    if (lane == 0) sh->part[slot] = t;
    __syncthreads();
  }
  t = lane < n * kWarps ? sh->part[lane] : Sum{-INF_F, 0.f};
  if (lane + 32 < n * kWarps) t = join(t, sh->part[lane + 32]);
  return warp_sum(t);
}

// The gradient of a row: entry v is coef * ([v = label] - 2^((x - base) log2 e - l2)),
// l2 the log2 of the row's sum; `zero`: every entry 0 (the logits are not looked at).
// log2 e is one fp32 here: what that leaves out moves an entry by 1.3e-8 (x - base) of
// itself (2e-7 where it is 4e-8 of the row's largest) and is not added up over rows.
struct Grad {
  int label;
  float base, l2, coef;
  bool zero;
};

template <typename E>
__device__ __forceinline__ uint4 grad_vector(const uint4& x, const Grad& g) {
  constexpr int kPairs = Elem<E>::kPairs;
  const uint64_t nb = pair_of(-g.base, -g.base), hi = pair_of(kLog2e, kLog2e), nl = pair_of(-g.l2, -g.l2);
  const uint64_t nc = pair_of(-g.coef, -g.coef);
  uint64_t f[kPairs];
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    float a, b;
    split(fma2(add2(Elem<E>::pair(x, j), nb), hi, nl), a, b);
    f[j] = mul2(nc, pair_of(ex2(a), ex2(b)));
  }
  return Elem<E>::pack(f);
}

// The entry of one element x, and of the label's.
__device__ __forceinline__ float grad_entry(float x, const Grad& g, bool at_label) {
  return (at_label ? g.coef : 0.f) - g.coef * ex2(fmaf(x - g.base, kLog2e, -g.l2));
}

// Write the gradient of vector k of a row's middle (x: its logits): a vector
// where the output row sits on the boundary of the logits row, else element by
// element; then the label's entry over what the vector left there.
template <typename E>
__device__ __forceinline__ void put_vector(E* out, const Cut<E>& c, int k, const uint4& x, const Grad& g, bool wide) {
  constexpr int kN = Elem<E>::kN;
  E* const dst = out + c.head + (long long)k * kN;
  const uint4 r = g.zero ? make_uint4(0, 0, 0, 0) : grad_vector<E>(x, g);
  if (wide) {
    *reinterpret_cast<uint4*>(dst) = r;
  } else {
#pragma unroll
    for (int j = 0; j < kN; ++j) dst[j] = Elem<E>::entry(r, j);
  }
  const int at = g.label - c.head - k * kN;
  if (!g.zero && (unsigned)at < (unsigned)kN) dst[at] = Elem<E>::put(grad_entry(Elem<E>::get(Elem<E>::entry(x, at)), g, true));
}

template <typename E>
__device__ __forceinline__ void put_edge(E* out, const Cut<E>& c, int e, const Grad& g) {
  if (e >= 0) out[e] = Elem<E>::put(g.zero ? 0.f : grad_entry(Elem<E>::get(c.row[e]), g, e == g.label));
}

// Zeros in this CTA's share of a row, by kT threads.
template <typename E, int kT>
__device__ __forceinline__ void zero_row(const Cut<E>& c, E* out, int V, int id) {
  constexpr int kN = Elem<E>::kN;
  E* const dst = out + c.head + (long long)c.v0 * kN;
  const int nv = c.v1 - c.v0, e = edge_of(c, V, id);
  if (on_boundary(out, c)) {
    for (int k = id; k < nv; k += kT) reinterpret_cast<uint4*>(dst)[k] = make_uint4(0, 0, 0, 0);
  } else {
    for (int k = id; k < nv * kN; k += kT) dst[k] = Elem<E>::put(0.f);
  }
  if (e >= 0) out[e] = Elem<E>::put(0.f);
}

// This CTA's share of a gradient row, by kT threads, from global memory.
template <typename E, int kT>
__device__ __forceinline__ void write_grad(const Cut<E>& c, E* out, int V, const Grad& g) {
  const uint4* mid = reinterpret_cast<const uint4*>(c.row + c.head);
  const bool wide = on_boundary(out, c);
  for (int i = c.v0 + (int)threadIdx.x; i < c.v1; i += kUnroll * kT) {
    uint4 r[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) r[u] = !g.zero && i + u * kT < c.v1 ? mid[i + u * kT] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (i + u * kT < c.v1) put_vector(out, c, i + u * kT, r[u], g, wide);
  }
  put_edge(out, c, edge_of(c, V, threadIdx.x), g);
}

struct RowArgs {
  int T;
  const void* logits;
  long long ld;
  const int32_t* labels;
  int V;
  float* logp;
  float* lse;   // or NULL
  float* top;   // for the gradient pass, or NULL: the sum's base (-inf: nothing visible),
  float* log2s;  // log2 of its sum
  float* coef;  // and its gradient coefficient (the sums set it to 0, the pairs what it is)
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
  long long probe;  // > 0: the timeout probe's wait limit in cycles (lora_debug_wait_probe)
};

// The timeout probe: true if it is armed (its wait ran out: the CTA reports it
// and leaves the outputs as they were).
__device__ __forceinline__ bool probed(const RowArgs& a, uint64_t* bar) {
  if (a.probe > 0 && threadIdx.x == 0 && !wait_probe(bar, a.probe)) report(a.err, LORA_DERR_TIMEOUT);
  return a.probe > 0;
}

// The label of the row, -1 if the row does not count.
__device__ __forceinline__ int row_label(const RowArgs& a, int t, bool lead) {
  const int label = a.labels[t];
  if (label >= a.V) {
    if (lead) report(a.err, LORA_DERR_BAD_LABEL);
    return -1;
  }
  return label < 0 ? -1 : label;
}

// The same in every call: a policy that has not moved has ratio 1.
__device__ __forceinline__ float label_logp(float x, const Sum& t, float logs) {
  return empty(t) ? -INF_F : (x - base_of(t.m)) - logs;
}

// What a counted row leaves besides its gradient.
__device__ __forceinline__ void put_sum(const RowArgs& a, int t, float x, const Sum& r) {
  const float logs = logf(r.s);
  a.logp[t] = label_logp(x, r, logs);
  if (a.lse != nullptr) a.lse[t] = base_of(r.m) + logs;
  if (a.top != nullptr) {
    a.top[t] = empty(r) ? r.m : base_of(r.m);
    a.log2s[t] = log2f(r.s);
    a.coef[t] = 0.f;
  }
}

// What a row that does not count leaves there.
__device__ __forceinline__ void put_nothing(const RowArgs& a, int t) {
  a.logp[t] = 0.f;
  if (a.lse != nullptr) a.lse[t] = 0.f;
  if (a.coef != nullptr) a.coef[t] = 0.f;
  if (a.loss != nullptr) a.loss[t] = 0.f;
  if (a.kl != nullptr) a.kl[t] = 0.f;
}

// A row's inputs of the policy loss.
struct PolicyRow {
  float x, old, ref, adv, w;  // x: the label's entry
};
__device__ __forceinline__ PolicyRow policy_row(const RowArgs& a, int t, float x) {
  return PolicyRow{x, a.old_logp[t], a.opt.kl_coef > 0.f ? a.ref_logp[t] : 0.f, a.advantage[t],
                   a.weight == nullptr ? 1.f : a.weight[t]};
}

// The policy loss of a row whose sum is r, written where `lead`; its gradient's
// coefficient.  (Every thread works it out: cheaper than another barrier.)
__device__ __forceinline__ Grad policy_grad(const RowArgs& a, int t, int label, const PolicyRow& p, const Sum& r, bool lead) {
  const float logs = logf(r.s), l2 = fmaf(logs, kLog2e, logs * kLog2eLo);
  const float lp = label_logp(p.x, r, logs), q = expf(lp - p.old);
  // comparisons that a NaN fails leave it in the ratio and the ratio open
  const float low = 1.f - a.opt.clip_low, high = 1.f + a.opt.clip_high;
  const float free_ = q * p.adv, held = (q < low ? low : q > high ? high : q) * p.adv;
  const bool open = !(free_ > held);
  float kl = 0.f, slope = 0.f;
  if (a.opt.kl_coef > 0.f) {
    const float d = p.ref - lp, g = expm1f(d);
    kl = d == INF_F ? d : g - d;
    slope = a.opt.kl_coef * g;
  }
  const float coef = p.w != 0.f ? -a.opt.grad_scale * p.w * (slope + (open ? free_ : 0.f)) : 0.f;
  if (lead) {
    a.logp[t] = lp;
    a.loss[t] = p.w != 0.f ? p.w * (a.opt.kl_coef * kl - (open ? free_ : held)) : 0.f;
    if (a.kl != nullptr) a.kl[t] = kl;
  }
  return Grad{label, base_of(r.m), l2, coef, coef == 0.f || empty(r)};
}

// The gradient of a row of the preference loss, from what its sum and its pair left.
__device__ __forceinline__ Grad pair_grad(const RowArgs& a, int t, int label) {
  const float coef = a.coef[t];
  if (label < 0 || coef == 0.f || a.top[t] == -INF_F) return Grad{label, 0.f, 0.f, 0.f, true};
  return Grad{label, a.top[t], a.log2s[t], coef, false};
}

// -------------------------------------------------------------------- pairs --

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
  int probed;  // the timeout probe is armed: the rows have no sums
};

// What a pair takes from one sequence's rows.
struct PairSums {
  Pair32 lp, d;
  int count;
};
__device__ __forceinline__ PairSums add_sums(const PairSums& x, const PairSums& y) {
  return PairSums{add_pair(x.lp, y.lp), add_pair(x.d, y.d), x.count + y.count};
}

__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }
__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

// What a pair gives its rows' gradients: their coefficient, by sequence.
struct PairOut {
  float coef[2];
};

// Whether the offsets are not ascending within [0, T], for a CTA of kT threads.
template <int kT>
__device__ __forceinline__ bool bad_offsets(const PairArgs& a) {
  int bad = 0;
  for (int k = threadIdx.x; k <= 2 * a.n_pairs; k += kT) {
    const int hi = a.indptr[k], lo = k > 0 ? a.indptr[k - 1] : 0;
    bad |= hi < lo || hi > a.T;
  }
  return __syncthreads_or(bad) != 0;
}

// No pair of a call with bad offsets has a loss.
__device__ __forceinline__ void no_pair(const PairArgs& a, int p) {
  a.loss[p] = 0.f;
  if (a.seq_logp != nullptr) a.seq_logp[2 * p] = a.seq_logp[2 * p + 1] = 0.f;
}

// Pair p by a CTA of kT threads, half of it a sequence: the two sums (in a fixed
// order), the loss (written where `write`) and its coefficients.  A latency: each
// thread reads four rows at a time.
template <int kT>
__device__ __forceinline__ PairOut eval_pair(const PairArgs& a, int p, PairSums (&sh)[2][kT / 64], bool write) {
  constexpr int kHalf = kT / 2;
  const int tid = threadIdx.x, half = tid / kHalf, id = tid % kHalf;
  const int t0 = a.indptr[2 * p + half], t1 = a.indptr[2 * p + half + 1];
  PairSums x{{0.f, 0.f}, {0.f, 0.f}, 0};
  for (long long t = t0 + id; t < t1; t += 4 * kHalf) {
    int label[4];
    float lp[4], ref[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const long long q = t + k * kHalf;
      label[k] = q < t1 ? a.labels[q] : -1;
      lp[k] = q < t1 ? a.logp[q] : 0.f;
      ref[k] = q < t1 && a.ref != nullptr ? a.ref[q] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (label[k] >= 0 && label[k] < a.V) x = add_sums(x, PairSums{{lp[k], 0.f}, two_sum(lp[k], -ref[k]), 1});
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    PairSums o;
    o.lp = Pair32{__shfl_xor_sync(0xffffffffu, x.lp.hi, s), __shfl_xor_sync(0xffffffffu, x.lp.lo, s)};
    o.d = Pair32{__shfl_xor_sync(0xffffffffu, x.d.hi, s), __shfl_xor_sync(0xffffffffu, x.d.lo, s)};
    o.count = __shfl_xor_sync(0xffffffffu, x.count, s);
    x = add_sums(x, o);
  }
  if ((tid & 31) == 0) sh[half][id >> 5] = x;
  __syncthreads();
  Pair32 ratio[2];
  float share[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    x = sh[s][0];
    for (int k = 1; k < kHalf / 32; ++k) x = add_sums(x, sh[s][k]);
    const bool mean = (a.opt.flags & LORA_PREF_AVERAGE) && x.count > 0;
    share[s] = mean ? 1.f / (float)x.count : 1.f;
    ratio[s] = mean ? Pair32{x.d.hi / (float)x.count, x.d.lo / (float)x.count} : x.d;
    if (write && tid == 0 && a.seq_logp != nullptr) a.seq_logp[2 * p + s] = x.lp.hi;
  }
  const Pair32 dif = add_pair(ratio[0], Pair32{-ratio[1].hi, -ratio[1].lo});
  const float D = dif.hi;
  const float z = fmaf(a.opt.beta, D, -a.opt.margin);
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
    const float off = D - 0.5f / a.opt.beta;
    loss = off * off;
    slope = 2.f * off;
  }
  if (write && tid == 0) a.loss[p] = loss;
  return PairOut{{slope * share[0] * a.opt.grad_scale, -slope * share[1] * a.opt.grad_scale}};
}

// One CTA a pair: its loss, and the coefficient of each of its rows.
constexpr int kPairThreads = 512;
__global__ void __launch_bounds__(kPairThreads) pair_kernel(const __grid_constant__ PairArgs a) {
  __shared__ PairSums sh[2][kPairThreads / 64];
  pdl_wait_then_release();
  if (a.probed) return;
  const int p = blockIdx.x;
  if (bad_offsets<kPairThreads>(a)) {
    if (threadIdx.x == 0) {
      if (p == 0) report(a.err, LORA_DERR_BAD_SEQ);
      no_pair(a, p);
    }
    return;
  }
  const PairOut o = eval_pair<kPairThreads>(a, p, sh, true);
  if (a.coef == nullptr) return;
  constexpr int kHalf = kPairThreads / 2;
  const int half = threadIdx.x / kHalf;
  for (long long t = a.indptr[2 * p + half] + threadIdx.x % kHalf; t < a.indptr[2 * p + half + 1]; t += kHalf)
    a.coef[t] = o.coef[half];
}

// ------------------------------------------------------------- streamed form --

// logp and lse of each row: one read of the logits.
template <typename E>
__global__ void __launch_bounds__(kThreads) row_sum_kernel(const __grid_constant__ RowArgs a) {
  __shared__ RowShared sh;
  const int n = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  pdl_wait_then_release();
  if (probed(a, &sh.probe_bar)) return;
  const int t = (int)cluster_id_x();
  const bool lead = rank == 0 && threadIdx.x == 0;
  const int label = row_label(a, t, lead);
  if (label < 0) {
    if (lead) put_nothing(a, t);
    return;
  }
  const E* row = static_cast<const E*>(a.logits) + (long long)t * a.ld;
  const Cut<E> c = cut_row(row, a.V, rank, n);
  cluster_started(n);
  const float x = lead ? Elem<E>::get(row[label]) : 0.f;
  const Sum r = row_sum(thread_sum(c, a.V), &sh, rank, n);
  if (lead) put_sum(a, t, x, r);
}

// The gradient rows from the rows' sums and coefficients, last rows first: those
// that the sums read last are still in L2.
template <typename E>
__global__ void __launch_bounds__(kThreads) row_grad_kernel(const __grid_constant__ RowArgs a) {
  const int n = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  pdl_wait_then_release();
  if (a.probe > 0) return;  // the sums of this call reported it
  const int t = a.T - 1 - (int)cluster_id_x();
  const Cut<E> c = cut_row(static_cast<const E*>(a.logits) + (long long)t * a.ld, a.V, rank, n);
  const Grad g = pair_grad(a, t, row_label(a, t, false));
  write_grad<E, kThreads>(c, static_cast<E*>(a.dlogits) + (long long)t * a.ldd, a.V, g);
}

// The same for calls of few rows, without the pairs' kernel before it: a row's CTAs
// work its pair out themselves, from L2; the first row's leave the pair's loss.
struct PairRowArgs {
  RowArgs r;
  PairArgs p;
};
template <typename E>
__global__ void __launch_bounds__(kThreads) pair_row_kernel(const __grid_constant__ PairRowArgs f) {
  __shared__ PairSums sh[2][kThreads / 64];
  __shared__ int mine;  // the row's pair
  const RowArgs& a = f.r;
  const PairArgs& b = f.p;
  const int n = (int)cluster_nctarank(), rank = (int)cluster_ctarank(), tid = threadIdx.x;
  pdl_wait_then_release();
  if (a.probe > 0) return;  // the sums of this call reported it
  const int t = (int)cluster_id_x(), label = row_label(a, t, false);
  const bool first_row = rank == 0 && t == 0;  // sees to pairs without rows, and to a bad call's
  if (tid == 0) mine = -1;
  const bool bad = bad_offsets<kThreads>(b);
  if (bad && first_row) {
    if (tid == 0) report(a.err, LORA_DERR_BAD_SEQ);
    for (int k = tid; k < b.n_pairs; k += kThreads) no_pair(b, k);
  }
  if (!bad) {
    for (int k = tid; k < b.n_pairs; k += kThreads)
      if (b.indptr[2 * k] <= t && t < b.indptr[2 * k + 2]) mine = k;
    if (first_row)
      for (int k = 0; k < b.n_pairs; ++k)
        if (b.indptr[2 * k] == b.indptr[2 * k + 2]) {
          eval_pair<kThreads>(b, k, sh, true);
          __syncthreads();
        }
  }
  __syncthreads();
  const int p = mine;
  Grad g{label, 0.f, 0.f, 0.f, true};
  if (p >= 0) {
    const bool write = rank == 0 && t == b.indptr[2 * p];
    if (label >= 0 || write) {
      const float coef = eval_pair<kThreads>(b, p, sh, write).coef[t < b.indptr[2 * p + 1] ? 0 : 1];
      if (label >= 0 && coef != 0.f && a.top[t] != -INF_F) g = Grad{label, a.top[t], a.log2s[t], coef, false};
    }
  }
  const Cut<E> c = cut_row(static_cast<const E*>(a.logits) + (long long)t * a.ld, a.V, rank, n);
  write_grad<E, kThreads>(c, static_cast<E*>(a.dlogits) + (long long)t * a.ldd, a.V, g);
}

// The policy loss of each row and its gradient row.
template <typename E>
__global__ void __launch_bounds__(kThreads) policy_kernel(const __grid_constant__ RowArgs a) {
  __shared__ RowShared sh;
  const int n = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  pdl_wait_then_release();
  if (probed(a, &sh.probe_bar)) return;
  const int t = (int)cluster_id_x();
  const bool lead = rank == 0 && threadIdx.x == 0;
  const int label = row_label(a, t, lead);
  const E* row = static_cast<const E*>(a.logits) + (long long)t * a.ld;
  E* out = a.dlogits == nullptr ? nullptr : static_cast<E*>(a.dlogits) + (long long)t * a.ldd;
  const Cut<E> c = cut_row(row, a.V, rank, n);
  if (label < 0) {
    if (lead) put_nothing(a, t);
    if (out != nullptr) write_grad<E, kThreads>(c, out, a.V, Grad{-1, 0.f, 0.f, 0.f, true});
    return;
  }
  cluster_started(n);
  // the label's entry before anyone writes the gradient, which may take its place
  const PolicyRow p = policy_row(a, t, Elem<E>::get(row[label]));
  const Sum r = row_sum(thread_sum(c, a.V), &sh, rank, n);
  const Grad g = policy_grad(a, t, label, p, r, lead);
  if (out != nullptr) write_grad<E, kThreads>(c, out, a.V, g);
}

// ----------------------------------------------------------------- held form --
//
// A row is held by a group of kG threads: a warp (kG = 32, eight rows a CTA at a
// time) or a CTA of kG threads of each of the n of a cluster, kVec vectors a thread.
// Groups take rows group, group + groups, ...
//
// With kG > 32 the coming row's share waits in shared memory: thread 0 starts its
// bulk copy as soon as every warp has the current row in registers, so memory
// works through the sum, its exchange and the gradient.  A warp leaves its sum
// with every CTA of the cluster by an asynchronous store that completes on that
// CTA's barrier for the row (a cluster barrier would first flush the gradient of
// the row before).  Two sets of slots are enough: a warp that leaves its sum for
// row j + 1 has every warp's sum of row j, which each left after it read row
// j - 1's.
//
// Every wait is bounded.  A warp whose wait runs out reports it and goes through
// the remaining rows without waiting, copying or writing, so that the CTA's
// barriers stay matched; whoever still counts on it runs out in turn.  At the end
// thread 0 waits for a copy that may be under way, and the cluster meets.

struct HeldShared {
  uint64_t probe_bar, full, sums[2];
  float4 part[2][kMaxCluster * kWarps];  // m, s, the label's entry, -
};

enum RowKind { kRowSum, kRowGrad, kRowPolicy };

// What a row passed over by the held form leaves.
template <typename E, int kG, int kKind>
__device__ __forceinline__ void pass_over(const RowArgs& a, long long t, int rank, int n, int id) {
  if (kKind != kRowGrad && rank == 0 && id == 0) put_nothing(a, (int)t);
  if (a.dlogits != nullptr && kKind != kRowSum) {
    const Cut<E> c = cut_row(static_cast<const E*>(a.logits) + t * a.ld, a.V, rank, n);
    zero_row<E, kG>(c, static_cast<E*>(a.dlogits) + t * a.ldd, a.V, id);
  }
}

// The first row from t on that counts; the rows before it are passed over.
// *label: row t's label, loaded before (so that its latency is not met here), and
// on return that of the row found.
template <typename E, int kG, int kKind>
__device__ __forceinline__ long long next_row(const RowArgs& a, long long t, int groups, int rank, int n, int id, int* label) {
  while (t < a.T) {
    if (*label >= a.V) {
      if (kKind != kRowGrad && rank == 0 && id == 0) report(a.err, LORA_DERR_BAD_LABEL);
      *label = -1;
    }
    if (*label >= 0) break;
    pass_over<E, kG, kKind>(a, t, rank, n, id);
    t += groups;
    if (t < a.T) *label = a.labels[t];
  }
  return t;
}

// The gradient of a held share: vectors r of thread id, its edge element e (of
// logit xe), and the label's entry (of logit x) by the thread that has just
// written its vector.
template <typename E, int kG, int kVec>
__device__ __forceinline__ void held_put(const Cut<E>& c, E* out, int V, const uint4 (&r)[kVec], int id, int e, float xe,
                                         float x, const Grad& g) {
  constexpr int kN = Elem<E>::kN;
  if (g.zero) {
    zero_row<E, kG>(c, out, V, id);
    return;
  }
  E* const dst = out + c.head + (long long)c.v0 * kN;
  const int nv = c.v1 - c.v0;
  if (on_boundary(out, c)) {
#pragma unroll
    for (int u = 0; u < kVec; ++u)
      if (u * kG + id < nv) reinterpret_cast<uint4*>(dst)[u * kG + id] = grad_vector<E>(r[u], g);
  } else {
#pragma unroll
    for (int u = 0; u < kVec; ++u)
      if (u * kG + id < nv) {
        const uint4 y = grad_vector<E>(r[u], g);
#pragma unroll
        for (int j = 0; j < kN; ++j) dst[(u * kG + id) * kN + j] = Elem<E>::entry(y, j);
      }
  }
  if (e >= 0) out[e] = Elem<E>::put(grad_entry(xe, g, e == g.label));
  const int at = g.label - c.head, v = at / kN - c.v0;
  if (at >= 0 && g.label < c.tail0 && v >= 0 && v < nv && v % kG == id) out[g.label] = Elem<E>::put(grad_entry(x, g, true));
}

// Threads of a CTA of the held form: its group, or eight warps that are groups.
constexpr int held_threads(int group) { return group == 32 ? kThreads : group; }

template <typename E, int kG, int kVec, int kKind>
__global__ void __launch_bounds__(held_threads(kG), (kVec > 8 ? 512 : 768) / held_threads(kG)) held_kernel(const __grid_constant__ RowArgs a) {
  constexpr int kN = Elem<E>::kN, kW = held_threads(kG) / 32;
  extern __shared__ __align__(128) uint4 coming[];  // kG > 32: the coming row's share
  __shared__ HeldShared sh;
  const int n = kG == 32 ? 1 : (int)cluster_nctarank(), rank = kG == 32 ? 0 : (int)cluster_ctarank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int id = kG == 32 ? lane : (int)threadIdx.x;  // of the group's threads in this CTA
  const int group = kG == 32 ? (int)blockIdx.x * kW + warp : (int)cluster_id_x();
  const int groups = kG == 32 ? (int)gridDim.x * kW : (int)ncluster_x();
  if (kG > 32) {
    if (threadIdx.x == 0) {
      mbar_init(smem_u32(&sh.full), 1);
      mbar_init(smem_u32(&sh.sums[0]), 1);
      mbar_init(smem_u32(&sh.sums[1]), 1);
      fence_mbar_init();
    }
    if (n > 1) cluster_sync();  // every CTA's barriers are there before a peer uses them
    else __syncthreads();
  }
  pdl_wait_then_release();
  if (probed(a, &sh.probe_bar)) return;
  const bool lead = rank == 0 && id == 0;
  // the copy of a row's share into shared memory, by thread 0
  auto fetch = [&](long long t) {
    const Cut<E> c = cut_row(static_cast<const E*>(a.logits) + t * a.ld, a.V, rank, n);
    const uint32_t bytes = 16u * (uint32_t)(c.v1 - c.v0), bar = smem_u32(&sh.full);
    if (bytes == 0) {
      mbar_arrive(bar);
      return;
    }
    mbar_arrive_expect_tx(bar, bytes);
    bulk_g2s(smem_u32(coming), reinterpret_cast<const uint4*>(c.row + c.head) + c.v0, bytes, bar);
  };
  auto label_at = [&](long long t) { return t < a.T ? a.labels[t] : -1; };
  int label = label_at(group), buf = 0;
  uint32_t parity = 0, sums_parity = 0;
  long long t = next_row<E, kG, kKind>(a, group, groups, rank, n, id, &label);
  if (kG > 32 && threadIdx.x == 0 && t < a.T) fetch(t);
  bool dead = false;  // a wait of this warp's ran out
  int nlabel = label_at(t + groups);
  while (t < a.T) {
    // the row's scalars: the label's entry is read before anyone writes the row's
    // gradient, which may take the logits' place
    const float x = Elem<E>::get(static_cast<const E*>(a.logits)[t * a.ld + label]);
    PolicyRow p{};
    Grad g{};
    if (kKind == kRowPolicy) p = policy_row(a, (int)t, x);
    if (kKind == kRowGrad) g = pair_grad(a, (int)t, label);
    const long long nt = next_row<E, kG, kKind>(a, t + groups, groups, rank, n, id, &nlabel);
    const int nnlabel = label_at(nt + groups);
    const Cut<E> c = cut_row(static_cast<const E*>(a.logits) + t * a.ld, a.V, rank, n);
    const int nv = c.v1 - c.v0, e = edge_of(c, a.V, id);
    const float xe = e >= 0 ? Elem<E>::get(c.row[e]) : 0.f;
    if (kG > 32 && !dead) {
      dead = __any_sync(0xffffffffu, !mbar_wait(smem_u32(&sh.full), parity));
      if (!dead) parity ^= 1;
    }
    const uint4* mid = kG > 32 ? coming : reinterpret_cast<const uint4*>(c.row + c.head) + c.v0;
    uint4 r[kVec];
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      r[u] = low_vector<E>();
      if (u * kG + id < nv) r[u] = mid[u * kG + id];
    }
    if (kG > 32) {
      __syncthreads();
      if (threadIdx.x == 0 && nt < a.T && !dead) fetch(nt);
    }
    Sum s{-INF_F, 0.f};
    if (kKind != kRowGrad) {
      // the warp's maximum first: its sums need no rescaling
      float m = e >= 0 ? fmaxf(xe, -INF_F) : -INF_F;
#pragma unroll
      for (int u = 0; u < kVec; u += 4)
        if (u * kG < nv) {
          const uint4 four[4] = {r[u], r[u + 1], r[u + 2], r[u + 3]};
          m = fmaxf(m, Elem<E>::top(four));
        }
      m = warp_max(m);
      const float base = base_of(m);
      float add = e >= 0 ? ex2(fmaf(xe - base, kLog2e, (xe - base) * kLog2eLo)) : 0.f;
#pragma unroll
      for (int u = 0; u < kVec; u += 4)
        if (u * kG < nv) {
          const uint4 four[4] = {r[u], r[u + 1], r[u + 2], r[u + 3]};
          add += exp_sum<E>(four, base);
        }
      s = Sum{m, warp_add(add)};
      if (kG > 32 && !dead) {
        const uint32_t bar = smem_u32(&sh.sums[buf]);
        if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, (uint32_t)(n * kW * sizeof(float4)));
        // x rides along: the load of the label's entry is over before any CTA can
        // write the gradient in its place
        if (lane < n)
          st_async_v4(mapa(smem_u32(&sh.part[buf][rank * kW + warp]), lane), make_float4(s.m, s.s, x, 0.f), mapa(bar, lane));
        dead = __any_sync(0xffffffffu, !mbar_wait_cluster(bar, sums_parity));
        s = Sum{-INF_F, 0.f};
        for (int k = lane; k < n * kW; k += 32) {
          const float4 q = sh.part[buf][k];
          s = join(s, Sum{q.x, q.y});
        }
        s = warp_sum(s);
        sums_parity ^= buf;
        buf ^= 1;
      }
    }
    if (kG > 32 && dead) {
      if (lane == 0) report(a.err, LORA_DERR_TIMEOUT);
      t = nt;
      label = nlabel;
      nlabel = nnlabel;
      continue;
    }
    if (kKind == kRowSum && lead) put_sum(a, (int)t, x, s);
    if (kKind == kRowPolicy) g = policy_grad(a, (int)t, label, p, s, lead);
    if (kKind != kRowSum && a.dlogits != nullptr)
      held_put<E, kG, kVec>(c, static_cast<E*>(a.dlogits) + t * a.ldd, a.V, r, id, e, xe, x, g);
    t = nt;
    label = nlabel;
    nlabel = nnlabel;
  }
  if (kG > 32 && dead && threadIdx.x == 0) mbar_wait(smem_u32(&sh.full), parity);
  if (n > 1) cluster_sync();
}

// ------------------------------------------------------------------- host --

// How the rows of a call run: held by groups of `group` threads with `vecs`
// vectors each (0: streamed), and CTAs a row.
struct RowPlan {
  int group, vecs, n;
};

// The form of the rows, by their vectors and their number (device times on a GB300,
// bf16; "streamed" against what the rule takes, us):
//  - at most 512 vectors: a warp holds the row.  8192 x 1024: policy 33.7 / 8.3,
//    sums 23.0 / 5.7; 8192 x 4096: policy 49.1 / 26.6, sums 27.5 / 13.3.  (Few rows
//    of more than 128 vectors go to a CTA: 64 x 4096 policy 4.8 / 3.4.)
//  - longer rows of the policy loss: a CTA or cluster holds the row.  While a row
//    to a CTA of four (then eight) vectors a thread leaves SMs idle, those: 64 x
//    32000 6.9 / 5.0; else 16 vectors a thread, in groups of 128 threads while
//    those hold the row (more rows under way on an SM: 8192 x 8192 57.1 / 45.4),
//    else of 256: 1200 x 50256 53.0 / 45.4, 8192 x 128256 826 / 607.  (The rule
//    does not ask whether the gradient is wanted.  Without it a row is touched once,
//    and 8192 x 32000 takes 82 / 100, 8192 x 50256 122 / 189.)
//  - longer rows of the other two, which touch a row once: streamed.  8192 x 32000
//    sums 80.6 / 94.2 held, 8192 x 50256 124 / 186.
//  - rows beyond eight CTAs of 16 vectors a thread: streamed.
RowPlan row_plan(int kind, int T, int V, int dtype) {
  const int per = dtype == LORA_LOGITS_BF16 ? 8 : 4;  // elements of a vector
  const long long vec = V / per, places = 2LL * sm_count();
  if (vec <= 128) return RowPlan{32, 4, 1};
  if (vec <= 512 && (T >= places || kind != kRowPolicy)) return RowPlan{32, 16, 1};
  auto ctas = [&](int vecs) {  // CTAs of 256 threads that hold a row
    int n = 1;
    while (vec > (long long)n * kThreads * vecs) n *= 2;
    return n;
  };
  if (kind == kRowPolicy && ctas(16) <= kMaxCluster) {
    for (int vecs = 4; vecs <= 8; vecs *= 2)
      if (ctas(vecs) <= kMaxCluster && (long long)T * ctas(vecs) <= places) return RowPlan{256, vecs, ctas(vecs)};
    if (vec <= 1024) return RowPlan{128, 8, 1};
    if (vec <= 2048) return RowPlan{128, 16, 1};
    return RowPlan{256, 16, ctas(16)};
  }
  RowPlan p{0, 0, 1};
  // more CTAs while the rows alone leave SMs idle and each CTA still has a vector
  // for every thread
  while (p.n < kMaxCluster && (long long)T * p.n < places && V / (2 * p.n) >= per * kThreads) p.n *= 2;
  return p;
}

template <typename E, int kKind>
const void* row_kernel(const RowPlan& p) {
  if (p.group == 32) return p.vecs == 4 ? (const void*)held_kernel<E, 32, 4, kKind> : (const void*)held_kernel<E, 32, 16, kKind>;
  return kKind == kRowSum ? (const void*)row_sum_kernel<E> : (const void*)row_grad_kernel<E>;
}
template <typename E>
const void* row_kernel(int kind, const RowPlan& p) {
  if (kind == kRowSum) return row_kernel<E, kRowSum>(p);
  if (kind == kRowGrad) return row_kernel<E, kRowGrad>(p);
  if (p.group == 32)
    return p.vecs == 4 ? (const void*)held_kernel<E, 32, 4, kRowPolicy> : (const void*)held_kernel<E, 32, 16, kRowPolicy>;
  if (p.group == 128)
    return p.vecs == 8 ? (const void*)held_kernel<E, 128, 8, kRowPolicy> : (const void*)held_kernel<E, 128, 16, kRowPolicy>;
  if (p.group == 256)
    return p.vecs == 4   ? (const void*)held_kernel<E, 256, 4, kRowPolicy>
           : p.vecs == 8 ? (const void*)held_kernel<E, 256, 8, kRowPolicy>
                         : (const void*)held_kernel<E, 256, 16, kRowPolicy>;
  return (const void*)policy_kernel<E>;
}

lora_status_t launch_rows(int kind, int dtype, RowArgs* a, int T, cudaStream_t s) {
  const RowPlan p = row_plan(kind, T, a->V, dtype);
  const void* f = dtype == LORA_LOGITS_BF16 ? row_kernel<uint16_t>(kind, p) : row_kernel<float>(kind, p);
  a->T = T;
  a->probe = wait_probe_cycles();
  long long ctas = (long long)T * p.n;
  int threads = kThreads;
  size_t smem = 0;
  if (p.group > 0) {
    threads = held_threads(p.group);
    if (p.group == 32) ctas = ((long long)T + kWarps - 1) / kWarps;
    else smem = (size_t)((a->V / (dtype == LORA_LOGITS_BF16 ? 8 : 4) + p.n - 1) / p.n) * 16;
    if (smem > 0 && ensure_smem_attr(f, smem) != cudaSuccess) return LORA_ERR_CUDA;
    ctas = std::min(ctas, (long long)max_active_clusters(f, threads, smem, p.n) * p.n);
  }
  if (ctas > 0x7fffffffLL) return LORA_ERR_UNSUPPORTED;
  return launch_pdl(f, dim3((unsigned)ctas), dim3((unsigned)threads), smem, s, p.n, a) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

// Whether the gradient's rows work their pairs out themselves.  It saves a launch
// (2.3 us of host time, which a captured step does not pay) and costs each row its
// pair's sums again.  On the device, one pair of rows of 32000 (bf16), us against the
// pairs apart: 16 rows 7.6 / 8.7, 48 9.9 / 9.5, 64 11.4 / 9.7, 96 9.8 / 10.2,
// 128 12.3 / 10.4.
bool pairs_by_rows(int T, int V, int n_pairs, int dtype) {
  return n_pairs > 0 && n_pairs <= 64 && T <= 128 && row_plan(kRowGrad, T, V, dtype).group == 0;
}

lora_status_t launch_pair_rows(int dtype, const RowArgs& a, const PairArgs& p, int T, cudaStream_t s) {
  const int n = row_plan(kRowGrad, T, a.V, dtype).n;
  PairRowArgs f;
  memset(&f, 0, sizeof(f));
  f.r = a;
  f.r.T = T;
  f.r.probe = wait_probe_cycles();
  f.p = p;
  const void* k = dtype == LORA_LOGITS_BF16 ? (const void*)pair_row_kernel<uint16_t> : (const void*)pair_row_kernel<float>;
  return launch_pdl(k, dim3((unsigned)(T * n)), dim3(kThreads), 0, s, n, &f) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
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
  p.probed = wait_probe_cycles() > 0;
  const bool grad = T > 0 && dlogits != nullptr;
  if (grad && pairs_by_rows(T, V, n_pairs, dtype)) return launch_pair_rows(dtype, a, p, T, s);
  if (n_pairs > 0 &&
      launch_pdl((const void*)pair_kernel, dim3((unsigned)n_pairs), dim3(kPairThreads), 0, s, 0, &p) != cudaSuccess)
    return LORA_ERR_CUDA;
  return grad ? launch_rows(kRowGrad, dtype, &a, T, s) : LORA_OK;
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
