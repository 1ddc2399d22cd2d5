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

// ----------------------------------------------------------------- divergence --

// p log(p / m) - p + m with x = log(m / p) and w = e^x - 1: p (w - x).
__device__ __forceinline__ float term(float p, float m, float x, float w) {
  // near 0 by the series of (w - x) / x^2: the next term is 1e-7 of the sum
  const float s = fmaf(x, fmaf(x, fmaf(x, fmaf(x, fmaf(x, 1.f / 5040.f, 1.f / 720.f), 1.f / 120.f), 1.f / 24.f), 1.f / 6.f), 0.5f);
  const float y = fabsf(x) < 0.35f ? p * (x * x) * s : x < 80.f ? p * (w - x) : m - p * x;
  return p == 0.f ? m : y;
}

// One outcome of probabilities e^lp (teacher) and e^lq (student).
struct Outcome {
  float kd;     // its term
  float mass;   // q e, of C
  float share;  // of its gradient: q (e - C) without C
};
// e of an outcome with d = log p - log q.
__device__ __forceinline__ float slope_of(int kind, float mix, float d) {
  if (kind == LORA_DISTILL_REVERSE) return -d;
  if (kind == LORA_DISTILL_FORWARD) return d < -80.f ? 1.f : -expm1f(d);
  return (mix - 1.f) * (d > 0.f ? d + log1pf((1.f - mix) * expm1f(-d)) : log1pf(mix * expm1f(d)));
}
__device__ __forceinline__ Outcome outcome(int kind, float mix, float lp, float lq) {
  const float p = expf(lp), q = expf(lq), d = lp - lq;
  Outcome o;
  if (kind == LORA_DISTILL_FORWARD) {
    const float w = expm1f(-d);  // q / p - 1
    o.kd = q == 0.f ? INF_F : term(p, q, -d, w);
    o.mass = 0.f;
    o.share = p == 0.f || d < -80.f ? q - p : p * w;
  } else if (kind == LORA_DISTILL_REVERSE) {
    o.kd = p == 0.f ? INF_F : term(q, p, d, expm1f(d));
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
    o.kd = mix * term(p, m, v, expm1f(v)) + (1.f - mix) * term(q, m, u, expm1f(u));
    o.mass = o.share = q == 0.f ? 0.f : q * (mix - 1.f) * u;
  }
  if (p == 0.f && q == 0.f) o.kd = o.mass = o.share = 0.f;
  return o;
}

__device__ __noinline__ Outcome other_outcome(int kind, float mix, float lp, float lq) { return outcome(kind, mix, lp, lq); }

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
  Terms terms, plain;  // of the temperature; of temperature 1
  int both;            // a cross-entropy at another temperature: two sums a row
  float* loss;
  float* kd;
  float* ce;
  void* dlogits;
  long long ldd;
  int32_t* err;
  long long probe;
};

// What the rows' gradients are made of: entry v (not listed, not the label) is
//     kd 2^((x - base) hi - l2) + ce 2^((x - base) log2 e - l2_plain).
struct Slope {
  float base, kd, l2, ce, l2_plain;
};

template <typename E, bool kBoth>
__device__ __forceinline__ uint4 slope_vector(const uint4& x, const Slope& g, const Terms& terms, const Terms& plain) {
  constexpr int kPairs = Elem<E>::kPairs;
  const uint64_t nb = pair_of(-g.base, -g.base), hi = pair_of(terms.hi, terms.hi), nl = pair_of(-g.l2, -g.l2);
  const uint64_t c = pair_of(g.kd, g.kd);
  uint64_t f[kPairs];
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    const uint64_t d = add2(Elem<E>::pair(x, j), nb);
    float a, b;
    split(fma2(d, hi, nl), a, b);
    f[j] = mul2(c, pair_of(ex2(a), ex2(b)));
    if (kBoth) {
      split(fma2(d, pair_of(plain.hi, plain.hi), pair_of(-g.l2_plain, -g.l2_plain)), a, b);
      f[j] = fma2(pair_of(g.ce, g.ce), pair_of(ex2(a), ex2(b)), f[j]);
    }
  }
  return Elem<E>::pack(f);
}
template <bool kBoth>
__device__ __forceinline__ float slope_entry(float x, const Slope& g, const Terms& terms, const Terms& plain) {
  const float d = x - g.base;
  float f = g.kd * ex2(fmaf(d, terms.hi, -g.l2));
  if (kBoth) f = fmaf(g.ce, ex2(fmaf(d, plain.hi, -g.l2_plain)), f);
  return f;
}

// A row's inputs but its logits.
struct RowIn {
  int label;
  float weight, tail;
};
__device__ __forceinline__ RowIn row_in(const DistillArgs& a, long long t, int label) {
  return RowIn{label, a.weight == nullptr ? 1.f : a.weight[t], a.tail == nullptr ? -INF_F : a.tail[t]};
}
__device__ __forceinline__ void put_nothing(const DistillArgs& a, long long t) {
  a.loss[t] = 0.f;
  if (a.kd != nullptr) a.kd[t] = 0.f;
  if (a.ce != nullptr) a.ce[t] = 0.f;
}
// The row's divergence (without a student: infinite, unless the teacher says nothing) and losses.
__device__ __forceinline__ void put_losses(const DistillArgs& a, long long t, const RowIn& in, float kd, float ce) {
  const float kw = a.opt.kd_weight, cw = a.opt.ce_weight;
  a.loss[t] = in.weight == 0.f ? 0.f : in.weight * ((kw > 0.f ? kw * kd : 0.f) + (cw > 0.f ? cw * ce : 0.f));
  if (a.kd != nullptr) a.kd[t] = kd;
  if (a.ce != nullptr) a.ce[t] = ce;
}

// ----------------------------------------------------------------- held form --
//
// A row is held in the registers of kG threads of a CTA, or of the n CTAs of a cluster,
// from its sum to its gradient, kVec vectors a thread, so it is read once; the coming
// row's share arrives in shared memory meanwhile by a bulk copy.  (The held policy loss
// of logits.cu in that.)  One more warp has the list, a row ahead:
//  - it looks up the entries' logits and takes their places out of the share in shared
//    memory (-inf) before the registers read it, so the sum is of the rest alone and the
//    rest's gradient needs no test;
//  - it works out each entry's outcome while the others write the rest's gradient, then
//    writes the entries' over what the vectors left there;
//  - a bit an entry of the share shows what is listed twice.
// (With the entries in the threads that hold the row, those warps kept the others waiting:
// 8192 x 128256 987 us.)
//
// Sums cross the cluster as there: a warp sends its own to every CTA by an asynchronous
// store on that CTA's barrier for the row; two sets of slots are enough.
// Every wait is bounded.  A warp whose wait ran out reports it and goes through the
// remaining rows without waiting, copying or writing, its barriers matched.
//
// What bounds it: memory, one read and one write of the logits; then the latency of a
// row's barriers, which the other CTA of the SM hides.

constexpr int kMaxCluster = 8;
constexpr int kMaxList = LORA_TOPK_MAX;

template <int kG>
struct HeldShared {
  static constexpr int kParts = kG / 32;  // warps that send
  uint64_t probe_bar, full, sums[2];
  float4 part[2][kMaxCluster * kParts];  // m, the rest's sum, its sum at temperature 1, a bad list
  float4 list[2];                        // the list's base (a value), log of its mass, student's maximum and sum
  float list_plain[2];                   // the student's sum at temperature 1
  float C;
  float label_logit;
  int bad[2];  // the list is
  int ids[2][kMaxList];  // -1: none
  float values[2][kMaxList], logits[2][kMaxList];
  float share[kMaxList];  // the entries' gradients, but for the factors
};

template <typename E, int kG>
__device__ __forceinline__ void zero_share(const Cut<E>& c, E* out, int V, int id) {
  constexpr int kN = Elem<E>::kN;
  E* const dst = out + c.head + (long long)c.v0 * kN;
  const int nv = c.v1 - c.v0, e = edge_of(c, V, id);
  if (on_boundary(out, c)) {
    for (int k = id; k < nv; k += kG) reinterpret_cast<uint4*>(dst)[k] = make_uint4(0, 0, 0, 0);
  } else {
    for (int k = id; k < nv * kN; k += kG) dst[k] = Elem<E>::put(0.f);
  }
  if (e >= 0) out[e] = Elem<E>::put(0.f);
}

// Barriers of a CTA's kCount threads; one that the first ones only arrive at.
template <int kBar, int kCount>
__device__ __forceinline__ void meet() {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"n"(kBar), "n"(kCount) : "memory");
}
template <int kBar, int kCount>
__device__ __forceinline__ void pass() {
  __syncwarp();
  asm volatile("bar.arrive %0, %1;" ::"n"(kBar), "n"(kCount) : "memory");
}

// A row's sums over all its parts, as every warp works them out.
struct RowSum {
  float m, rest, plain;
  bool bad;
};
__device__ __forceinline__ RowSum join_parts(const float4* part, int parts, const Terms& terms, bool both, int lane) {
  RowSum r{-INF_F, 0.f, 0.f, false};
  for (int k = lane; k < parts; k += 32) r.m = fmaxf(r.m, part[k].x);
  r.m = warp_max(r.m);
  for (int k = lane; k < parts; k += 32) {
    const float4 q = part[k];
    r.rest += q.y * expf((q.x - base_of(r.m)) * terms.inv);
    if (both) r.plain += q.z * expf(q.x - base_of(r.m));
    r.bad |= q.w != 0.f;
  }
  r.rest = warp_add(r.rest);
  if (both) r.plain = warp_add(r.plain);
  r.bad = __any_sync(0xffffffffu, r.bad);
  return r;
}

// With the list: the student's totals and what both kinds of warps take from them.
struct RowTotal {
  float base, rest, lt, l1;  // lt: log of the sum at the temperature, l1: at temperature 1
  float lr;                  // log of the rest's share
  bool none, taught;         // nothing is visible; the teacher says something (and the student too)
};
__device__ __forceinline__ RowTotal row_total(const RowSum& s, const float4& list, float list_plain, const Terms& terms, bool both) {
  RowTotal r;
  // the two sums over the greater base
  const bool some = list.w != 0.f, lists = some && list.z > s.m;
  r.base = base_of(lists ? list.z : s.m);
  const float fall = some ? fminf(s.m, list.z) - r.base : 0.f;  // of the other
  const float e = expf(fall * terms.inv);
  r.rest = lists ? s.rest * e : s.rest;
  const float total = r.rest + (lists ? list.w : some ? list.w * e : 0.f);
  r.lt = r.l1 = logf(total);
  if (both) {
    const float e1 = expf(fall);
    r.l1 = logf(lists ? fmaf(s.plain, e1, list_plain) : some ? fmaf(list_plain, e1, s.plain) : s.plain);
  }
  r.none = total == 0.f;
  r.taught = list.y != -INF_F && !r.none;
  r.lr = logf(__fdividef(r.rest, total));
  return r;
}

template <typename E, int kG, int kVec, bool kBoth>
__global__ void __launch_bounds__(kG + 32, kG > 256 ? 1 : kVec > 8 ? 2 : 3) held_kernel(const __grid_constant__ DistillArgs a) {
  constexpr int kN = Elem<E>::kN, kAll = kG + 32;
  using Shared = HeldShared<kG>;
  extern __shared__ __align__(128) uint4 coming[];  // the coming row's share, then its bits
  __shared__ Shared sh;
  const int n = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, id = (int)threadIdx.x;
  const int group = (int)cluster_id_x(), groups = (int)ncluster_x();
  const int share = (a.V / kN + n - 1) / n;  // vectors of the largest share
  uint32_t* const bits = reinterpret_cast<uint32_t*>(coming + share);
  for (int i = id; i < (share * kN + 16 + 31) / 32; i += kAll) bits[i] = 0;
  if (id == 0) {
    mbar_init(smem_u32(&sh.full), 1);
    mbar_init(smem_u32(&sh.sums[0]), 1);
    mbar_init(smem_u32(&sh.sums[1]), 1);
    fence_mbar_init();
  }
  if (n > 1) cluster_sync();  // every CTA's barriers are there before a peer uses them
  else __syncthreads();
  pdl_wait_then_release();
  if (a.probe > 0) {
    if (id == 0 && !wait_probe(&sh.probe_bar, a.probe)) report(a.err, LORA_DERR_TIMEOUT);
    return;
  }
  const bool forward = a.opt.kind == LORA_DISTILL_FORWARD;
  const Terms terms = a.terms, plain = a.plain;
  auto row_at = [&](long long t) { return static_cast<const E*>(a.logits) + t * a.ld; };
  auto cut_at = [&](long long t) { return cut_row(row_at(t), a.V, rank, n); };
  auto out_at = [&](long long t) { return static_cast<E*>(a.dlogits) + t * a.ldd; };
  auto label_at = [&](long long t) { return a.labels != nullptr && t < a.T ? a.labels[t] : -1; };
  // The first row from t on that counts (without labels all do; their label is -1); the
  // rows before it are passed over.  *label: row t's, loaded before, then that row's.
  auto next_row = [&](long long t, int* label) {
    while (a.labels != nullptr && t < a.T) {
      if (*label >= 0 && *label < a.V) break;
      if (id == 0 && rank == 0) {
        if (*label >= a.V) report(a.err, LORA_DERR_BAD_LABEL);
        put_nothing(a, t);
      }
      if (id < kG && a.dlogits != nullptr) zero_share<E, kG>(cut_at(t), out_at(t), a.V, id);
      t += groups;
      *label = label_at(t);
    }
    return t;
  };
  // this warp's part of a row to every CTA
  auto send = [&](int buf, const float4& part) {
    const uint32_t bar = smem_u32(&sh.sums[buf]);
    if (lane < n) st_async_v4(mapa(smem_u32(&sh.part[buf][rank * Shared::kParts + warp]), lane), part, mapa(bar, lane));
  };
  // The factors of a row's gradient, of its divergence (C known) and of its cross-entropy.
  auto factors = [&](const RowTotal& r, const RowIn& in, bool bad, float C, float* kw, float* cw) {
    const float gs = r.none || in.weight == 0.f || bad ? 0.f : a.opt.grad_scale * in.weight;
    *kw = gs != 0.f && fabsf(C) != INF_F ? gs * a.opt.kd_weight * terms.inv : 0.f;
    *cw = a.opt.ce_weight > 0.f ? gs * a.opt.ce_weight : 0.f;
  };

  int label = label_at(group), buf = 0;
  uint32_t parity = 0, sums_parity = 0;
  long long t = next_row(group, &label);
  int nlabel = label_at(t + groups);
  bool dead = false;  // a wait of this warp's ran out

  if (id < kG) {
    // ------------------------------------------------------------ the row --
    auto fetch = [&](long long t) {  // by thread 0
      const Cut<E> c = cut_at(t);
      const uint32_t bytes = 16u * (uint32_t)(c.v1 - c.v0), bar = smem_u32(&sh.full);
      if (bytes == 0) {
        mbar_arrive(bar);
        return;
      }
      mbar_arrive_expect_tx(bar, bytes);
      bulk_g2s(smem_u32(coming), reinterpret_cast<const uint4*>(c.row + c.head) + c.v0, bytes, bar);
    };
    if (id == 0 && t < a.T) fetch(t);
    for (int turn = 0; t < a.T; turn ^= 1) {
      const RowIn in = row_in(a, t, label);
      const long long nt = next_row(t + groups, &nlabel);
      const int nnlabel = label_at(nt + groups);
      const Cut<E> c = cut_at(t);
      const int nv = c.v1 - c.v0, e = edge_of(c, a.V, id);
      float xe = e >= 0 ? Elem<E>::get(c.row[e]) : -INF_F;
      if (!dead) {
        dead = __any_sync(0xffffffffu, !mbar_wait(smem_u32(&sh.full), parity));
        if (!dead) parity ^= 1;
      }
      meet<1, kAll>();  // the listed places are taken out
      if (e >= 0) {
        const int at = e - (c.first ? 0 : c.head + c.v0 * kN);
        if (bits[at >> 5] >> (at & 31) & 1) xe = -INF_F;
      }
      uint4 r[kVec];
#pragma unroll
      for (int u = 0; u < kVec; ++u) {
        r[u] = low_vector<E>();
        if (u * kG + id < nv) r[u] = coming[u * kG + id];
      }
      meet<2, kAll>();  // everyone has its vectors: the place is free
      if (id == 0 && nt < a.T && !dead) fetch(nt);
      // the rest's sum: the warp's maximum first, then its terms, then every warp's
      float m = fmaxf(xe, -INF_F);
#pragma unroll
      for (int u = 0; u < kVec; u += 4)
        if (u * kG < nv) {
          const uint4 four[4] = {r[u], r[u + 1], r[u + 2], r[u + 3]};
          m = fmaxf(m, Elem<E>::top(four));
        }
      m = warp_max(m);
      float rest = e >= 0 ? terms.power(xe, base_of(m)) : 0.f, rest_plain = kBoth && e >= 0 ? plain.power(xe, base_of(m)) : 0.f;
#pragma unroll
      for (int u = 0; u < kVec; u += 4)
        if (u * kG < nv) {
          const uint4 four[4] = {r[u], r[u + 1], r[u + 2], r[u + 3]};
          rest += power_sum<E>(terms, four, base_of(m));
          if (kBoth) rest_plain += power_sum<E>(plain, four, base_of(m));
        }
      rest = warp_add(rest);
      if (kBoth) rest_plain = warp_add(rest_plain);
      if (!dead) {
        const uint32_t bar = smem_u32(&sh.sums[buf]);
        if (id == 0) mbar_arrive_expect_tx(bar, (uint32_t)(n * Shared::kParts * sizeof(float4)));
        send(buf, make_float4(m, rest, rest_plain, sh.bad[turn] ? 1.f : 0.f));
        dead = __any_sync(0xffffffffu, !mbar_wait_cluster(bar, sums_parity));
      }
      const RowSum s = join_parts(sh.part[buf], n * Shared::kParts, terms, kBoth, lane);
      sums_parity ^= buf;
      buf ^= 1;
      const float4 list = sh.list[turn];
      const RowTotal r_ = row_total(s, list, sh.list_plain[turn], terms, kBoth);
      // the rest's slope
      float slope = 0.f, C = 0.f;
      if (!forward) meet<3, kAll>();
      if (!forward) C = sh.C;
      if (r_.taught && !(r_.rest == 0.f)) {
        const float d = in.tail - list.x * terms.inv - list.y - r_.lr;
        slope = slope_of(a.opt.kind, a.opt.mix, d) - C;
      }
      float kw, cw;
      factors(r_, in, s.bad, C, &kw, &cw);
      // at temperature 1 the two parts of the gradient share their powers
      Slope g{r_.base, kw != 0.f ? kw * slope : 0.f, r_.lt * kLog2e + r_.lt * kLog2eLo, cw, r_.l1 * kLog2e + r_.l1 * kLog2eLo};
      if (!kBoth) g.kd += cw;
      E* const out = a.dlogits == nullptr || dead ? nullptr : out_at(t);
      if (out != nullptr) {
        if (g.kd == 0.f && (!kBoth || cw == 0.f)) {
          zero_share<E, kG>(c, out, a.V, id);
        } else {
          E* const dst = out + c.head + (long long)c.v0 * kN;
          if (on_boundary(out, c)) {
#pragma unroll
            for (int u = 0; u < kVec; ++u)
              if (u * kG + id < nv) reinterpret_cast<uint4*>(dst)[u * kG + id] = slope_vector<E, kBoth>(r[u], g, terms, plain);
          } else {
#pragma unroll
            for (int u = 0; u < kVec; ++u)
              if (u * kG + id < nv) {
                const uint4 y = slope_vector<E, kBoth>(r[u], g, terms, plain);
#pragma unroll
                for (int j = 0; j < kN; ++j) dst[(u * kG + id) * kN + j] = Elem<E>::entry(y, j);
              }
          }
          if (e >= 0) out[e] = Elem<E>::put(slope_entry<kBoth>(xe, g, terms, plain));
        }
      }
      pass<4, kAll>();  // the listed places may be written
      if (dead && lane == 0) report(a.err, LORA_DERR_TIMEOUT);
      t = nt;
      label = nlabel;
      nlabel = nnlabel;
    }
    if (dead && id == 0) mbar_wait(smem_u32(&sh.full), parity);
  } else {
    // ----------------------------------------------------------- the list --
    // Entry j is lane j % 32's; a lane's eight go through registers on their way to shared
    // memory, so that a row's loads are under way together.
    constexpr int kOwn = kMaxList / 32;
    const int rounds = (a.k + 31) / 32;
    int v[kOwn];
    float value[kOwn], x[kOwn];
    auto load_list = [&](long long t) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int j = i * 32 + lane;
        const bool on = i < rounds && j < a.k && t < a.T;
        v[i] = on ? a.ids[t * a.k + j] : -1;
        value[i] = on ? a.values[t * a.k + j] : -INF_F;
      }
    };
    auto load_logits = [&](long long t) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        if (value[i] == -INF_F) v[i] = -1;
        x[i] = v[i] >= 0 && v[i] < a.V ? Elem<E>::get(row_at(t)[v[i]]) : -INF_F;
      }
    };
    auto load_label = [&](long long t, int label) { return label >= 0 && t < a.T ? Elem<E>::get(row_at(t)[label]) : 0.f; };
    // the list to its places, with its maxima and sums
    auto put_list = [&](const RowIn& in, int turn) {
      float mv = -INF_F, mx = -INF_F;
#pragma unroll
      for (int i = 0; i < kOwn; ++i)
        if (i < rounds) {
          sh.ids[turn][i * 32 + lane] = v[i];
          sh.values[turn][i * 32 + lane] = value[i];
          sh.logits[turn][i * 32 + lane] = x[i];
          if (v[i] >= 0) mv = fmaxf(mv, value[i]), mx = fmaxf(mx, x[i]);
        }
      mv = warp_max(mv);
      mx = base_of(warp_max(mx));
      const float high = base_of(fmaxf(mv, in.tail * a.opt.temperature));  // in the values' measure
      float sv = 0.f, sx = 0.f, s1 = 0.f;
#pragma unroll
      for (int i = 0; i < kOwn; ++i)
        if (i < rounds) {
          sv += v[i] >= 0 ? expf((value[i] - high) * terms.inv) : 0.f;
          sx += v[i] >= 0 ? expf((x[i] - mx) * terms.inv) : 0.f;
          if (kBoth) s1 += v[i] >= 0 ? expf(x[i] - mx) : 0.f;
        }
      sv = warp_add(sv) + expf(in.tail - high * terms.inv);
      sx = warp_add(sx);
      if (kBoth) s1 = warp_add(s1);
      if (lane == 0) {
        sh.list[turn] = make_float4(high, logf(sv), mx, sx);
        sh.list_plain[turn] = s1;
      }
      __syncwarp();
    };
    auto input_at = [&](long long t, int label) { return t < a.T ? row_in(a, t, label) : RowIn{-1, 0.f, -INF_F}; };
    load_list(t);
    load_logits(t);
    float xl = load_label(t, label);
    RowIn in = input_at(t, label);
    put_list(in, 0);
    for (int turn = 0; t < a.T; turn ^= 1) {
      const long long nt = next_row(t + groups, &nlabel);
      const int nnlabel = label_at(nt + groups);
      load_list(nt);
      const RowIn nin = input_at(nt, nlabel);
      const Cut<E> c = cut_at(t);
      const int first = c.first ? 0 : c.head + c.v0 * kN, end = c.last ? a.V : c.head + c.v1 * kN;  // the share's entries
      const int* const ids = sh.ids[turn];
      const float *const values = sh.values[turn], *const logits = sh.logits[turn];
      const float4 list = sh.list[turn];
      const float list_plain = sh.list_plain[turn];
      auto mine = [&](int v) { return v >= first && v < end; };
      if (!dead) {
        dead = __any_sync(0xffffffffu, !mbar_wait(smem_u32(&sh.full), parity));
        if (!dead) parity ^= 1;
      }
      bool bad = false;
      for (int i = 0, j = lane; i < rounds; ++i, j += 32) {
        const int v = ids[j], at = v - first, k = v - c.head - c.v0 * kN;
        bad |= v >= a.V;
        if (!mine(v)) continue;
        bad |= (atomicOr(&bits[at >> 5], 1u << (at & 31)) >> (at & 31) & 1) != 0;
        if (!dead && k >= 0 && k < (c.v1 - c.v0) * kN) reinterpret_cast<E*>(coming)[k] = Elem<E>::put(-INF_F);
      }
      bad = __any_sync(0xffffffffu, bad);
      // The loads of the row's logits are over before any CTA can write a gradient in their
      // place, which takes this CTA's sums: they are in shared memory, the label's too.
      if (lane == 0) {
        sh.bad[turn] = bad;
        sh.label_logit = xl;
      }
      const bool label_mine = mine(label), label_listed = label_mine && (bits[(label - first) >> 5] >> ((label - first) & 31) & 1);
      // (written as threads write, before the next copy takes its place)
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      meet<1, kAll>();
      meet<2, kAll>();
      for (int i = 0, j = lane; i < rounds; ++i, j += 32)
        if (mine(ids[j])) bits[(ids[j] - first) >> 5] = 0;
      load_logits(nt);
      const float nxl = load_label(nt, nlabel);
      if (!dead) dead = __any_sync(0xffffffffu, !mbar_wait_cluster(smem_u32(&sh.sums[buf]), sums_parity));
      const RowSum s = join_parts(sh.part[buf], n * Shared::kParts, terms, kBoth, lane);
      sums_parity ^= buf;
      buf ^= 1;
      const RowTotal r = row_total(s, list, list_plain, terms, kBoth);
      // the outcomes: the entries', and the rest's as entry k
      const float tail_p = in.tail - list.x * terms.inv - list.y, tail_q = r.lr;
      float kd = 0.f, C = 0.f;
      for (int i0 = 0; i0 * 32 <= a.k; i0 += 3) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const int j = (i0 + i) * 32 + lane;
          const bool entry = j < a.k && ids[j] >= 0;
          if (!r.taught || !(entry || j == a.k)) continue;
          const float lp = entry ? (values[j] - list.x) * terms.inv - list.y : tail_p;
          const float lq = entry ? (logits[j] - r.base) * terms.inv - r.lt : tail_q;
          const Outcome o = forward ? outcome(LORA_DISTILL_FORWARD, 0.f, lp, lq) : other_outcome(a.opt.kind, a.opt.mix, lp, lq);
          if (entry) sh.share[j] = o.share;
          kd += o.kd;
          C += o.mass;
        }
      }
      kd = warp_add(kd);
      if (!forward) {
        C = warp_add(C);
        if (lane == 0) sh.C = C;
        meet<3, kAll>();
      }
      if (rank == 0 && lane == 0 && !dead) {
        if (s.bad) {
          report(a.err, LORA_DERR_BAD_LABEL);
          put_nothing(a, t);
        } else {
          const float ce = a.opt.ce_weight > 0.f ? (r.none ? INF_F : r.l1 - (xl - r.base)) : 0.f;
          put_losses(a, t, in, r.none ? (list.y != -INF_F ? INF_F : 0.f) : kd, ce);
        }
      }
      put_list(nin, turn ^ 1);
      meet<4, kAll>();  // the rest's gradient is written
      if (a.dlogits != nullptr && !dead) {
        E* const out = out_at(t);
        float kw, cw;
        factors(r, in, s.bad, C, &kw, &cw);
        if (kw != 0.f || cw != 0.f) {
          for (int i = 0, j = lane; i < rounds; ++i, j += 32) {
            const int v = ids[j];
            if (!mine(v)) continue;
            const float x = logits[j] - r.base;
            float y = kw != 0.f && r.taught ? kw * sh.share[j] : 0.f;
            if (!forward || cw != 0.f) {
              const float q = expf(x * terms.inv - r.lt);
              if (!forward && kw != 0.f) y -= kw * q * C;
              if (cw != 0.f) y += cw * ((kBoth ? expf(x - r.l1) : q) - (v == label ? 1.f : 0.f));
            }
            out[v] = Elem<E>::put(y);
          }
          if (lane == 0 && label_mine && !label_listed && cw != 0.f) {
            const float slope =
                kw != 0.f && r.taught && !(r.rest == 0.f) ? slope_of(a.opt.kind, a.opt.mix, tail_p - tail_q) - C : 0.f;
            const float x = xl - r.base, q = expf(x * terms.inv - r.lt);
            out[label] = Elem<E>::put(kw * slope * q + cw * ((kBoth ? expf(x - r.l1) : q) - 1.f));
          }
        }
      }
      if (dead && lane == 0) report(a.err, LORA_DERR_TIMEOUT);
      t = nt;
      label = nlabel;
      nlabel = nnlabel;
      xl = nxl;
      in = nin;
    }
  }
  if (n > 1) cluster_sync();
}

// ----------------------------------------------------------------- long rows --

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

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

// Rows longer than the held form takes: a CTA a row, which it reads three times, with a
// bit a logit that says whether it is listed.
template <typename E>
__global__ void __launch_bounds__(kThreads) long_row_kernel(const __grid_constant__ DistillArgs a) {
  extern __shared__ uint32_t bits[];
  __shared__ float sh[kWarps];
  __shared__ int bad;
  __shared__ uint64_t probe_bar;
  pdl_wait_then_release();
  if (a.probe > 0) {
    if (threadIdx.x == 0 && !wait_probe(&probe_bar, a.probe)) report(a.err, LORA_DERR_TIMEOUT);
    return;
  }
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
    if (tid == 0) put_nothing(a, t);
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
  const float high = base_of(fmaxf(block_max(value * inv, sh), tail));  // in the tail's measure
  const float mass = block_add(id >= 0 ? expf(value * inv - high) : 0.f, sh) + expf(tail - high), lm = logf(mass);
  Outcome o{0.f, 0.f, 0.f}, r = o;
  const float dt = tail - high - lm - (logf(rest) - lt);
  if (mass != 0.f && total != 0.f) {
    if (id >= 0) o = outcome(a.opt.kind, a.opt.mix, value * inv - high - lm, x * inv - lt);
    r = outcome(a.opt.kind, a.opt.mix, tail - high - lm, logf(rest) - lt);
  }
  const float kd = block_add(o.kd, sh) + r.kd, C = block_add(o.mass, sh) + r.mass;
  bool none = total == 0.f;  // nothing is visible
  const float ce = a.opt.ce_weight > 0.f ? (none ? INF_F : logf(all) - xl) : 0.f;
  if (tid == 0) put_losses(a, t, RowIn{label, w, tail}, none && mass > 0.f ? INF_F : kd, ce);
  if (out == nullptr) return;
  __syncthreads();
  none = none || w == 0.f;
  const bool zero = fabsf(C) == INF_F;
  const float gs = a.opt.grad_scale * w, kw = gs * a.opt.kd_weight * inv, cw = a.opt.ce_weight > 0.f ? gs * a.opt.ce_weight : 0.f;
  const float slope = rest == 0.f || mass == 0.f ? 0.f : slope_of(a.opt.kind, a.opt.mix, dt) - C;
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

// -------------------------------------------------------------------- host --

template <typename E, int kG, int kVec>
lora_status_t launch_held(DistillArgs& a, int n, cudaStream_t s) {
  const void* f = a.both ? (const void*)held_kernel<E, kG, kVec, true> : (const void*)held_kernel<E, kG, kVec, false>;
  const size_t share = (size_t)(a.V / Elem<E>::kN + n - 1) / n;
  const size_t smem = share * 16 + (share * Elem<E>::kN + 16 + 31) / 32 * 4;
  if (ensure_smem_attr(f, smem) != cudaSuccess) return LORA_ERR_CUDA;
  const long long ctas = std::min((long long)a.T * n, (long long)max_active_clusters(f, kG + 32, smem, n) * n);
  return launch_pdl(f, dim3((unsigned)ctas), dim3(kG + 32), smem, s, n, &a) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

// The form of the rows, as the policy loss's are chosen (logits.cu): CTAs of four, then
// eight vectors a thread while a row to each group leaves SMs idle, else of sixteen.
template <typename E>
lora_status_t launch(DistillArgs& a, cudaStream_t s) {
  const long long vec = a.V / Elem<E>::kN, places = 2LL * sm_count();
  auto ctas = [&](int threads, int vecs) {
    int n = 1;
    while (vec > (long long)n * threads * vecs) n *= 2;
    return n;
  };
  if (vec <= 1024) return launch_held<E, 256, 4>(a, 1, s);
  if (ctas(256, 4) <= kMaxCluster && (long long)a.T * ctas(256, 4) <= places) return launch_held<E, 256, 4>(a, ctas(256, 4), s);
  if (vec <= 2048 || (ctas(256, 8) <= kMaxCluster && (long long)a.T * ctas(256, 8) <= places))
    return launch_held<E, 256, 8>(a, ctas(256, 8), s);
  if (ctas(256, 16) <= kMaxCluster) return launch_held<E, 256, 16>(a, ctas(256, 16), s);
  if (ctas(512, 16) <= kMaxCluster) return launch_held<E, 512, 16>(a, ctas(512, 16), s);
  const void* f = (const void*)long_row_kernel<E>;
  const size_t smem = ((size_t)a.V + 31) / 32 * 4;
  if (smem > 200000) return LORA_ERR_UNSUPPORTED;
  if (ensure_smem_attr(f, smem) != cudaSuccess) return LORA_ERR_CUDA;
  return launch_pdl(f, dim3((unsigned)a.T), dim3(kThreads), smem, s, 0, &a) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
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
  a.terms = terms_of(opts->temperature);
  a.plain = terms_of(1.f);
  a.both = opts->ce_weight > 0.f && opts->temperature != 1.f;
  a.probe = wait_probe_cycles();
  return dtype == LORA_LOGITS_BF16 ? launch<uint16_t>(a, (cudaStream_t)stream) : launch<float>(a, (cudaStream_t)stream);
}

}  // extern "C"
