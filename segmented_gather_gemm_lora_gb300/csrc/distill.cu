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
//
// What vanishes is told by logarithms: e^lq is 0 in fp32 from lq = -104 on, where p (lp - lq) is
// still a number.  From -745 on, where 64 bits end too, a share counts as nothing, as that of
// an entry at -inf does: a finite mask hides.
// The rest's entries share its gradient by their part of the rest's sum, taken over the rest's own
// largest logit, so nothing is divided by a share that has vanished.
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
  // (from x = 16 on without p w, in which a p of few bits would count)
  const float y = fabsf(x) < 0.35f ? p * (x * x) * s : x < 16.f ? p * (w - x) : m - p * (x + 1.f);
  return p == 0.f ? m : y;
}

constexpr float kNothing = -745.f;  // a logarithm below it is that of no share at all

// One outcome of probabilities e^lp (teacher) and e^lq (student).
struct Outcome {
  float kd;     // its term
  float mass;   // q e, of C
  float share;  // of its gradient: q (e - C) without C
};
// e of an outcome with d = log p - log q (reverse and jsd).
__device__ __forceinline__ float slope_of(int kind, float mix, float d) {
  if (kind == LORA_DISTILL_REVERSE) return -d;
  return (mix - 1.f) * (d > 0.f ? d + log1pf((1.f - mix) * expm1f(-d)) : log1pf(mix * expm1f(d)));
}
__device__ __forceinline__ Outcome outcome(int kind, float mix, float lp, float lq) {
  if (lp < kNothing) lp = -INF_F;
  if (lq < kNothing) lq = -INF_F;
  const float p = expf(lp), q = expf(lq), d = lp - lq;
  Outcome o;
  if (kind == LORA_DISTILL_FORWARD) {
    const float w = expm1f(-d);  // q / p - 1
    o.kd = lq == -INF_F ? INF_F : term(p, q, -d, w);
    o.mass = 0.f;
    o.share = d < -16.f ? q - p : p * w;
  } else if (kind == LORA_DISTILL_REVERSE) {
    o.kd = lp == -INF_F ? INF_F : term(q, p, d, expm1f(d));
    o.mass = o.share = lq == -INF_F ? 0.f : lp == -INF_F ? INF_F : q * -d;
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
  if (lp == -INF_F && lq == -INF_F) o.kd = o.mass = o.share = 0.f;
  return o;
}
// q (e - C) of the rest, whose entries share it: 0 where the student gives the rest nothing.
__device__ __forceinline__ float rest_share(int kind, float mix, float lp, float lq, float C) {
  if (lq < kNothing) return 0.f;
  const float d = lp - lq;
  if (kind == LORA_DISTILL_FORWARD) {  // q - p by the greater of the two
    const float s = expf(fmaxf(lp, lq)) * expm1f(-fabsf(d));
    return d > 0.f ? s : -s;
  }
  const float q = expf(lq);
  return q == 0.f ? 0.f : q * (slope_of(kind, mix, d) - C);
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
//     kd 2^((x - base) log2(e) / temperature) + ce 2^((x - base) log2 e - l2_plain).
struct Slope {
  float base, kd, ce, l2_plain;
};

template <typename E, bool kBoth>
__device__ __forceinline__ uint4 slope_vector(const uint4& x, const Slope& g, const Terms& terms, const Terms& plain) {
  constexpr int kPairs = Elem<E>::kPairs;
  const uint64_t nb = pair_of(-g.base, -g.base), hi = pair_of(terms.near, terms.near);
  const uint64_t c = pair_of(g.kd, g.kd);
  uint64_t f[kPairs];
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    const uint64_t d = add2(Elem<E>::pair(x, j), nb);
    float a, b;
    split(mul2(d, hi), a, b);
    f[j] = mul2(c, pair_of(ex2(a), ex2(b)));
    if (kBoth) {
      split(fma2(d, pair_of(plain.near, plain.near), pair_of(-g.l2_plain, -g.l2_plain)), a, b);
      f[j] = fma2(pair_of(g.ce, g.ce), pair_of(ex2(a), ex2(b)), f[j]);
    }
  }
  return Elem<E>::pack(f);
}
template <bool kBoth>
__device__ __forceinline__ float slope_entry(float x, const Slope& g, const Terms& terms, const Terms& plain) {
  const float d = x - g.base;
  float f = g.kd * ex2(d * terms.near);
  if (kBoth) f = fmaf(g.ce, ex2(fmaf(d, plain.near, -g.l2_plain)), f);
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
constexpr int kHeld = 256;  // threads that hold a row's share
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
  float base, lt, l1;  // lt: log of the sum at the temperature, l1: at temperature 1
  float lr;            // log of the rest's share
  float m, rest;       // the rest's largest logit and its sum over that
  float scale;         // an entry's share of the row over its term of that sum
  bool none, taught;   // nothing is visible; the teacher says something (and the student too)
};
__device__ __forceinline__ RowTotal row_total(const RowSum& s, const float4& list, float list_plain, const Terms& terms, bool both) {
  RowTotal r;
  // the two sums over the greater base
  const bool some = list.w != 0.f, lists = some && list.z > s.m;
  r.base = base_of(lists ? list.z : s.m);
  const float fall = some ? fminf(s.m, list.z) - r.base : 0.f;  // of the other
  const float e = expf(fall * terms.inv);
  const float down = lists ? e : 1.f, rest = s.rest * down;
  const float total = rest + (lists ? list.w : some ? list.w * e : 0.f);
  r.m = base_of(s.m);
  r.rest = s.rest;
  r.scale = __fdividef(down, total);
  r.lt = r.l1 = logf(total);
  if (both) {
    const float e1 = expf(fall);
    r.l1 = logf(lists ? fmaf(s.plain, e1, list_plain) : some ? fmaf(list_plain, e1, s.plain) : s.plain);
  }
  r.none = total == 0.f;
  r.taught = list.y != -INF_F && !r.none;
  // (from far below the list by the logarithm of the rest's own sum: its part of the row's vanishes)
  const bool far = lists && fall * terms.inv < -60.f;
  r.lr = logf(far ? s.rest : __fdividef(rest, total)) + (far ? fall * terms.inv - r.lt : 0.f);
  return r;
}
// The slope of a row whose gradient of kd has the factor kw and of ce cw, with the rest's share of the former.  At
// temperature 1 the two share their powers.
template <bool kBoth>
__device__ __forceinline__ Slope rest_slope(const RowTotal& r, float kw, float cw, float share) {
  const float l1 = r.l1 + (r.base - r.m);
  Slope g{r.m, share == 0.f ? 0.f : kw * __fdividef(share, r.rest), cw, l1 * kLog2e + l1 * kLog2eLo};
  if (!kBoth && cw != 0.f) g.kd += cw * r.scale;
  return g;
}

template <typename E, int kG, int kVec, bool kBoth>
__global__ void __launch_bounds__(kG + 32, kVec > 8 ? 2 : 3) held_kernel(const __grid_constant__ DistillArgs a) {
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
      float C = 0.f;
      if (!forward) meet<3, kAll>();
      if (!forward) C = sh.C;
      float kw, cw;
      factors(r_, in, s.bad, C, &kw, &cw);
      const float share =
          kw != 0.f && r_.taught ? rest_share(a.opt.kind, a.opt.mix, in.tail - list.x * terms.inv - list.y, r_.lr, C) : 0.f;
      const Slope g = rest_slope<kBoth>(r_, kw, cw, share);
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
      // place, which takes this CTA's sums, sent after the barriers below: they are in shared
      // memory, the label's too (read back from there, so that its load ends here).
      if (lane == 0) {
        sh.bad[turn] = bad;
        sh.label_logit = xl;
      }
      const bool label_mine = mine(label), label_listed = label_mine && (bits[(label - first) >> 5] >> ((label - first) & 31) & 1);
      // (written as threads write, before the next copy takes its place)
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      meet<1, kAll>();
      meet<2, kAll>();
      xl = sh.label_logit;
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
            const float share = kw != 0.f && r.taught ? rest_share(a.opt.kind, a.opt.mix, tail_p, tail_q, C) : 0.f;
            const float x = xl - r.base, part = share == 0.f ? 0.f : share * __fdividef(expf((xl - r.m) * terms.inv), r.rest);
            out[label] = Elem<E>::put(kw * part + cw * ((kBoth ? expf(x - r.l1) : expf(x * terms.inv - r.lt)) - 1.f));
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

// -------------------------------------------------------------- streamed form --
//
// Many rows, short rows and the longest: a CTA a row, which it reads for its
// sum and again for its gradient.  Few rows are under way (one to sixteen an SM), so the
// second read finds the row in L2; outputs are written past it.  A row costs its barriers
// once, not once in each of a cluster's CTAs, and its CTA has no other to wait for.
//
// Listed entries: a bit an entry and a bit a vector.  A vector with a listed entry is left
// out of the sum as it goes by; the thread of the lowest entry of such a vector adds what
// is not listed of it.

constexpr int kBatch = 4;  // vectors a thread takes at once

template <int kT>
struct StreamShared {
  uint64_t probe_bar;
  float4 part[kT / 32];               // m, the sum, its sum at temperature 1
  float4 lists[kMaxList / 32];        // a warp's entries: teacher's maximum and sum, student's
  float lists_plain[kMaxList / 32];
  float2 outcomes[kMaxList / 32 + 1];  // kd, mass; the rest's last
};

// What L2 does with lines: keeps those that will be read again, gives up the others first.
__device__ __forceinline__ uint64_t keep_lines() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t drop_lines() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint4 load_as(const uint4* p, uint64_t policy) {
  uint4 v;
  asm volatile("ld.global.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p), "l"(policy)
               : "memory");
  return v;
}
__device__ __forceinline__ void store_as(void* p, const uint4& v, uint64_t policy) {
  asm volatile("st.global.L2::cache_hint.v4.u32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w),
               "l"(policy)
               : "memory");
}

template <typename E, int kT, bool kBoth>
__global__ void __launch_bounds__(kT, 1024 / kT) stream_kernel(const __grid_constant__ DistillArgs a) {
  constexpr int kN = Elem<E>::kN, kW = kT / 32;
  extern __shared__ uint32_t bits[];  // of the entries, then of the vectors
  __shared__ StreamShared<kT> sh;
  const int id = (int)threadIdx.x, lane = id & 31, warp = id >> 5;
  uint32_t* const flags = bits + (a.V + 31) / 32;
  const int words = (a.V + 31) / 32 + (a.V / kN / (kBatch * kT) + 1) * kBatch * kW;
  for (int i = id; i < words; i += kT) bits[i] = 0;
  pdl_wait_then_release();
  if (a.probe > 0) {
    if (id == 0 && !wait_probe(&sh.probe_bar, a.probe)) report(a.err, LORA_DERR_TIMEOUT);
    return;
  }
  const bool forward = a.opt.kind == LORA_DISTILL_FORWARD, lists = warp * 32 < a.k;
  const Terms terms = a.terms, plain = a.plain;
  __syncthreads();
  auto row_at = [&](long long t) { return static_cast<const E*>(a.logits) + t * a.ld; };
  // batch i0 .. of a row's middle
  uint4 next[kBatch];
  const uint64_t keep = keep_lines(), drop = drop_lines();
  auto load = [&](const uint4* mid, int nvec, int i0, uint64_t policy) {
    const uint4* const p = mid + i0 + id;
    if (i0 + kBatch * kT <= nvec) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) next[u] = load_as(p + u * kT, policy);
    } else {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) next[u] = i0 + u * kT + id < nvec ? load_as(p + u * kT, policy) : low_vector<E>();
    }
  };
  long long loaded = -1;  // the row whose first batch is in next
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int label = a.labels != nullptr ? a.labels[t] : -1;
    const E* const row = row_at(t);
    E* const out = a.dlogits == nullptr ? nullptr : static_cast<E*>(a.dlogits) + t * a.ldd;
    const Cut<E> c = cut_row(row, a.V, 0, 1);
    if (a.labels != nullptr && (label < 0 || label >= a.V)) {
      if (id == 0) {
        if (label >= a.V) report(a.err, LORA_DERR_BAD_LABEL);
        put_nothing(a, t);
      }
      if (out != nullptr) zero_share<E, kT>(c, out, a.V, id);
      continue;
    }
    const uint4* const mid = reinterpret_cast<const uint4*>(row + c.head);
    if (loaded != t) load(mid, c.nvec, 0, keep);
    const RowIn in = row_in(a, t, label);
    // the list
    int v = -1;
    float value = -INF_F, x = -INF_F;
    if (id < a.k) {
      v = a.ids[t * a.k + id];
      value = a.values[t * a.k + id];
      if (value == -INF_F) v = -1;
      if (v < 0) value = -INF_F;
    }
    const float xl = label >= 0 ? Elem<E>::get(row[label]) : 0.f;
    const int e = edge_of(c, a.V, id);
    float xe = e >= 0 ? Elem<E>::get(row[e]) : -INF_F;
    bool bad = v >= a.V;
    const bool on = v >= 0 && !bad;
    const int vec = on && v >= c.head && v < c.tail0 ? (v - c.head) / kN : -1;
    if (on) {
      x = Elem<E>::get(row[v]);
      bad = (atomicOr(&bits[v >> 5], 1u << (v & 31)) >> (v & 31) & 1) != 0;
      if (vec >= 0) atomicOr(&flags[vec >> 5], 1u << (vec & 31));
    }
    if (lists) {
      const float mv = warp_max(value), sv = warp_add(v >= 0 ? expf((value - base_of(mv)) * terms.inv) : 0.f);
      const float mx = warp_max(x), sx = warp_add(on ? expf((x - base_of(mx)) * terms.inv) : 0.f);
      const float s1 = kBoth ? warp_add(on ? expf(x - base_of(mx)) : 0.f) : 0.f;
      if (lane == 0) {
        sh.lists[warp] = make_float4(mv, sv, mx, sx);
        sh.lists_plain[warp] = s1;
      }
    }
    if (__syncthreads_or(bad)) {
      if (id == 0) {
        report(a.err, LORA_DERR_BAD_LABEL);
        put_nothing(a, t);
      }
      if (out != nullptr) zero_share<E, kT>(c, out, a.V, id);
      if (on) bits[v >> 5] = 0;
      if (vec >= 0) flags[vec >> 5] = 0;
      __syncthreads();
      continue;
    }
    auto listed = [&](int i) { return (bits[i >> 5] >> (i & 31) & 1) != 0; };
    if (e >= 0 && listed(e)) xe = -INF_F;
    const bool label_listed = label >= 0 && listed(label);
    // the rest's sum
    Sum s{-INF_F, 0.f};
    float s1 = 0.f;  // over the same base
    auto add = [&](const auto& r, float top) {
      const float m = fmaxf(s.m, top), base = base_of(m);
      const float more = power_sum<E>(terms, r, base), more1 = kBoth ? power_sum<E>(plain, r, base) : 0.f;
      if (m != s.m) {
        s.s *= expf((s.m - base) * terms.inv);
        if (kBoth) s1 *= expf(s.m - base);
      }
      s = Sum{m, s.s + more};
      s1 += more1;
    };
    for (int i0 = 0; i0 < c.nvec; i0 += kBatch * kT) {
      uint4 r[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) r[u] = next[u];
      // the next batch, or the gradient's first
      const int i1 = i0 + kBatch * kT;
      load(mid, c.nvec, i1 < c.nvec ? i1 : 0, i1 < c.nvec ? keep : drop);
      // (the words are the warp's, a bit a lane; those past the row's end are 0)
      uint32_t some[kBatch], any = 0;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) any |= some[u] = flags[(i0 >> 5) + u * kW + warp];
      if (any != 0)
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (some[u] >> lane & 1) r[u] = low_vector<E>();
      add(r, Elem<E>::top(r));
    }
    {  // a listed entry's vector, and the edges
      uint4 r[1] = {low_vector<E>()};
      if (vec >= 0) {
        uint32_t which = 0;
        const int from = c.head + vec * kN;
#pragma unroll
        for (int j = 0; j < kN; ++j) which |= (uint32_t)listed(from + j) << j;
        if (v == from + __ffs(which) - 1) r[0] = without(mid[vec], which, E{});
      }
      add(r, Elem<E>::top(r));
      if (e >= 0) {
        const float m = fmaxf(s.m, xe), base = base_of(m), fall = s.m - base;
        s = Sum{m, s.s * expf(fall * terms.inv) + expf((xe - base) * terms.inv)};
        if (kBoth) s1 = s1 * expf(fall) + expf(xe - base);
      }
    }
    {
      const float m = warp_max(s.m), fall = s.m - base_of(m);
      const float sum = warp_add(s.s * expf(fall * terms.inv)), sum1 = kBoth ? warp_add(s1 * expf(fall)) : 0.f;
      if (lane == 0) sh.part[warp] = make_float4(m, sum, sum1, 0.f);
    }
    __syncthreads();
    if (on) bits[v >> 5] = 0;
    if (vec >= 0) flags[vec >> 5] = 0;
    // the row's sums and the lists', as every warp works them out
    const RowSum rs = join_parts(sh.part, kW, terms, kBoth, lane);
    float4 list;
    float list_plain;
    {
      const bool has = lane * 32 < a.k;
      const float4 q = has ? sh.lists[lane] : make_float4(-INF_F, 0.f, -INF_F, 0.f);
      const float high = base_of(fmaxf(warp_max(q.x), in.tail * a.opt.temperature)), mx = base_of(warp_max(q.z));
      // (a part with nothing has base 0, which can lie above the row's by any amount: no factor for it)
      auto part_of = [](float sum, float power) { return sum == 0.f ? 0.f : sum * expf(power); };
      const float mass = warp_add(part_of(q.y, (base_of(q.x) - high) * terms.inv)) + expf(in.tail - high * terms.inv);
      list = make_float4(high, logf(mass), mx, warp_add(part_of(q.w, (base_of(q.z) - mx) * terms.inv)));
      list_plain = kBoth ? warp_add(has ? part_of(sh.lists_plain[lane], base_of(q.z) - mx) : 0.f) : 0.f;
    }
    const RowTotal r = row_total(rs, list, list_plain, terms, kBoth);
    const float tail_p = in.tail - list.x * terms.inv - list.y, tail_q = r.lr;
    // the outcomes: the entries', and the rest's by the last warp
    Outcome o{0.f, 0.f, 0.f};
    if (r.taught && (lists ? v >= 0 : id == kT - 1)) {
      const float lp = lists ? (value - list.x) * terms.inv - list.y : tail_p;
      const float lq = lists ? (x - r.base) * terms.inv - r.lt : tail_q;
      o = forward ? outcome(LORA_DISTILL_FORWARD, 0.f, lp, lq) : other_outcome(a.opt.kind, a.opt.mix, lp, lq);
    }
    if (lists || warp == kW - 1) {
      const float kd = warp_add(o.kd), mass = warp_add(o.mass);
      if (lane == 0) sh.outcomes[lists ? warp : kMaxList / 32] = make_float2(kd, mass);
    }
    auto all_outcomes = [&] {
      const float2 q = lane * 32 < a.k || lane == kMaxList / 32 ? sh.outcomes[lane] : make_float2(0.f, 0.f);
      return make_float2(warp_add(q.x), warp_add(q.y));
    };
    float C = 0.f;
    if (!forward) {
      __syncthreads();
      C = all_outcomes().y;
    }
    const float gs = r.none || in.weight == 0.f ? 0.f : a.opt.grad_scale * in.weight;
    const float kw = gs != 0.f && fabsf(C) != INF_F ? gs * a.opt.kd_weight * terms.inv : 0.f;
    const float cw = a.opt.ce_weight > 0.f ? gs * a.opt.ce_weight : 0.f;
    const float share = kw != 0.f && r.taught ? rest_share(a.opt.kind, a.opt.mix, tail_p, tail_q, C) : 0.f;
    const Slope g = rest_slope<kBoth>(r, kw, cw, share);
    if (out != nullptr) {
      if (g.kd == 0.f && (!kBoth || cw == 0.f)) {
        zero_share<E, kT>(c, out, a.V, id);
      } else {
        const bool wide = on_boundary(out, c);
        E* const dst = out + c.head;
        for (int i0 = 0; i0 < c.nvec; i0 += kBatch * kT) {
          uint4 y[kBatch];
#pragma unroll
          for (int u = 0; u < kBatch; ++u) y[u] = next[u];
          const int i1 = i0 + kBatch * kT;
          if (i1 < c.nvec) {
            load(mid, c.nvec, i1, drop);
          } else if (t + gridDim.x < a.T) {  // the next row's first
            loaded = t + gridDim.x;
            const Cut<E> d = cut_row(row_at(loaded), a.V, 0, 1);
            load(reinterpret_cast<const uint4*>(d.row + d.head), d.nvec, 0, keep);
          }
          E* const to = dst + (long long)(i0 + id) * kN;
          if (wide && i1 <= c.nvec) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) store_as(to + u * kT * kN, slope_vector<E, kBoth>(y[u], g, terms, plain), drop);
          } else {
            for (int u = 0; u < kBatch && i0 + u * kT + id < c.nvec; ++u) {
              uint4 x = y[0];
#pragma unroll
              for (int k = 1; k < kBatch; ++k) x = u == k ? y[k] : x;
              const uint4 z = slope_vector<E, kBoth>(x, g, terms, plain);
              if (wide) {
                store_as(to + u * kT * kN, z, drop);
              } else {
#pragma unroll
                for (int j = 0; j < kN; ++j) to[u * kT * kN + j] = Elem<E>::entry(z, j);
              }
            }
          }
        }
        // (the edge's logit again: the sum's may be taken out)
        if (e >= 0) out[e] = Elem<E>::put(slope_entry<kBoth>(xe, g, terms, plain));
      }
    }
    __syncthreads();  // the listed places are written last
    if (out != nullptr && (kw != 0.f || cw != 0.f)) {
      if (on) {
        const float d = x - r.base;
        float y = kw != 0.f && r.taught ? kw * o.share : 0.f;
        if (!forward || cw != 0.f) {
          const float q = expf(d * terms.inv - r.lt);
          if (!forward && kw != 0.f) y -= kw * q * C;
          if (cw != 0.f) y += cw * ((kBoth ? expf(d - r.l1) : q) - (v == label ? 1.f : 0.f));
        }
        out[v] = Elem<E>::put(y);
      }
      if (id == kT - 1 && label >= 0 && !label_listed && cw != 0.f) {
        const float d = xl - r.base, part = share == 0.f ? 0.f : share * __fdividef(expf((xl - r.m) * terms.inv), r.rest);
        out[label] = Elem<E>::put(kw * part + cw * ((kBoth ? expf(d - r.l1) : expf(d * terms.inv - r.lt)) - 1.f));
      }
    }
    if (warp == kW - 1) {
      const float kd = all_outcomes().x;
      if (lane == 0) {
        const float ce = a.opt.ce_weight > 0.f ? (r.none ? INF_F : r.l1 - (xl - r.base)) : 0.f;
        put_losses(a, t, in, r.none ? (list.y != -INF_F ? INF_F : 0.f) : kd, ce);
      }
    }
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

template <typename E, int kT>
lora_status_t launch_stream(DistillArgs& a, cudaStream_t s) {
  const void* f = a.both ? (const void*)stream_kernel<E, kT, true> : (const void*)stream_kernel<E, kT, false>;
  const size_t batch = (size_t)kBatch * kT;  // flags for whole batches
  const size_t smem = 4 * (((size_t)a.V + 31) / 32 + (a.V / Elem<E>::kN / batch + 1) * (batch / 32));
  if (smem > 200000) return LORA_ERR_UNSUPPORTED;
  if (ensure_smem_attr(f, smem) != cudaSuccess) return LORA_ERR_CUDA;
  const int ctas = std::min(a.T, 1024 / kT * sm_count());
  return launch_pdl(f, dim3((unsigned)ctas), dim3(kT), smem, s, 0, &a) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

// The form of the rows (device times in us on a GB300, 64 listed, forward; streamed with 256 /
// 512 / 1024 threads a row, 4 / 2 / 1 rows an SM at once):
//  - held while the rows' clusters of 16 vectors a thread are one wave and a row is more than
//    64 KB.  16 x 128256 bf16: 8.5, streamed 17.7 / 15.3 / 15.9; 64: 12.5, 21.4 / 16.6 / 16.7;
//    150 (two waves): 27.2, 23.4 / 19.0 / 18.4.  64 x 32000: 8.7, 8.1 / 8.0 / 9.1.
//  - else streamed, with so many rows at once that L2 holds them.  8192 x 32000 bf16: 216 / 308 /
//    463 (held 245); 4000 x 50257 with jsd 178 / 224 / 350 (270); 8192 x 128256 929 / 806 / 933
//    (935); 2000 x 151936 fp32 584 / 545 / 509.
//  - of short rows more at once, 64 / 128 / 256 threads: 8192 x 1000 34 / 50 / 87; 8192 x 5000 56 / 73 /
//    99; 4096 x 10000 41 / 50 / 69; 4096 x 20000 74 / 72 / 88; 4096 x 32000 124 / 113 / 110. Few rows:
//    600 x 5000 7.6 / 7.6 / 8.8, 300 x 10000 8.4 / 7.3 / 7.5.
// The last warp has no entries: it works out the rest.
template <typename E>
lora_status_t launch(DistillArgs& a, cudaStream_t s) {
  const int sms = sm_count(), last = 32;
  const long long vec = a.V / Elem<E>::kN, places = 2LL * sms, bytes = (long long)a.V * (long long)sizeof(E);
  auto ctas = [&](int vecs) {
    int n = 1;
    while (vec > (long long)n * kHeld * vecs) n *= 2;
    return n;
  };
  if (bytes > 65536 && ctas(16) <= kMaxCluster && (long long)a.T * ctas(16) <= places) {
    for (int vecs = 4; vecs <= 8; vecs *= 2)
      if (ctas(vecs) <= kMaxCluster && (long long)a.T * ctas(vecs) <= places)
        return vecs == 4 ? launch_held<E, kHeld, 4>(a, ctas(4), s) : launch_held<E, kHeld, 8>(a, ctas(8), s);
    return launch_held<E, kHeld, 16>(a, ctas(16), s);
  }
  if (bytes <= 24000 && a.T > 2 * sms && a.k <= 64 - last) return launch_stream<E, 64>(a, s);
  if (bytes <= 48000 && a.T > sms && a.k <= 128 - last) return launch_stream<E, 128>(a, s);
  if (a.k <= 256 - last && bytes * 4 * sms <= 64 << 20 && (a.T > sms || bytes <= 32768)) return launch_stream<E, 256>(a, s);
  if (bytes * 2 * sms <= 96 << 20) return launch_stream<E, 512>(a, s);
  return launch_stream<E, 1024>(a, s);
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
  if (!temperature_ok(opts->temperature)) return LORA_ERR_INVALID_ARG;
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
