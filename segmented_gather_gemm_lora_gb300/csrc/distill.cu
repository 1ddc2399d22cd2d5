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

template <typename E>
__device__ __forceinline__ uint4 slope_vector(const uint4& x, const Slope& g, const Terms& terms, const Terms& plain, bool both) {
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
    if (both) {
      split(fma2(d, pair_of(plain.hi, plain.hi), pair_of(-g.l2_plain, -g.l2_plain)), a, b);
      f[j] = fma2(pair_of(g.ce, g.ce), pair_of(ex2(a), ex2(b)), f[j]);
    }
  }
  return Elem<E>::pack(f);
}
__device__ __forceinline__ float slope_entry(float x, const Slope& g, const Terms& terms, const Terms& plain, bool both) {
  const float d = x - g.base;
  float f = g.kd * ex2(fmaf(d, terms.hi, -g.l2));
  if (both) f = fmaf(g.ce, ex2(fmaf(d, plain.hi, -g.l2_plain)), f);
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
// A row is held in the registers of a CTA of kG threads, or of the n CTAs of a cluster,
// from its sum to its gradient, kVec vectors a thread, so it is read once; the coming
// row's share arrives in shared memory meanwhile by a bulk copy.  (The held policy loss
// of logits.cu in that.)  What a list adds:
//  - thread j has the list's entry j, its place looked up in the row a row ahead; it takes
//    the place out of the share in shared memory (-inf) before the registers read it, so
//    the sum is of the rest alone and the rest's gradient needs no test;
//  - the listed entries' own maxima and sums go by warps through shared memory, each
//    entry's outcome is worked out by its thread once the rest's sum is known, and its
//    gradient is written over what the vectors left there;
//  - a bit an entry of the share shows what is listed twice.
// Sums cross the cluster as there: a warp sends its own to every CTA by an asynchronous
// store on that CTA's barrier for the row; two sets of slots are enough.
// Every wait is bounded.  A warp whose wait ran out reports it and goes through the
// remaining rows without waiting, copying or writing, its barriers matched.
//
// What bounds it: memory, one read and one write of the logits; then the latency of a
// row's barriers, which the other CTA of the SM hides.

constexpr int kMaxCluster = 8;

template <int kG>
struct HeldShared {
  uint64_t probe_bar, full, sums[2];
  float4 part[2][kMaxCluster * (kG / 32)];  // m, the rest's sum, its sum at temperature 1, a bad list
  float4 lists[kG / 32];                    // a warp's entries: teacher's maximum and sum, student's
  float lists_plain[kG / 32];               // student's sum at temperature 1
  float2 outcomes[kG / 32];                 // kd, mass
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

template <typename E, int kG, int kVec>
__global__ void __launch_bounds__(kG, (kVec > 8 ? 512 : 768) / kG) held_kernel(const __grid_constant__ DistillArgs a) {
  constexpr int kN = Elem<E>::kN, kW = kG / 32;
  extern __shared__ __align__(128) uint4 coming[];  // the coming row's share, then its bits
  __shared__ HeldShared<kG> sh;
  const int n = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, id = (int)threadIdx.x;
  const int group = (int)cluster_id_x(), groups = (int)ncluster_x();
  const int share = (a.V / kN + n - 1) / n;  // vectors of the largest share
  uint32_t* const bits = reinterpret_cast<uint32_t*>(coming + share);
  for (int i = id; i < (share * kN + 16 + 31) / 32; i += kG) bits[i] = 0;
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
  const bool lead = rank == 0 && id == 0, both = a.both != 0;
  const Terms terms = a.terms, plain = a.plain;
  auto row_at = [&](long long t) { return static_cast<const E*>(a.logits) + t * a.ld; };
  auto cut_at = [&](long long t) { return cut_row(row_at(t), a.V, rank, n); };
  auto out_at = [&](long long t) { return static_cast<E*>(a.dlogits) + t * a.ldd; };
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
  // The first row from t on that counts (without labels all do; their label is -1); the
  // rows before it are passed over.  *label: row t's, loaded before, then that row's.
  auto label_at = [&](long long t) { return a.labels != nullptr && t < a.T ? a.labels[t] : -1; };
  auto next_row = [&](long long t, int* label) {
    while (a.labels != nullptr && t < a.T) {
      if (*label >= 0 && *label < a.V) break;
      if (*label >= a.V && lead) report(a.err, LORA_DERR_BAD_LABEL);
      if (lead) put_nothing(a, t);
      if (a.dlogits != nullptr) zero_share<E, kG>(cut_at(t), out_at(t), a.V, id);
      t += groups;
      *label = label_at(t);
    }
    return t;
  };
  // Thread id's entry of row t's list (value -inf: none), and its place's logit.
  struct Listed {
    int id;
    float value;
  };
  auto list_at = [&](long long t) {
    Listed l{-1, -INF_F};
    if (id < a.k && t < a.T) {
      l.id = a.ids[t * a.k + id];
      l.value = a.values[t * a.k + id];
    }
    if (l.id < 0 || l.value == -INF_F) l = Listed{-1, -INF_F};
    return l;
  };
  auto logit_at = [&](long long t, int v) { return v >= 0 && v < a.V ? Elem<E>::get(row_at(t)[v]) : -INF_F; };

  int label = label_at(group), buf = 0;
  uint32_t parity = 0, sums_parity = 0;
  long long t = next_row(group, &label);
  if (id == 0 && t < a.T) fetch(t);
  bool dead = false;  // a wait of this warp's ran out
  Listed l = list_at(t);
  float x = t < a.T ? logit_at(t, l.id) : 0.f, xl = t < a.T ? logit_at(t, label) : 0.f;
  int nlabel = label_at(t + groups);
  while (t < a.T) {
    const RowIn in = row_in(a, t, label);
    const long long nt = next_row(t + groups, &nlabel);
    const int nnlabel = label_at(nt + groups);
    const Listed nl = list_at(nt);
    const Cut<E> c = cut_at(t);
    const int nv = c.v1 - c.v0, e = edge_of(c, a.V, id);
    float xe = e >= 0 ? Elem<E>::get(c.row[e]) : -INF_F;
    // the share's entries: [lo, hi)
    const int lo = c.first ? 0 : c.head + c.v0 * kN, hi = c.last ? a.V : c.head + c.v1 * kN;
    bool bad = l.id >= a.V;
    {  // the list's maxima and sums
      const float mv = warp_max(l.value), sv = warp_add(l.id >= 0 ? expf((l.value - base_of(mv)) * terms.inv) : 0.f);
      const float mx = warp_max(l.id >= 0 ? x : -INF_F), bx = base_of(mx);
      const float sx = warp_add(l.id >= 0 ? expf((x - bx) * terms.inv) : 0.f);
      const float s1 = both ? warp_add(l.id >= 0 ? expf(x - bx) : 0.f) : 0.f;
      if (lane == 0) {
        sh.lists[warp] = make_float4(mv, sv, mx, sx);
        sh.lists_plain[warp] = s1;
      }
    }
    if (!dead) {
      dead = __any_sync(0xffffffffu, !mbar_wait(smem_u32(&sh.full), parity));
      if (!dead) parity ^= 1;
    }
    const bool mine = l.id >= lo && l.id < hi;
    if (mine) {
      const int at = l.id - lo, v = l.id - c.head - c.v0 * kN;
      bad |= (atomicOr(&bits[at >> 5], 1u << (at & 31)) >> (at & 31) & 1) != 0;
      if (!dead && v >= 0 && v < nv * kN) reinterpret_cast<E*>(coming)[v] = Elem<E>::put(-INF_F);
      // (written as threads write, before the next copy takes its place)
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    bad = __any_sync(0xffffffffu, bad);
    __syncthreads();
    auto listed = [&](int v) { return (bits[(v - lo) >> 5] >> ((v - lo) & 31) & 1) != 0; };
    if (e >= 0 && listed(e)) xe = -INF_F;
    const bool label_mine = label >= lo && label < hi, label_listed = label_mine && listed(label);
    uint4 r[kVec];
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      r[u] = low_vector<E>();
      if (u * kG + id < nv) r[u] = coming[u * kG + id];
    }
    __syncthreads();
    if (mine) bits[(l.id - lo) >> 5] = 0;
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
    float rest = e >= 0 ? terms.power(xe, base_of(m)) : 0.f, rest_plain = both && e >= 0 ? plain.power(xe, base_of(m)) : 0.f;
#pragma unroll
    for (int u = 0; u < kVec; u += 4)
      if (u * kG < nv) {
        const uint4 four[4] = {r[u], r[u + 1], r[u + 2], r[u + 3]};
        rest += power_sum<E>(terms, four, base_of(m));
        if (both) rest_plain += power_sum<E>(plain, four, base_of(m));
      }
    rest = warp_add(rest);
    if (both) rest_plain = warp_add(rest_plain);
    bool bad_row = false;
    if (!dead) {
      const uint32_t bar = smem_u32(&sh.sums[buf]);
      if (id == 0) mbar_arrive_expect_tx(bar, (uint32_t)(n * kW * sizeof(float4)));
      // the load of the label's logit is over before any CTA can write a gradient in its
      // place: its value decides the sign of this zero
      const float flag = bad ? 1.f : __float_as_uint(xl) == 0x7fc0d15cu ? -0.f : 0.f;
      if (lane < n)
        st_async_v4(mapa(smem_u32(&sh.part[buf][rank * kW + warp]), lane), make_float4(m, rest, rest_plain, flag), mapa(bar, lane));
      dead = __any_sync(0xffffffffu, !mbar_wait_cluster(bar, sums_parity));
      m = -INF_F;
      for (int k = lane; k < n * kW; k += 32) m = fmaxf(m, sh.part[buf][k].x);
      m = warp_max(m);
      rest = rest_plain = 0.f;
      for (int k = lane; k < n * kW; k += 32) {
        const float4 q = sh.part[buf][k];
        rest += q.y * expf((q.x - base_of(m)) * terms.inv);
        if (both) rest_plain += q.z * expf(q.x - base_of(m));
        bad_row |= q.w != 0.f;
      }
      rest = warp_add(rest);
      if (both) rest_plain = warp_add(rest_plain);
      bad_row = __any_sync(0xffffffffu, bad_row);
      sums_parity ^= buf;
      buf ^= 1;
    }
    // the coming row's logits of its list (its ids are here by now)
    const float nx = nt < a.T ? logit_at(nt, nl.id) : 0.f, nxl = nt < a.T ? logit_at(nt, nlabel) : 0.f;
    // the lists' sums over the warps, and the row's
    const float4 q = lane < kW ? sh.lists[lane] : make_float4(-INF_F, 0.f, -INF_F, 0.f);
    const float mv = warp_max(q.x), mx = warp_max(q.z);
    const float high = base_of(fmaxf(mv, in.tail * a.opt.temperature));  // in the values' measure
    const float sv = warp_add(q.y * expf((q.x - high) * terms.inv));
    const float base = base_of(fmaxf(m, mx));
    const float sx = warp_add(q.w * expf((q.z - base) * terms.inv));
    rest *= expf((base_of(m) - base) * terms.inv);
    const float total = rest + sx, lt = logf(total);
    float all = total;
    if (both)
      all = rest_plain * expf(base_of(m) - base) + warp_add(lane < kW ? sh.lists_plain[lane] * expf(q.z - base) : 0.f);
    const float tail = in.tail - high * terms.inv, mass = sv + expf(tail), lm = logf(mass);
    Outcome o{0.f, 0.f, 0.f, 0.f}, r_ = o;
    const bool none = total == 0.f;  // nothing is visible
    const float lq = (x - base) * terms.inv - lt;
    if (mass != 0.f && !none) {
      if (l.id >= 0) o = outcome(a.opt.kind, a.opt.mix, (l.value - high) * terms.inv - lm, lq);
      r_ = outcome(a.opt.kind, a.opt.mix, tail - lm, logf(rest) - lt);
    }
    {
      const float kd = warp_add(o.kd), taken = warp_add(o.mass);
      if (lane == 0) sh.outcomes[warp] = make_float2(kd, taken);
    }
    float C = 0.f, kd = 0.f;
    if (a.opt.kind != LORA_DISTILL_FORWARD) {
      __syncthreads();
      const float2 s = lane < kW ? sh.outcomes[lane] : make_float2(0.f, 0.f);
      kd = warp_add(s.x) + r_.kd;
      C = warp_add(s.y) + r_.mass;
    }
    const bool cew = a.opt.ce_weight > 0.f;
    const float gs = none || in.weight == 0.f || bad_row ? 0.f : a.opt.grad_scale * in.weight;
    const bool kd_on = gs != 0.f && fabsf(C) != INF_F;
    const float kw = kd_on ? gs * a.opt.kd_weight * terms.inv : 0.f, cw = cew ? gs * a.opt.ce_weight : 0.f;
    // at temperature 1 the two parts of the gradient share their powers
    Slope g{base, rest > 0.f || rest != rest ? kw * (r_.slope - C) : 0.f, lt * kLog2e + lt * kLog2eLo, cw, 0.f};
    if (kw == 0.f) g.kd = 0.f;
    const float l1 = both ? logf(all) : lt;
    if (both) g.l2_plain = l1 * kLog2e + l1 * kLog2eLo;
    else g.kd += cw;
    const bool zero = (g.kd == 0.f && (!both || cw == 0.f)) || gs == 0.f;
    E* const out = a.dlogits == nullptr || dead ? nullptr : out_at(t);
    if (out != nullptr) {
      if (zero) {
        zero_share<E, kG>(c, out, a.V, id);
      } else {
        E* const dst = out + c.head + (long long)c.v0 * kN;
        if (on_boundary(out, c)) {
#pragma unroll
          for (int u = 0; u < kVec; ++u)
            if (u * kG + id < nv) reinterpret_cast<uint4*>(dst)[u * kG + id] = slope_vector<E>(r[u], g, terms, plain, both);
        } else {
#pragma unroll
          for (int u = 0; u < kVec; ++u)
            if (u * kG + id < nv) {
              const uint4 y = slope_vector<E>(r[u], g, terms, plain, both);
#pragma unroll
              for (int j = 0; j < kN; ++j) dst[(u * kG + id) * kN + j] = Elem<E>::entry(y, j);
            }
        }
        if (e >= 0) out[e] = Elem<E>::put(slope_entry(xe, g, terms, plain, both));
      }
    }
    __syncthreads();  // the listed places are written last
    if (out != nullptr && gs != 0.f) {
      if (mine) {
        const float q_ = expf(lq);
        float y = kw != 0.f ? kw * (a.opt.kind == LORA_DISTILL_FORWARD ? o.share : o.share - q_ * C) : 0.f;
        if (cw != 0.f) y += cw * ((both ? expf(x - base - l1) : q_) - (l.id == label ? 1.f : 0.f));
        out[l.id] = Elem<E>::put(y);
      }
      if (id == 0 && label_mine && !label_listed && cw != 0.f) out[label] = Elem<E>::put(slope_entry(xl, g, terms, plain, both) - cw);
    }
    if (lead && !dead) {
      if (bad_row) {
        report(a.err, LORA_DERR_BAD_LABEL);
        put_nothing(a, t);
      } else {
        if (a.opt.kind == LORA_DISTILL_FORWARD) {
          kd = r_.kd;
          for (int w = 0; w < kW; ++w) kd += sh.outcomes[w].x;
        }
        const float ce = cew ? (none ? INF_F : l1 - (xl - base)) : 0.f;
        put_losses(a, t, in, none ? (mass > 0.f ? INF_F : 0.f) : kd, ce);
      }
    }
    if (dead && lane == 0) report(a.err, LORA_DERR_TIMEOUT);
    t = nt;
    label = nlabel;
    nlabel = nnlabel;
    l = nl;
    x = nx;
    xl = nxl;
  }
  if (dead && id == 0) mbar_wait(smem_u32(&sh.full), parity);
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
  Outcome o{0.f, 0.f, 0.f, 0.f}, r = o;
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

// -------------------------------------------------------------------- host --

template <typename E, int kG, int kVec>
lora_status_t launch_held(DistillArgs& a, int n, cudaStream_t s) {
  const void* f = (const void*)held_kernel<E, kG, kVec>;
  const size_t share = (size_t)(a.V / Elem<E>::kN + n - 1) / n;
  const size_t smem = share * 16 + (share * Elem<E>::kN + 16 + 31) / 32 * 4;
  if (ensure_smem_attr(f, smem) != cudaSuccess) return LORA_ERR_CUDA;
  const long long ctas = std::min((long long)a.T * n, (long long)max_active_clusters(f, kG, smem, n) * n);
  return launch_pdl(f, dim3((unsigned)ctas), dim3(kG), smem, s, n, &a) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
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
