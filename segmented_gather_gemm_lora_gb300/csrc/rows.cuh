// Rows of logits: their elements by vectors of 16 bytes, running sums of
// exponentials, and the checks that every call on logits makes of its rows.
#pragma once

#include "common.cuh"
#include "lora_train.h"
#include "pairs.cuh"

namespace lora {

constexpr float kLog2e = 1.4426950408889634f;    // log2 e to fp32 and what that leaves (the rounding
constexpr float kLog2eLo = 1.9259629911267e-8f;  // has one sign in every row: sums of logp gather it)
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
  // a word's elements as a pair, a pair as a word, the larger of a word's
  static constexpr int kPairs = 4;
  static __device__ __forceinline__ uint64_t pair(const uint4& v, int k) {
    const uint32_t u = k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w;
    return pair_of(bf_lo(u), bf_hi(u));
  }
  static __device__ __forceinline__ uint4 pack(const uint64_t (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a, b;
      split(f[k], a, b);
      w[k] = pack_bf16x2(a, b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ uint16_t entry(const uint4& v, int k) {
    const uint32_t u = k < 2 ? v.x : k < 4 ? v.y : k < 6 ? v.z : v.w;
    return (uint16_t)(u >> (16 * (k & 1)));
  }
  // The largest element of some vectors: two at a time, as bf16 (no rounding).
  template <int N>
  static __device__ __forceinline__ float top(const uint4 (&v)[N]) {
    __nv_bfloat162 t = word(v[0].x);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      t = __hmax2(t, __hmax2(word(v[u].x), word(v[u].y)));
      t = __hmax2(t, __hmax2(word(v[u].z), word(v[u].w)));
    }
    return fmaxf(__low2float(t), __high2float(t));
  }
  static __device__ __forceinline__ __nv_bfloat162 word(uint32_t u) { return *reinterpret_cast<__nv_bfloat162*>(&u); }
};
template <>
struct Elem<float> {
  static constexpr int kN = 4;
  static constexpr uint32_t kMinusInf = 0xff800000u;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
  static constexpr int kPairs = 2;
  static __device__ __forceinline__ uint64_t pair(const uint4& v, int k) {
    return k == 0 ? pair_of(__uint_as_float(v.x), __uint_as_float(v.y)) : pair_of(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  static __device__ __forceinline__ uint4 pack(const uint64_t (&f)[2]) {
    float a, b, c, d;
    split(f[0], a, b);
    split(f[1], c, d);
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
  }
  static __device__ __forceinline__ float entry(const uint4& v, int k) {
    return __uint_as_float(k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w);
  }
  template <int N>
  static __device__ __forceinline__ float top(const uint4 (&v)[N]) {
    float t = -INF_F;
#pragma unroll
    for (int u = 0; u < N; ++u)
      t = fmaxf(fmaxf(t, fmaxf(__uint_as_float(v[u].x), __uint_as_float(v[u].y))),
                fmaxf(__uint_as_float(v[u].z), __uint_as_float(v[u].w)));
    return t;
  }
};

// A running sum of exponentials: its maximum m, and s = sum of exp(x - base(m)).
// Terms take the hardware's 2^x.  The few rescalings use expf: 2^x is 5e-8 low on
// average, which a rescaling would put on the whole sum, and a loss adds logp over
// hundreds of rows.
struct Sum {
  float m, s;
};
__device__ __forceinline__ float base_of(float m) { return fabsf(m) == INF_F ? 0.f : m; }
// The sum of two.  An empty one is {-inf, 0}.
__device__ __forceinline__ Sum join(const Sum& x, const Sum& y) {
  Sum r;
  r.m = fmaxf(x.m, y.m);
  const float base = base_of(r.m);
  r.s = x.s * expf(x.m - base) + y.s * expf(y.m - base);
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
__device__ __forceinline__ int edge_of(const Cut<E>& c, int V, int t) {
  if (c.first && t < c.head) return t;  // head and tail are below eight elements each
  if (c.last && t >= 16 && t - 16 < V - c.tail0) return c.tail0 + t - 16;
  return -1;
}

// The sum of exp(x - base) over some vectors.
template <typename E, int N>
__device__ __forceinline__ float exp_sum(const uint4 (&r)[N], float base) {
  constexpr int kPairs = Elem<E>::kPairs;
  const uint64_t hi = pair_of(kLog2e, kLog2e), lo = pair_of(kLog2eLo, kLog2eLo), nb = pair_of(-base, -base);
  uint64_t part = pair_of(0.f, 0.f);
#pragma unroll
  for (int u = 0; u < N; ++u) {
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      const uint64_t d = add2(Elem<E>::pair(r[u], k), nb);
      float a, b;
      split(fma2(d, hi, mul2(d, lo)), a, b);
      part = add2(part, pair_of(ex2(a), ex2(b)));
    }
  }
  float a, b;
  split(part, a, b);
  return a + b;
}

// Some vectors joined to t (their sum first: the running sum takes one addition).
template <typename E, int N>
__device__ __forceinline__ Sum add_vectors(Sum t, const uint4 (&r)[N]) {
  const float m = fmaxf(t.m, Elem<E>::top(r)), base = base_of(m);
  const float s = exp_sum<E>(r, base);
  if (m != t.m) t.s *= expf(t.m - base);
  return Sum{m, t.s + s};
}

// One element x, joined to t.
__device__ __forceinline__ Sum add_one(Sum t, float x) {
  return join(t, Sum{x, x == x ? (x == -INF_F ? 0.f : x == INF_F ? x : 1.f) : x});
}

template <typename E>
__device__ __forceinline__ uint4 low_vector() {
  return make_uint4(Elem<E>::kMinusInf, Elem<E>::kMinusInf, Elem<E>::kMinusInf, Elem<E>::kMinusInf);
}

// The sum of the lanes' sums: the maximum first, then one rescaling a lane.
__device__ __forceinline__ float warp_max(float m) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  return m;
}
__device__ __forceinline__ float warp_add(float s) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  return s;
}
__device__ __forceinline__ Sum warp_sum(const Sum& t) {
  const float m = warp_max(t.m);
  return Sum{m, warp_add(t.s * expf(t.m - base_of(m)))};
}

// Nothing of the row is visible (a NaN among the masked entries is).
__device__ __forceinline__ bool empty(const Sum& t) { return t.m == -INF_F && t.s == 0.f; }

template <typename E>
__device__ __forceinline__ bool on_boundary(const E* out, const Cut<E>& c) {
  return (reinterpret_cast<uintptr_t>(out + c.head) & 15) == 0;
}

// Terms exp((x - base) / temperature): log2(e) / temperature rounded, and the temperature's inverse.
struct Terms {
  float near, inv;
  __device__ __forceinline__ Sum join(const Sum& x, const Sum& y) const {
    Sum r;
    r.m = fmaxf(x.m, y.m);
    const float base = base_of(r.m);
    r.s = x.s * expf((x.m - base) * inv) + y.s * expf((y.m - base) * inv);
    return r;
  }
  __device__ __forceinline__ float power(float x, float base) const {  // of finite base
    return ex2((x - base) * near);
  }
  __device__ __forceinline__ Sum add(const Sum& t, float x) const {
    return join(t, Sum{x, x == x ? (x == -INF_F ? 0.f : x == INF_F ? x : 1.f) : x});
  }
  __device__ __forceinline__ Sum across(const Sum& t) const {  // the warp's lanes
    const float m = warp_max(t.m);
    return Sum{m, warp_add(t.s * expf((t.m - base_of(m)) * inv))};
  }
};

// The sum of exp((x - base) / temperature) over some vectors.  The factor is its greater part
// alone: the difference comes first, so what that leaves out moves a term by 1e-8 (x - base)
// of itself, and the terms that make the sum have small differences.
template <typename E, int N>
__device__ __forceinline__ float power_sum(const Terms& e, const uint4 (&r)[N], float base) {
  constexpr int kPairs = Elem<E>::kPairs;
  const uint64_t hi = pair_of(e.near, e.near), nb = pair_of(-base, -base);
  uint64_t part = pair_of(0.f, 0.f);
#pragma unroll
  for (int u = 0; u < N; ++u) {
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      float a, b;
      split(mul2(add2(Elem<E>::pair(r[u], k), nb), hi), a, b);
      part = add2(part, pair_of(ex2(a), ex2(b)));
    }
  }
  float a, b;
  split(part, a, b);
  return a + b;
}

// Some vectors, whose largest element is top, joined to t.
template <typename E, int N>
__device__ __forceinline__ Sum add_vectors(const Terms& e, Sum t, const uint4 (&r)[N], float top) {
  const float m = fmaxf(t.m, top), base = base_of(m);
  const float s = power_sum<E>(e, r, base);
  if (m != t.m) t.s *= expf((t.m - base) * e.inv);
  return Sum{m, t.s + s};
}

// The largest element of a vector, NaN if one is.
__device__ __forceinline__ float top_nan(const uint4& v, uint16_t) {
  const __nv_bfloat162 t = __hmax2_nan(__hmax2_nan(Elem<uint16_t>::word(v.x), Elem<uint16_t>::word(v.y)),
                                       __hmax2_nan(Elem<uint16_t>::word(v.z), Elem<uint16_t>::word(v.w)));
  const __nv_bfloat16 m = __hmax_nan(__low2bfloat16(t), __high2bfloat16(t));
  return __bfloat162float(m);
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float top_nan(const uint4& v, float) {
  return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)), max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
}

// Which elements of a vector do not lie below `least` (a NaN does not).
__device__ __forceinline__ uint32_t reaching(const uint4& v, float least, uint16_t) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t w = k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w;
    m |= (bf_lo(w) < least ? 0u : 1u << (2 * k)) | (bf_hi(w) < least ? 0u : 2u << (2 * k));
  }
  return m;
}
__device__ __forceinline__ uint32_t reaching(const uint4& v, float least, float) {
  return (__uint_as_float(v.x) < least ? 0u : 1u) | (__uint_as_float(v.y) < least ? 0u : 2u) |
         (__uint_as_float(v.z) < least ? 0u : 4u) | (__uint_as_float(v.w) < least ? 0u : 8u);
}

// A vector without the elements that `m` says.
__device__ __forceinline__ uint32_t word_without(uint32_t w, uint32_t m) {
  if (m & 1) w = (w & 0xffff0000u) | 0xff80u;
  if (m & 2) w = (w & 0xffffu) | 0xff800000u;
  return w;
}
__device__ __forceinline__ uint4 without(const uint4& v, uint32_t m, uint16_t) {
  return make_uint4(word_without(v.x, m), word_without(v.y, m >> 2), word_without(v.z, m >> 4), word_without(v.w, m >> 6));
}
__device__ __forceinline__ uint4 without(const uint4& v, uint32_t m, float) {
  return make_uint4(m & 1 ? 0xff800000u : v.x, m & 2 ? 0xff800000u : v.y, m & 4 ? 0xff800000u : v.z, m & 8 ? 0xff800000u : v.w);
}

// ------------------------------------------------------------------- host --

inline Terms terms_of(float temperature) { return Terms{(float)(1.4426950408889634 / (double)temperature), 1.f / temperature}; }

// A temperature whose factors are finite: a difference of 0 times them stays 0.
inline bool temperature_ok(float temperature) {
  return temperature >= 1.1754943508222875e-38f && temperature <= 3.402823466e38f;  // normal numbers
}

inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline bool f32_ok(const void* p) { return p != nullptr && aligned_to(p, 4); }

inline bool overlap(const void* a, long long abytes, const void* b, long long bbytes) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + (uintptr_t)bbytes && b0 < a0 + (uintptr_t)abytes;
}

inline lora_status_t check_logits(const void* logits, long long ld, int dtype, const int32_t* labels, int T, int V) {
  if (T < 0 || V < 1) return LORA_ERR_INVALID_ARG;
  if (dtype != LORA_LOGITS_BF16 && dtype != LORA_LOGITS_F32) return LORA_ERR_INVALID_ARG;
  if (T == 0) return LORA_OK;
  if (ld < V || ld > (1LL << 40) / T) return LORA_ERR_INVALID_ARG;
  const size_t b = dtype == LORA_LOGITS_BF16 ? 2 : 4;
  if (logits == nullptr || !aligned_to(logits, b) || !f32_ok(labels)) return LORA_ERR_INVALID_ARG;
  return LORA_OK;
}

// The gradient's place: the logits' own (same rows), or apart from them.
inline lora_status_t check_grad(const void* logits, long long ld, int dtype, const void* d, long long ldd, int T, int V) {
  if (d == nullptr || T == 0) return LORA_OK;
  const long long b = dtype == LORA_LOGITS_BF16 ? 2 : 4;
  if (ldd < V || ldd > (1LL << 40) / T || !aligned_to(d, b)) return LORA_ERR_INVALID_ARG;
  if (d == logits && ldd == ld) return LORA_OK;
  if (ldd == ld) {  // rows that take turns (halves of one buffer) do not overlap either
    const long long step = ld * b, off = (long long)(reinterpret_cast<uintptr_t>(d) - reinterpret_cast<uintptr_t>(logits)) % step;
    const long long at = off < 0 ? off + step : off;
    if (at >= V * b && at <= step - V * b) return LORA_OK;
  }
  const long long rows = T - 1;
  return overlap(logits, (rows * ld + V) * b, d, (rows * ldd + V) * b) ? LORA_ERR_INVALID_ARG : LORA_OK;
}

}  // namespace lora
