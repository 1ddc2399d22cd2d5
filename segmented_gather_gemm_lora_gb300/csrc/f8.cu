// The base in 8-bit floating point (lora_f8.h): quantising, and the entry points of
// the product and its input's gradient (f8_gemm.cu).
//
// Quantising: a group's largest magnitude a is an integer maximum of the values'
// bits without their signs (which orders a NaN above everything, so it is kept);
// its scale is s = fp32(a / M), or a power of two that a's bits give: M is 1.75 times
// a power of two for both types, so M 2^e >= a exactly if a's significand is at
// most 1.75 or e is one more.  A code is that of the correctly rounded quotient
// x / s: with r the reciprocal of s and q = x r, q + (x - q s) r rounds to it (Markstein; it
// could miss only within 2^-22 of a unit of the middle of two fp32), and x - q s is exact
// where it matters since a >= 2^-64.
#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "lora_f8.h"
#include "pairs.cuh"

namespace lora {

namespace {

// --------------------------------------------------------------- quantising --

constexpr uint32_t kTinyBits = 0x1f800000u;  // 2^-64
constexpr uint32_t kInfBits = 0x7f800000u;

// fp32(a / M) of a finite a >= 2^-64: with r the rounded 1 / M and q = a r, q + (a - q M) r
// rounds to it (all 2^23 significands agree with the division).
template <int kType>
__device__ __forceinline__ float over_largest(float a) {
  constexpr float kM = kType == LORA_F8_E4M3 ? 448.f : 57344.f, kR = 1.f / kM;
  const float q = a * kR;
  return fmaf(fmaf(-q, kM, a), kR, q);
}

// The scale of a group whose largest magnitude has these bits.
template <int kType>
__device__ __forceinline__ float scale_of(uint32_t top, bool pow2) {
  if (top < kTinyBits) return 0.f;
  if (top >= kInfBits) return __uint_as_float(top);
  if (!pow2) return over_largest<kType>(__uint_as_float(top));
  const uint32_t e = (top >> 23) - (kType == LORA_F8_E4M3 ? 8 : 15) + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float(e << 23);
}

// Of a scale: its negative and its reciprocal, twice each.  The reciprocal of the hardware
// (a unit off at most) after one Newton step is off by half a unit or a little more.  A
// scale of 0 has reciprocal 0, so that its quotients are 0.
struct Inverse {
  uint64_t ns, r;
};
__device__ __forceinline__ Inverse inverse_of(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  r = s == 0.f ? 0.f : fmaf(fmaf(-s, r, 1.f), r, r);
  return Inverse{pair_of(-s, -s), pair_of(r, r)};
}
__device__ __forceinline__ uint64_t quotients(uint64_t x, const Inverse& v) {
  const uint64_t q = mul2(x, v.r);
  return fma2(fma2(q, v.ns, x), v.r, q);
}

// Four codes, the first in the low byte.
template <int kType>
__device__ __forceinline__ uint32_t pack_f8(float a, float b, float c, float d) {
  uint32_t r;
  if constexpr (kType == LORA_F8_E4M3)
    asm("{\n\t.reg .b16 l, h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
  else
    asm("{\n\t.reg .b16 l, h;\n\t"
        "cvt.rn.satfinite.e5m2x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e5m2x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// A unit's place, and its step to the next without a division.
struct Place {
  long long r;
  int s;
  __device__ __forceinline__ void next(int step_r, int step_s, int spans) {
    r += step_r;
    s += step_s;
    if (s >= spans) {
      s -= spans;
      ++r;
    }
  }
};

struct QuantArgs {
  const void* x;
  long long ldx;
  lora_f8_matrix_t q;
  int groups;       // of a row
  long long units;  // rows of blocks x spans: what a warp (or, of blocks, a CTA) takes at once
  int spans;        // of a row of units
  int step_r, step_s;  // from a unit to its taker's next one
  int pow2;
  int wide;  // rows of x on 16-byte boundaries
  int32_t* err;
};

// One 16-byte vector of x: its values, and the largest magnitude's bits.  Entries from
// `left` on are not there.
template <typename E>
struct Vec;
template <>
struct Vec<uint16_t> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ uint4 load(const uint16_t* p, int left, bool wide) {
    if (wide && left >= kN) return *reinterpret_cast<const uint4*>(p);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (i < left) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ uint32_t top(const uint4& v) {
    // two magnitudes a word, as 16-bit integers
    const uint32_t m = 0x7fff7fffu;
    const uint32_t t = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
    return max(t & 0xffff0000u, t << 16);
  }
  // elements 2 i and 2 i + 1
  static __device__ __forceinline__ uint64_t pair(const uint4& v, int i) {
    const uint32_t u = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    return pair_of(bf_lo(u), bf_hi(u));
  }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ uint4 load(const float* p, int left, bool wide) {
    if (wide && left >= kN) return *reinterpret_cast<const uint4*>(p);
    return make_uint4(left > 0 ? __float_as_uint(p[0]) : 0, left > 1 ? __float_as_uint(p[1]) : 0,
                      left > 2 ? __float_as_uint(p[2]) : 0, left > 3 ? __float_as_uint(p[3]) : 0);
  }
  static __device__ __forceinline__ uint32_t top(const uint4& v) {
    const uint32_t m = 0x7fffffffu;
    return max(max(v.x & m, v.y & m), max(v.z & m, v.w & m));
  }
  static __device__ __forceinline__ uint64_t pair(const uint4& v, int i) {
    return i == 0 ? pair_of(__uint_as_float(v.x), __uint_as_float(v.y)) : pair_of(__uint_as_float(v.z), __uint_as_float(v.w));
  }
};

// The codes of a vector of a group with scale s (rows of codes start on 16-byte boundaries,
// groups on 128).
template <typename E, int kType>
__device__ __forceinline__ void put_codes(uint8_t* dst, const uint4& v, int left, float s, const Inverse& inv) {
  constexpr int kN = Vec<E>::kN;
  const bool finite = s < __uint_as_float(kInfBits);
  uint32_t w[kN / 4];
#pragma unroll
  for (int i = 0; i < kN / 4; ++i) {
    float e[4];
    split(quotients(Vec<E>::pair(v, 2 * i), inv), e[0], e[1]);
    split(quotients(Vec<E>::pair(v, 2 * i + 1), inv), e[2], e[3]);
    if (!finite) {  // by the division itself: 0, or NaN from what is not finite
      split(Vec<E>::pair(v, 2 * i), e[0], e[1]);
      split(Vec<E>::pair(v, 2 * i + 1), e[2], e[3]);
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] = fabsf(e[j]) < __uint_as_float(kInfBits) && s == s ? copysignf(0.f, e[j]) : s - s;
    }
    w[i] = pack_f8<kType>(e[0], e[1], e[2], e[3]);
  }
  if (left >= kN) {
    if constexpr (kN == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(dst) = w[0];
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (i < left) dst[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

// Rows: a warp takes kSteps vectors a lane of one row at a time (a group is 16 lanes for
// bf16, 32 for fp32), and has the next ones on their way meanwhile.
constexpr int kQThreads = 256, kSteps = 4, kRowCtas = 6;  // CTAs an SM in a grid
template <typename E, int kType>
__global__ void __launch_bounds__(kQThreads) quantize_rows_kernel(const __grid_constant__ QuantArgs a) {
  constexpr int kN = Vec<E>::kN, kLanes = LORA_F8_BLOCK / kN, kPer = 32 / kLanes;  // groups a step
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31, in = lane % kLanes;
  const long long stride = (long long)gridDim.x * (kQThreads / 32);
  long long unit = (long long)blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5);
  Place at{unit / a.spans, (int)(unit % a.spans)};
  auto load = [&](bool on, const Place& p, uint4 (&v)[kSteps]) {
    const int g0 = p.s * kSteps * kPer + lane / kLanes;
    const E* const row = static_cast<const E*>(a.x) + p.r * a.ldx;
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int c = (g0 + u * kPer) * LORA_F8_BLOCK + in * kN;
      v[u] = on && c < a.q.cols ? Vec<E>::load(row + c, a.q.cols - c, a.wide) : make_uint4(0, 0, 0, 0);
    }
  };
  uint4 v[kSteps], next[kSteps];
  load(unit < a.units, at, v);
  bool bad = false;
  for (; unit < a.units; unit += stride) {
    const long long r = at.r;
    const int g0 = at.s * kSteps * kPer + lane / kLanes;
    at.next(a.step_r, a.step_s, a.spans);
    load(unit + stride < a.units, at, next);
    uint8_t* const codes = static_cast<uint8_t*>(a.q.codes) + r * a.q.ld;
    uint32_t top[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) top[u] = Vec<E>::top(v[u]);
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1)
#pragma unroll
      for (int u = 0; u < kSteps; ++u) top[u] = max(top[u], __shfl_xor_sync(0xffffffffu, top[u], d));
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int g = g0 + u * kPer, c = g * LORA_F8_BLOCK + in * kN;
      const float s = scale_of<kType>(top[u], a.pow2);
      if (in == 0 && g < a.groups) a.q.scales[r * a.q.scale_row + g * a.q.scale_col] = s;
      if (c < a.q.cols) put_codes<E, kType>(codes + c, v[u], a.q.cols - c, s, inverse_of(s));
      bad |= top[u] >= kInfBits;
      v[u] = next[u];
    }
  }
  if (bad && in == 0) report(a.err, LORA_DERR_NONFINITE);
}

// Blocks: a CTA a block of 128 x 128, kept in registers between its maximum and its codes
// while the next one's values are on their way.
// Threads of its CTA: eight vectors each.
template <typename E>
constexpr int kBThreads = LORA_F8_BLOCK * LORA_F8_BLOCK / 8 / Vec<E>::kN;
template <typename E, int kType>
__global__ void __launch_bounds__(kBThreads<E>, 512 / kBThreads<E>) quantize_block_kernel(const __grid_constant__ QuantArgs a) {
  constexpr int kN = Vec<E>::kN, kLanes = LORA_F8_BLOCK / kN, kRows = kBThreads<E> / kLanes, kVec = LORA_F8_BLOCK / kRows;
  __shared__ uint32_t part[2][kBThreads<E> / 32];
  pdl_wait_then_release();
  const int in_row = threadIdx.x / kLanes, in_col = threadIdx.x % kLanes * kN;
  auto load = [&](bool on, const Place& p, uint4 (&v)[kVec]) {
    const long long r0 = p.r * LORA_F8_BLOCK + in_row;
    const int c = p.s * LORA_F8_BLOCK + in_col, left = a.q.cols - c;
    const E* const x = static_cast<const E*>(a.x) + c;
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      const long long r = r0 + u * kRows;
      v[u] = on && left > 0 && r < a.q.rows ? Vec<E>::load(x + r * a.ldx, left, a.wide) : make_uint4(0, 0, 0, 0);
    }
  };
  uint4 v[kVec], next[kVec];
  Place at{blockIdx.x / a.spans, (int)(blockIdx.x % a.spans)};
  load(true, at, v);
  int turn = 0;
  for (long long unit = blockIdx.x; unit < a.units; unit += gridDim.x, turn ^= 1) {
    const long long b = at.r;
    const int g = at.s;
    at.next(a.step_r, a.step_s, a.spans);
    load(unit + gridDim.x < a.units, at, next);
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < kVec; ++u) top = max(top, Vec<E>::top(v[u]));
    top = __reduce_max_sync(0xffffffffu, top);
    // (two sets of places: a warp can be one block ahead of the slowest, not two)
    if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kBThreads<E> / 32; ++i) top = max(top, part[turn][i]);
    const long long r0 = b * LORA_F8_BLOCK + in_row;
    const int c = g * LORA_F8_BLOCK + in_col, left = a.q.cols - c;
    const float s = scale_of<kType>(top, a.pow2);
    const Inverse inv = inverse_of(s);
    if (threadIdx.x == 0) {
      a.q.scales[b * a.q.scale_row + g * a.q.scale_col] = s;
      if (top >= kInfBits) report(a.err, LORA_DERR_NONFINITE);
    }
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      const long long r = r0 + u * kRows;
      if (left > 0 && r < a.q.rows) put_codes<E, kType>(static_cast<uint8_t*>(a.q.codes) + r * a.q.ld + c, v[u], left, s, inv);
      v[u] = next[u];
    }
  }
}

// -------------------------------------------------------------------- host --

template <typename E>
const void* rows_kernel(int type) {
  return type == LORA_F8_E4M3 ? (const void*)quantize_rows_kernel<E, LORA_F8_E4M3> : (const void*)quantize_rows_kernel<E, LORA_F8_E5M2>;
}
template <typename E>
const void* block_kernel(int type) {
  return type == LORA_F8_E4M3 ? (const void*)quantize_block_kernel<E, LORA_F8_E4M3> : (const void*)quantize_block_kernel<E, LORA_F8_E5M2>;
}

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool overlap(const void* a, long long abytes, const void* b, long long bbytes) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + (uintptr_t)bbytes && b0 < a0 + (uintptr_t)abytes;
}

long long blocks_of(long long n, int b) { return (n + b - 1) / b; }

// Bytes from the first code to past the last one; of the scales likewise.
long long code_bytes(const lora_f8_matrix_t& m) { return (m.rows - 1) * m.ld + m.cols; }
long long scale_bytes(const lora_f8_matrix_t& m) {
  return 4 * ((blocks_of(m.rows, m.block_rows) - 1) * m.scale_row + (blocks_of(m.cols, LORA_F8_BLOCK) - 1) * m.scale_col + 1);
}

// Rows and columns of tiles, the last one's ends too, stay within 32 bits.
constexpr int kMostRows = 0x7fff0000;

lora_status_t check_f8(const lora_f8_matrix_t* m) {
  if (m == nullptr || m->rows < 0 || m->cols < 1) return LORA_ERR_INVALID_ARG;
  if (m->type != LORA_F8_E4M3 && m->type != LORA_F8_E5M2) return LORA_ERR_INVALID_ARG;
  if (m->block_rows != 1 && m->block_rows != LORA_F8_BLOCK) return LORA_ERR_INVALID_ARG;
  if (m->ld < m->cols || m->ld % 16 != 0 || m->scale_row < 0 || m->scale_col < 0) return LORA_ERR_INVALID_ARG;
  if (m->rows == 0) return LORA_OK;
  if (m->rows > kMostRows || m->cols > kMostRows) return LORA_ERR_UNSUPPORTED;
  const long long most = 1LL << 40;
  if (m->ld > most / m->rows || m->scale_row > most / m->rows || m->scale_col > most / m->cols) return LORA_ERR_INVALID_ARG;
  if (m->codes == nullptr || !aligned_to(m->codes, 16)) return LORA_ERR_INVALID_ARG;
  if (m->scales == nullptr || !aligned_to(m->scales, 4)) return LORA_ERR_INVALID_ARG;
  return LORA_OK;
}

// A plain matrix [rows, cols] beside 8-bit ones.
lora_status_t check_plain(const void* p, long long ld, int dtype, int rows, int cols) {
  if (dtype != LORA_F8_FROM_BF16 && dtype != LORA_F8_FROM_F32) return LORA_ERR_INVALID_ARG;
  if (rows == 0) return LORA_OK;
  if (ld < cols || ld > (1LL << 40) / rows) return LORA_ERR_INVALID_ARG;
  return p == nullptr || !aligned_to(p, dtype == LORA_F8_FROM_BF16 ? 2 : 4) ? LORA_ERR_INVALID_ARG : LORA_OK;
}
long long plain_bytes(long long ld, int dtype, int rows, int cols) {
  return ((rows - 1) * ld + cols) * (dtype == LORA_F8_FROM_BF16 ? 2 : 4);
}

lora_status_t product(const lora_f8_matrix_t* x, const lora_f8_matrix_t* w, void* y, long long ldy, int dtype, int back,
                      int32_t* err, cudaStream_t s) {
  lora_status_t st = check_f8(x);
  if (st != LORA_OK || (st = check_f8(w)) != LORA_OK) return st;
  if (x->block_rows != 1 || w->block_rows != LORA_F8_BLOCK || w->rows < 1) return LORA_ERR_INVALID_ARG;
  const int inner = back ? w->rows : w->cols, outer = back ? w->cols : w->rows;
  if (x->cols != inner) return LORA_ERR_INVALID_ARG;
  if ((st = check_plain(y, ldy, dtype, x->rows, outer)) != LORA_OK || x->rows == 0) return st;
  const long long bytes = plain_bytes(ldy, dtype, x->rows, outer);
  for (const lora_f8_matrix_t* m : {x, w})
    if (overlap(y, bytes, m->codes, code_bytes(*m)) || overlap(y, bytes, m->scales, scale_bytes(*m))) return LORA_ERR_INVALID_ARG;
  return launch_f8_product(x, w, y, ldy, dtype == LORA_F8_FROM_F32, back, err, s);
}

}  // namespace

}  // namespace lora

using namespace lora;

extern "C" {

lora_status_t lora_f8_quantize(const void* x, int64_t ldx, int32_t dtype, const lora_f8_matrix_t* q, uint32_t flags,
                               int32_t* dev_err, lora_stream_t stream) {
  lora_status_t st = check_f8(q);
  if (st != LORA_OK) return st;
  if (flags & ~(uint32_t)LORA_F8_POW2) return LORA_ERR_INVALID_ARG;
  if ((st = check_plain(x, ldx, dtype, q->rows, q->cols)) != LORA_OK || q->rows == 0) return st;
  const long long rows = blocks_of(q->rows, q->block_rows), groups = blocks_of(q->cols, LORA_F8_BLOCK);
  // every group's scale has a place of its own
  if ((rows > 1 && q->scale_row < 1) || (groups > 1 && q->scale_col < 1)) return LORA_ERR_INVALID_ARG;
  if (rows > 1 && groups > 1 && q->scale_row <= (groups - 1) * q->scale_col && q->scale_col <= (rows - 1) * q->scale_row)
    return LORA_ERR_INVALID_ARG;
  const long long bytes = plain_bytes(ldx, dtype, q->rows, q->cols);
  if (overlap(x, bytes, q->codes, code_bytes(*q)) || overlap(x, bytes, q->scales, scale_bytes(*q)) ||
      overlap(q->codes, code_bytes(*q), q->scales, scale_bytes(*q)))
    return LORA_ERR_INVALID_ARG;
  QuantArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x;
  a.ldx = ldx;
  a.q = *q;
  a.groups = (int)groups;
  a.pow2 = (flags & LORA_F8_POW2) != 0;
  a.err = dev_err;
  const bool bf16 = dtype == LORA_F8_FROM_BF16;
  a.wide = aligned_to(x, 16) && ldx * (bf16 ? 2 : 4) % 16 == 0;
  const bool by_rows = q->block_rows == 1;
  a.spans = by_rows ? (int)blocks_of(groups, kSteps * (bf16 ? 2 : 1)) : a.groups;
  a.units = rows * a.spans;
  const int takers = by_rows ? kQThreads / 32 : 1;  // of a CTA
  const long long ctas = std::min(blocks_of(a.units, takers), (long long)sm_count() * (by_rows ? kRowCtas : bf16 ? 2 : 1));
  a.step_r = (int)(ctas * takers / a.spans);
  a.step_s = (int)(ctas * takers % a.spans);
  const void* f = by_rows ? (bf16 ? rows_kernel<uint16_t>(q->type) : rows_kernel<float>(q->type))
                          : (bf16 ? block_kernel<uint16_t>(q->type) : block_kernel<float>(q->type));
  const int threads = by_rows ? kQThreads : bf16 ? kBThreads<uint16_t> : kBThreads<float>;
  return launch_pdl(f, dim3((unsigned)ctas), dim3((unsigned)threads), 0, (cudaStream_t)stream, 0, &a) == cudaSuccess ? LORA_OK
                                                                                                                     : LORA_ERR_CUDA;
}

lora_status_t lora_base_f8(const lora_f8_matrix_t* x, const lora_f8_matrix_t* w, void* y, int64_t ldy, int32_t out_dtype,
                           int32_t* dev_err, lora_stream_t stream) {
  return product(x, w, y, ldy, out_dtype, 0, dev_err, (cudaStream_t)stream);
}

lora_status_t lora_base_f8_backward(const lora_f8_matrix_t* dy, const lora_f8_matrix_t* w, void* dx, int64_t lddx,
                                    int32_t out_dtype, int32_t* dev_err, lora_stream_t stream) {
  return product(dy, w, dx, lddx, out_dtype, 1, dev_err, (cudaStream_t)stream);
}

}  // extern "C"
