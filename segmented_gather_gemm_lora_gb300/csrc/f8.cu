// The base in 8-bit floating point (lora_f8.h): quantising, and the entry points of
// the product and its input's gradient (f8_gemm.cu).
//
// Quantising: a group's largest magnitude a is an integer maximum of the values'
// bits without their signs (which orders a NaN above everything, so it is kept);
// its scale is s = fp32(a / M), or a power of two that a's bits give: M is 1.75 times
// a power of two for both types, so M 2^e >= a exactly if a's significand is at
// most 1.75 or e is one more.  A code is that of the correctly rounded quotient
// x / s: with r the rounded reciprocal of s and q = x r, q + (x - q s) r rounds to it
// (Markstein), and x - q s is exact where it matters since a >= 2^-64.
#include <cuda_fp8.h>

#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "lora_f8.h"

namespace lora {

namespace {

// --------------------------------------------------------------- quantising --

constexpr uint32_t kTinyBits = 0x1f800000u;  // 2^-64
constexpr uint32_t kInfBits = 0x7f800000u;

// The scale of a group whose largest magnitude has these bits.
__device__ __forceinline__ float scale_of(uint32_t top, int type, bool pow2) {
  if (top < kTinyBits) return 0.f;
  if (top >= kInfBits || !pow2) return __fdiv_rn(__uint_as_float(top), type == LORA_F8_E4M3 ? 448.f : 57344.f);
  const uint32_t e = (top >> 23) - (type == LORA_F8_E4M3 ? 8 : 15) + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float(e << 23);
}

struct Inverse {
  float s, r;
  bool odd;  // a zero or non-finite scale
};
__device__ __forceinline__ Inverse inverse_of(float s) {
  const bool odd = !(s > 0.f && s < __uint_as_float(kInfBits));
  return Inverse{s, odd ? 0.f : __frcp_rn(s), odd};
}
__device__ __forceinline__ float quotient(float x, const Inverse& v) {
  if (v.odd) return v.s == 0.f ? 0.f : __fdiv_rn(x, v.s);
  const float q = x * v.r;
  return fmaf(fmaf(-q, v.s, x), v.r, q);
}

// Two codes, `a` in the low byte.
__device__ __forceinline__ uint32_t pack_f8(float a, float b, int type) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, type == LORA_F8_E4M3 ? __NV_E4M3 : __NV_E5M2);
}

struct QuantArgs {
  const void* x;
  long long ldx;
  lora_f8_matrix_t q;
  int groups, spans;  // of a row: groups, spans of groups that a warp takes
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
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    const uint32_t u = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return i & 1 ? bf_hi(u) : bf_lo(u);
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
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
  }
};

// The codes of a vector (rows of codes start on 16-byte boundaries, groups on 128).
template <typename E>
__device__ __forceinline__ void put_codes(uint8_t* dst, const uint4& v, int left, const Inverse& s, int type) {
  constexpr int kN = Vec<E>::kN;
  uint32_t w[kN / 4];
#pragma unroll
  for (int i = 0; i < kN / 4; ++i)
    w[i] = pack_f8(quotient(Vec<E>::get(v, 4 * i), s), quotient(Vec<E>::get(v, 4 * i + 1), s), type) |
           pack_f8(quotient(Vec<E>::get(v, 4 * i + 2), s), quotient(Vec<E>::get(v, 4 * i + 3), s), type) << 16;
  if (left >= kN) {
    if constexpr (kN == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(dst) = w[0];
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (i < left) dst[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

// Rows: a warp takes kSteps vectors a lane of one row: a group is 16 lanes (bf16) or 32.
constexpr int kQThreads = 256, kSteps = 4;
template <typename E>
__global__ void __launch_bounds__(kQThreads) quantize_rows_kernel(const __grid_constant__ QuantArgs a) {
  constexpr int kN = Vec<E>::kN, kLanes = LORA_F8_BLOCK / kN, kPer = 32 / kLanes;  // groups a step
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31, in = lane % kLanes;
  const long long unit = (long long)blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5), r = unit / a.spans;
  if (r >= a.q.rows) return;
  const int g0 = (int)(unit - r * a.spans) * kSteps * kPer + lane / kLanes;
  const E* const row = static_cast<const E*>(a.x) + r * a.ldx;
  uint8_t* const codes = static_cast<uint8_t*>(a.q.codes) + r * a.q.ld;
  uint4 v[kSteps];
  uint32_t top[kSteps];
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int c = (g0 + u * kPer) * LORA_F8_BLOCK + in * kN;
    v[u] = c < a.q.cols ? Vec<E>::load(row + c, a.q.cols - c, a.wide) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int u = 0; u < kSteps; ++u) top[u] = Vec<E>::top(v[u]);
#pragma unroll
  for (int d = kLanes / 2; d > 0; d >>= 1)
#pragma unroll
    for (int u = 0; u < kSteps; ++u) top[u] = max(top[u], __shfl_xor_sync(0xffffffffu, top[u], d));
  bool bad = false;
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int g = g0 + u * kPer, c = g * LORA_F8_BLOCK + in * kN;
    const float s = scale_of(top[u], a.q.type, a.pow2);
    if (in == 0 && g < a.groups) a.q.scales[r * a.q.scale_row + g * a.q.scale_col] = s;
    if (c < a.q.cols) put_codes<E>(codes + c, v[u], a.q.cols - c, inverse_of(s), a.q.type);
    bad |= top[u] >= kInfBits;
  }
  if (bad && in == 0) report(a.err, LORA_DERR_NONFINITE);
}

// Blocks: a CTA a block of 128 x 128, kept in registers between its maximum and its codes.
template <typename E>
__global__ void __launch_bounds__(kQThreads) quantize_block_kernel(const __grid_constant__ QuantArgs a) {
  constexpr int kN = Vec<E>::kN, kLanes = LORA_F8_BLOCK / kN, kRows = kQThreads / kLanes, kVec = LORA_F8_BLOCK / kRows;
  __shared__ uint32_t part[kQThreads / 32];
  pdl_wait_then_release();
  const long long b = blockIdx.x / a.groups, r0 = b * LORA_F8_BLOCK + threadIdx.x / kLanes;
  const int g = blockIdx.x % a.groups, c = g * LORA_F8_BLOCK + threadIdx.x % kLanes * kN, left = a.q.cols - c;
  uint4 v[kVec];
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < kVec; ++u) {
    const long long r = r0 + u * kRows;
    v[u] = left > 0 && r < a.q.rows ? Vec<E>::load(static_cast<const E*>(a.x) + r * a.ldx + c, left, a.wide) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int u = 0; u < kVec; ++u) top = max(top, Vec<E>::top(v[u]));
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kQThreads / 32; ++i) top = max(top, part[i]);
  const float s = scale_of(top, a.q.type, a.pow2);
  const Inverse inv = inverse_of(s);
  if (threadIdx.x == 0) {
    a.q.scales[b * a.q.scale_row + g * a.q.scale_col] = s;
    if (top >= kInfBits) report(a.err, LORA_DERR_NONFINITE);
  }
#pragma unroll
  for (int u = 0; u < kVec; ++u) {
    const long long r = r0 + u * kRows;
    if (left > 0 && r < a.q.rows) put_codes<E>(static_cast<uint8_t*>(a.q.codes) + r * a.q.ld + c, v[u], left, inv, a.q.type);
  }
}

// -------------------------------------------------------------------- host --

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

lora_status_t check_f8(const lora_f8_matrix_t* m) {
  if (m == nullptr || m->rows < 0 || m->cols < 1) return LORA_ERR_INVALID_ARG;
  if (m->type != LORA_F8_E4M3 && m->type != LORA_F8_E5M2) return LORA_ERR_INVALID_ARG;
  if (m->block_rows != 1 && m->block_rows != LORA_F8_BLOCK) return LORA_ERR_INVALID_ARG;
  if (m->ld < m->cols || m->ld % 16 != 0 || m->scale_row < 0 || m->scale_col < 0) return LORA_ERR_INVALID_ARG;
  if (m->rows == 0) return LORA_OK;
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
  const void* f;
  long long ctas;
  if (q->block_rows == 1) {
    a.spans = (int)blocks_of(groups, kSteps * (bf16 ? 2 : 1));
    ctas = blocks_of(rows * a.spans, kQThreads / 32);
    f = bf16 ? (const void*)quantize_rows_kernel<uint16_t> : (const void*)quantize_rows_kernel<float>;
  } else {
    ctas = rows * groups;
    f = bf16 ? (const void*)quantize_block_kernel<uint16_t> : (const void*)quantize_block_kernel<float>;
  }
  if (ctas > 0x7fffffffLL) return LORA_ERR_UNSUPPORTED;
  return launch_pdl(f, dim3((unsigned)ctas), dim3(kQThreads), 0, (cudaStream_t)stream, 0, &a) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
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
