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
  int bf16, pow2;
  int32_t* err;
};

__device__ __forceinline__ float value_at(const QuantArgs& a, long long r, int c) {
  if (a.bf16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.x)[r * a.ldx + c] << 16);
  return static_cast<const float*>(a.x)[r * a.ldx + c];
}

// A CTA a group: rows of it (1 or 128) by 128 columns.
constexpr int kQThreads = 128;
__global__ void __launch_bounds__(kQThreads) quantize_kernel(const __grid_constant__ QuantArgs a) {
  __shared__ uint32_t part[kQThreads / 32];
  pdl_wait_then_release();
  const int groups = (a.q.cols + LORA_F8_BLOCK - 1) / LORA_F8_BLOCK;
  const long long b = blockIdx.x / groups;
  const int g = blockIdx.x % groups, c = g * LORA_F8_BLOCK + threadIdx.x;
  const long long r0 = b * a.q.block_rows, r1 = min((long long)a.q.rows, r0 + a.q.block_rows);
  uint32_t top = 0;
  if (c < a.q.cols)
    for (long long r = r0; r < r1; ++r) top = max(top, __float_as_uint(value_at(a, r, c)) & 0x7fffffffu);
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
  __syncthreads();
  top = max(max(part[0], part[1]), max(part[2], part[3]));
  const float s = scale_of(top, a.q.type, a.pow2);
  const Inverse v = inverse_of(s);
  if (threadIdx.x == 0) {
    a.q.scales[b * a.q.scale_row + g * a.q.scale_col] = s;
    if (top >= kInfBits) report(a.err, LORA_DERR_NONFINITE);
  }
  if (c < a.q.cols)
    for (long long r = r0; r < r1; ++r)
      static_cast<uint8_t*>(a.q.codes)[r * a.q.ld + c] = (uint8_t)pack_f8(quotient(value_at(a, r, c), v), 0.f, a.q.type);
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
  if (rows * groups > 0x7fffffffLL) return LORA_ERR_UNSUPPORTED;
  QuantArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x;
  a.ldx = ldx;
  a.q = *q;
  a.bf16 = dtype == LORA_F8_FROM_BF16;
  a.pow2 = (flags & LORA_F8_POW2) != 0;
  a.err = dev_err;
  return launch_pdl((const void*)quantize_kernel, dim3((unsigned)(rows * groups)), dim3(kQThreads), 0, (cudaStream_t)stream,
                    0, &a) == cudaSuccess
             ? LORA_OK
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
