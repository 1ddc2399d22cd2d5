// Optimizer step of adapter training (lora_train.h): AdamW over the elements of
// the listed adapters, in their pages, and the gradient norms it clips by.
//
// Work is cut into chunks of consecutive elements of one matrix (A or B) of one
// projection of one listed adapter; a CTA takes one chunk, span by span.  The grid is
// sized by max_rank (the host does not know the ranks); CTAs past the adapter's
// rank end at once.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "lora_train.h"
#include "pairs.cuh"

namespace lora {

namespace {

constexpr int kThreads = 128;
constexpr int kGroup = 8;                     // consecutive elements a thread takes: one page each (d % 8 == 0, pages >= 64)
constexpr int kSpan = kThreads * kGroup;      // elements the CTA takes at once
constexpr int kSumGroups = 4;                 // spans of the sum that are read together and share a slot of its workspace
constexpr int kSumMost = 4;                   // slots of a chunk of the sum at most
constexpr int kMaxProj = 16;                  // projections of one launch (kernel parameters below 4 KB)
constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100
constexpr int kBlockLanes = LORA_ADAMW_BLOCK / kGroup;  // lanes that share a block's scale

struct DevProj {
  DevView v;
  float* grad;
  float* master;
  void* m;
  void* r;  // second moments
  uint16_t* m_scale;
  uint16_t* r_scale;
  int chunk0;   // first chunk of the projection in the launch
  int chunks_a;  // chunks of A at max_rank
  int slot0;    // the same of the sum's slots
  int slots_a;
  int slots_b;
};

struct TrainArgs {
  DevProj p[kMaxProj];
  int n_proj;
  const int32_t* ids;
  const lora_adamw_hyper_t* hyper;
  const float* sumsq;
  float* partial;       // the sum's slots [n_ids][partial_stride]; the launch's begin at partial0
  int partial_stride;
  int partial0;
  int zero_grad;
  int spans;    // spans of a chunk
  int reverse;  // chunks in reverse order
  int32_t* err;
};
static_assert(sizeof(TrainArgs) <= 4096, "kernel parameters");

// A chunk's place: which adapter, projection and matrix, and its elements.
struct Place {
  int entry;  // of the list
  int ad;
  int g;
  bool is_b;
  long long e0, size;  // first element; elements of the matrix (0: of no good adapter)
  long long slot0;     // page-list slot of the matrix
  bool lead;           // the CTA that reports the adapter's errors
  int bad;
  int twice;           // this thread saw the id earlier in the list
};

// Resolve blockIdx into a Place.  The threads still have to agree on `twice` (an
// id listed before is passed over: its elements have one writer).
__device__ __forceinline__ Place find_place(const TrainArgs& a) {
  Place q;
  const int chunk = a.spans * kSpan;
  const int e = a.reverse ? gridDim.y - 1 - blockIdx.y : blockIdx.y, c = a.reverse ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
  q.entry = e;
  q.ad = a.ids[e];
  q.g = 0;
  while (q.g + 1 < a.n_proj && c >= a.p[q.g + 1].chunk0) ++q.g;
  const DevProj& p = a.p[q.g];
  const int cg = c - p.chunk0;
  q.lead = cg == 0;
  q.is_b = cg >= p.chunks_a;
  q.e0 = (long long)(q.is_b ? cg - p.chunks_a : cg) * chunk;
  const lora_adapter_desc_t d = adapter_desc(p.v, q.ad);
  q.twice = 0;
  for (int k = threadIdx.x; k < e; k += blockDim.x) q.twice |= a.ids[k] == q.ad;
  q.slot0 = q.is_b ? d.b_page0 : d.a_page0;
  q.bad = q.ad < 0 || q.ad >= p.v.n_adapters ? LORA_DERR_BAD_ADAPTER : d.rank < 1 || d.rank > p.v.max_rank ? LORA_DERR_BAD_RANK : 0;
  q.size = q.bad ? 0 : (long long)d.rank * (q.is_b ? p.v.d_out : p.v.d_in);
  return q;
}

// Whether the chunk holds elements of a good adapter, the same in every thread.
__device__ __forceinline__ bool agree(const TrainArgs& a, Place& q) {
  if (__syncthreads_or(q.twice)) q.bad = LORA_DERR_BAD_ADAPTER;
  if (q.bad && q.lead && threadIdx.x == 0) report(a.err, q.bad);
  return !q.bad && q.e0 < q.size;
}

// Pool position of element e of the place's matrix, or -1 off the pool.
__device__ __forceinline__ long long pool_pos(const DevView& v, const Place& q, long long e) {
  const long long slot = q.slot0 + (e >> v.page_shift);
  if (slot < 0 || slot >= v.n_page_list) return -1;
  const long long page = v.page_list[slot];
  if (page < 0 || page >= v.n_pages) return -1;
  return (page << v.page_shift) + (e & ((1LL << v.page_shift) - 1));
}

// Eight elements as four pairs.
struct Eight {
  uint64_t p[4];
};
__device__ __forceinline__ Eight from_f32(const float4& a, const float4& b) {
  return Eight{{pair_of(a.x, a.y), pair_of(a.z, a.w), pair_of(b.x, b.y), pair_of(b.z, b.w)}};
}
__device__ __forceinline__ Eight from_bf16(const uint4& v) {
  return Eight{{pair_of(bf_lo(v.x), bf_hi(v.x)), pair_of(bf_lo(v.y), bf_hi(v.y)), pair_of(bf_lo(v.z), bf_hi(v.z)),
                pair_of(bf_lo(v.w), bf_hi(v.w))}};
}
__device__ __forceinline__ void store8(float* p, const Eight& x) {
  float f[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) split(x.p[k], f[2 * k], f[2 * k + 1]);
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ uint4 to_bf16(const Eight& x) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float a, b;
    split(x.p[k], a, b);
    w[k] = pack_bf16x2(a, b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight e4m3 codes as fp32, and back (to nearest, ties to even, saturating).
__device__ __forceinline__ Eight from_e4m3(const uint2& c) {
  Eight x;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint16_t two = (uint16_t)((k < 2 ? c.x : c.y) >> (16 * (k & 1)));
    uint32_t h;
    float a, b;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    asm("{\n\t.reg .f16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}" : "=f"(a), "=f"(b) : "r"(h));
    x.p[k] = pair_of(a, b);
  }
  return x;
}
__device__ __forceinline__ uint2 to_e4m3(const Eight& x) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float a, b;
    uint16_t two;
    split(x.p[k], a, b);
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(b), "f"(a));
    w[k >> 1] |= (uint32_t)two << (16 * (k & 1));
  }
  return make_uint2(w[0], w[1]);
}

// a / b where ib is near 1 / b and b has few bits (a scale, or 448): the approximate
// quotient is a few units off, so its residual is exact, and one Newton step leaves a
// quotient that rounds to the code or scale of the true one.  (a ib alone falls on
// the other side of a boundary that a / b sits on or beside.)
__device__ __forceinline__ float quotient(float a, float b, float ib) {
  const float q = a * ib;
  return fmaf(fmaf(-q, b, a), ib, q);
}
__device__ __forceinline__ uint64_t quotient2(uint64_t a, uint64_t minus_b, uint64_t ib) {
  const uint64_t q = mul2(a, ib);
  return fma2(fma2(q, minus_b, a), ib, q);
}

// The scale of a block of 64 whose elements the eight lanes around this one hold.
__device__ __forceinline__ uint16_t block_scale(const Eight& x) {
  float top = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float a, b;
    split(x.p[k], a, b);
    top = fmaxf(top, fmaxf(fabsf(a), fabsf(b)));
  }
#pragma unroll
  for (int s = 1; s < kBlockLanes; s <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
  return __bfloat16_as_ushort(__float2bfloat16_rn(top < kTiny ? 0.f : quotient(top, 448.f, 1.f / 448.f)));
}

__device__ __forceinline__ float bf16_value(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// Two roots, within a hair of half a unit: from g near 1 / sqrt(x), x g and one step
// of Newton's iteration.  Arguments below 2^-126 count as zero; infinity and NaN are
// their own roots.
__device__ __forceinline__ float rsqrt_fast(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaxf(x, 1.17549435e-38f)));
  return y;
}
__device__ __forceinline__ uint64_t roots(uint64_t x) {
  asm("mul.rn.ftz.f32x2 %0, %0, %1;" : "+l"(x) : "l"(pair_of(1.f, 1.f)));
  float u, v, a, b;
  split(x, u, v);
  const uint64_t g = pair_of(rsqrt_fast(u), rsqrt_fast(v)), y = mul2(x, g);
  split(fma2(fma2(y, y, pair_of(-u, -v)), mul2(g, pair_of(-0.5f, -0.5f)), y), a, b);
  const float inf = __int_as_float(0x7f800000);
  return pair_of(u < inf ? a : u, v < inf ? b : v);
}
__device__ __forceinline__ float rcp_fast(float x) {  // one unit
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));  // of normal values: a root is 0 or above 2^-75
  return y;
}

// What the step takes from an adapter's settings, worked out by one thread.
struct StepShared {
  float gs, b1, n1, b2, n2, size, iroot, eps, decay;
  int skip;
};

// Asynchronous copies into a thread's own places in shared memory.
template <int kBytes>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(kBytes) : "memory");
}

// What a thread works on: eight elements of a span.
struct Work {
  Eight g, w, m, r;  // r: the second moments
};

// fp32 moments, read when they are worked on.
__device__ __forceinline__ Eight read_f32(const float* at) {
  return from_f32(reinterpret_cast<const float4*>(at)[0], reinterpret_cast<const float4*>(at)[1]);
}
__device__ __forceinline__ Work read_work(const DevProj& p, long long pos) {
  Work x;
  x.g = read_f32(p.grad + pos);
  x.m = read_f32(static_cast<const float*>(p.m) + pos);
  x.r = read_f32(static_cast<const float*>(p.r) + pos);
  x.w = p.master != nullptr ? read_f32(p.master + pos) : from_bf16(*reinterpret_cast<const uint4*>(p.v.pool + pos));
  return x;
}

// 8-bit moments: a CTA's threads read a span ahead into shared memory, each into
// its own places.
struct Stage {
  float4 g[2][kThreads], w[2][kThreads];  // w: bf16 in w[0], or fp32
  float4 codes[kThreads];                 // of m, then of the roots
};
__device__ __forceinline__ void read_ahead(Stage& st, const DevProj& p, long long pos) {
  const int t = threadIdx.x;
#pragma unroll
  for (int k = 0; k < 2; ++k) copy_async<16>(&st.g[k][t], p.grad + pos + 4 * k);
  copy_async<8>(&st.codes[t].x, static_cast<const uint8_t*>(p.m) + pos);
  copy_async<8>(&st.codes[t].z, static_cast<const uint8_t*>(p.r) + pos);
  if (p.master != nullptr) {
#pragma unroll
    for (int k = 0; k < 2; ++k) copy_async<16>(&st.w[k][t], p.master + pos + 4 * k);
  } else {
    copy_async<16>(&st.w[0][t], p.v.pool + pos);
  }
}
__device__ __forceinline__ Work take_work(const Stage& st, bool master, uint32_t scales) {
  const int t = threadIdx.x;
  Work x;
  x.g = from_f32(st.g[0][t], st.g[1][t]);
  x.w = master ? from_f32(st.w[0][t], st.w[1][t]) : from_bf16(*reinterpret_cast<const uint4*>(&st.w[0][t]));
  const uint4 c = *reinterpret_cast<const uint4*>(&st.codes[t]);
  x.m = from_e4m3(make_uint2(c.x, c.y));
  x.r = from_e4m3(make_uint2(c.z, c.w));
  const float sm = bf16_value((uint16_t)scales), sr = bf16_value((uint16_t)(scales >> 16));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x.m.p[k] = mul2(x.m.p[k], pair_of(sm, sm));
    x.r.p[k] = mul2(x.r.p[k], pair_of(sr, sr));
    x.r.p[k] = mul2(x.r.p[k], x.r.p[k]);
  }
  return x;
}
struct NoStage {};
template <bool kE4M3>
using StageOf = std::conditional_t<kE4M3, Stage, NoStage>;

// AdamW.  Bound by memory: per element 24 bytes (fp32 moments), 30 (and fp32
// weights), 12 (8-bit moments), 4 more to clear the gradient; one pass, each
// byte moved once.  A thread's eight elements lie on one page, a block's 64 in
// eight neighbouring lanes, so a block's scale takes three shuffles.  Products
// work on pairs.  With fp32 moments roots and quotients are IEEE's, which memory
// hides (188 M elements with their norms 1075 us, 1077 with the hardware's
// approximations; 9.4 M elements 57.3 and 56.3).  With 8-bit moments instructions
// set the time, and the quotient of an update is approximate (2^-22 of it, a small
// part of a weight).  There a thread
// also has its next eight on their way into its own places in shared memory (no
// thread waits for another, no register is held): few bytes an element leave
// latency to set the time (48 M elements with their norms: 190 us without, 169
// with, 201 with two spans ahead; 188 M elements with fp32 moments, whose loads
// are many, 1095 without and 1289 with).
// What an 8-bit state keeps is rounded as its definition says: scales, codes and
// roots carry the correction steps above (3 us of 166 for 48 M elements with their
// norms, where the IEEE forms of everything cost 13; 1.4 M elements in pages of 64 take
// 12 us with and without them, 13.3 with the IEEE forms).
template <bool kE4M3>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ TrainArgs a) {
  __shared__ StepShared sh;
  __shared__ __align__(16) StageOf<kE4M3> stages[2];
  pdl_wait_then_release();
  Place q = find_place(a);
  const DevProj& p = a.p[q.g];
  // the pool position of this thread's eight elements of span j: -2 for none, -1
  // off the pool
  auto place = [&](int j) -> long long {
    const long long e = q.e0 + (long long)(j * kThreads + threadIdx.x) * kGroup;
    return j < a.spans && e < q.size ? pool_pos(p.v, q, e) : -2;
  };
  if (threadIdx.x == 0 && q.size > 0) {
    const lora_adamw_hyper_t h = a.hyper[q.ad];
    float gs = h.grad_scale;
    sh.skip = h.step < 1;
    if (a.sumsq != nullptr) {
      const float ss = a.sumsq[q.ad];
      if (!(ss < __int_as_float(0x7f800000))) {
        if (q.lead && !sh.skip) report(a.err, LORA_DERR_NONFINITE);
        sh.skip = 1;
      } else if (h.max_norm > 0.f) {
        gs *= fminf(1.f, h.max_norm / (sqrtf(ss) * fabsf(gs) + 1e-6f));
      }
    }
    // 1 - beta^t = -expm1(t log1p(beta - 1)): beta - 1 is exact, nothing cancels
    const float c1 = -expm1f((float)h.step * log1pf(h.beta1 - 1.f));
    const float c2 = -expm1f((float)h.step * log1pf(h.beta2 - 1.f));
    sh.gs = gs;
    sh.b1 = h.beta1;
    sh.n1 = 1.f - h.beta1;
    sh.b2 = h.beta2;
    sh.n2 = 1.f - h.beta2;
    sh.size = h.lr / c1;
    sh.iroot = 1.f / sqrtf(c2);
    sh.eps = h.eps;
    sh.decay = 1.f - h.lr * h.weight_decay;
  }
  if (!agree(a, q) || sh.skip) return;
  const uint64_t gs = pair_of(sh.gs, sh.gs), b1 = pair_of(sh.b1, sh.b1), n1 = pair_of(sh.n1, sh.n1);
  const uint64_t b2 = pair_of(sh.b2, sh.b2), n2 = pair_of(sh.n2, sh.n2), down = pair_of(-sh.size, -sh.size);
  const uint64_t iroot = pair_of(sh.iroot, sh.iroot), eps = pair_of(sh.eps, sh.eps), decay = pair_of(sh.decay, sh.decay);
  uint16_t* const pool = const_cast<uint16_t*>(p.v.pool);
  long long pos = place(0), npos = -2;
  uint32_t scales = 0, nscales = 0;
  auto ahead = [&](int j, long long at) -> uint32_t {
    uint32_t two = 0;
    if constexpr (kE4M3) {
      if (at >= 0) {
        read_ahead(stages[j & 1], p, at);
        two = p.m_scale[at / LORA_ADAMW_BLOCK] | (uint32_t)p.r_scale[at / LORA_ADAMW_BLOCK] << 16;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    return two;
  };
  scales = ahead(0, pos);
  for (int j = 0; j < a.spans && q.e0 + (long long)j * kSpan < q.size; ++j) {
    npos = place(j + 1);
    nscales = ahead(j + 1, npos);
    if (pos == -1) report(a.err, LORA_DERR_BAD_PAGE);
    Eight m{}, r{};
    if constexpr (kE4M3) asm volatile("cp.async.wait_group 1;" ::: "memory");
    if (pos >= 0) {
      Work x;
      if constexpr (kE4M3) x = take_work(stages[j & 1], p.master != nullptr, scales);
      else x = read_work(p, pos);
      const Eight& g = x.g;
      Eight& w = x.w;
      m = x.m;
      r = x.r;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint64_t gk = mul2(g.p[k], gs);
        m.p[k] = fma2(b1, m.p[k], mul2(n1, gk));
        r.p[k] = fma2(b2, r.p[k], mul2(n2, mul2(gk, gk)));
      }
      if (!kE4M3) {
        store8(static_cast<float*>(p.m) + pos, m);
        store8(static_cast<float*>(p.r) + pos, r);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float u, v;
        if (kE4M3) {
          r.p[k] = roots(r.p[k]);
        } else {
          split(r.p[k], u, v);
          r.p[k] = pair_of(__fsqrt_rn(u), __fsqrt_rn(v));
        }
        split(fma2(r.p[k], iroot, eps), u, v);
        uint64_t up;
        if (kE4M3) {
          up = mul2(m.p[k], pair_of(rcp_fast(u), rcp_fast(v)));
        } else {
          float a, b;
          split(m.p[k], a, b);
          up = pair_of(__fdiv_rn(a, u), __fdiv_rn(b, v));
        }
        w.p[k] = fma2(w.p[k], decay, mul2(down, up));
      }
      if (p.master != nullptr) store8(p.master + pos, w);
      *reinterpret_cast<uint4*>(pool + pos) = to_bf16(w);
      if (a.zero_grad) store8(p.grad + pos, Eight{});
    }
    if (kE4M3) {  // lanes without elements hold zeros, which no scale sees
      const uint16_t bm = block_scale(m), br = block_scale(r);
      if (pos >= 0) {
        const float sm = bf16_value(bm), sr = bf16_value(br);
        const float im = sm > 0.f ? rcp_fast(sm) : 0.f, ir = sr > 0.f ? rcp_fast(sr) : 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float u, v;
          m.p[k] = quotient2(m.p[k], pair_of(-sm, -sm), pair_of(im, im));
          split(quotient2(r.p[k], pair_of(-sr, -sr), pair_of(ir, ir)), u, v);
          if (u > 0.f) u = fmaxf(u, 0.001953125f);  // 2^-9, the smallest code
          if (v > 0.f) v = fmaxf(v, 0.001953125f);
          r.p[k] = pair_of(u, v);
        }
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.m) + pos) = to_e4m3(m);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.r) + pos) = to_e4m3(r);
        if (threadIdx.x % kBlockLanes == 0) {
          p.m_scale[pos / LORA_ADAMW_BLOCK] = bm;
          p.r_scale[pos / LORA_ADAMW_BLOCK] = br;
        }
      }
    }
    pos = npos;
    scales = nscales;
  }
}

template <bool kE4M3>
__global__ void __launch_bounds__(kThreads) adamw_init_kernel(const __grid_constant__ TrainArgs a) {
  pdl_wait_then_release();
  Place q = find_place(a);
  if (!agree(a, q)) return;
  const DevProj& p = a.p[q.g];
  for (int j = 0; j < a.spans; ++j) {
    const long long e = q.e0 + (long long)(j * kThreads + threadIdx.x) * kGroup;
    if (e >= q.size) return;
    const long long pos = pool_pos(p.v, q, e);
    if (pos < 0) {
      report(a.err, LORA_DERR_BAD_PAGE);
      continue;
    }
    const Eight zero{};
    store8(p.grad + pos, zero);
    if (kE4M3) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.m) + pos) = make_uint2(0, 0);
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.r) + pos) = make_uint2(0, 0);
      if (threadIdx.x % kBlockLanes == 0) {
        p.m_scale[pos / LORA_ADAMW_BLOCK] = 0;
        p.r_scale[pos / LORA_ADAMW_BLOCK] = 0;
      }
    } else {
      store8(static_cast<float*>(p.m) + pos, zero);
      store8(static_cast<float*>(p.r) + pos, zero);
    }
    if (p.master != nullptr) {
      store8(p.master + pos, from_bf16(*reinterpret_cast<const uint4*>(p.v.pool + pos)));
    }
  }
}

// Sum of squares of one chunk of gradients (4 bytes an element, read once) into its
// slots of the workspace, one for each kSumGroups spans however long the chunk is: an
// adapter's sum has one order, whatever is listed beside it.
__global__ void __launch_bounds__(kThreads) sumsq_kernel(const __grid_constant__ TrainArgs a) {
  __shared__ float sh[kSumMost][kThreads];
  pdl_wait_then_release();
  Place q = find_place(a);
  const DevProj& p = a.p[q.g];
  const int groups = a.spans / kSumGroups, slot = (int)(q.e0 / (kSumGroups * kSpan));
  float* const out = a.partial + (long long)q.entry * a.partial_stride + a.partial0 + p.slot0 + (q.is_b ? p.slots_a : 0) + slot;
  const int slots = min(groups, (q.is_b ? p.slots_b : p.slots_a) - slot);
  if (!agree(a, q)) {
    if ((int)threadIdx.x < slots) out[threadIdx.x] = 0.f;
    return;
  }
  for (int k = 0; k < groups; ++k) {
    long long pos[kSumGroups];  // all first, then all loads: a thread has its 128 bytes in flight
#pragma unroll
    for (int j = 0; j < kSumGroups; ++j) {
      const long long e = q.e0 + (long long)((k * kSumGroups + j) * kThreads + threadIdx.x) * kGroup;
      pos[j] = e < q.size ? pool_pos(p.v, q, e) : -2;
    }
    Eight g[kSumGroups] = {};
#pragma unroll
    for (int j = 0; j < kSumGroups; ++j)
      if (pos[j] >= 0) g[j] = read_f32(p.grad + pos[j]);
    uint64_t two = pair_of(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kSumGroups; ++j) {
      if (pos[j] == -1) report(a.err, LORA_DERR_BAD_PAGE);
#pragma unroll
      for (int i = 0; i < 4; ++i) two = fma2(g[j].p[i], g[j].p[i], two);
    }
    float u, v;
    split(two, u, v);
    sh[k][threadIdx.x] = u + v;
  }
  __syncthreads();
  // a warp a slot
  const int k = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (k >= slots) return;
  float t = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) t += sh[k][32 * w + lane];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
  if (lane == 0) out[k] = t;
}
static_assert(kSumMost <= kThreads / 32, "a warp a slot");

struct FinishArgs {
  const int32_t* ids;
  int n_adapters;
  const float* partial;
  int stride;
  int accumulate;
  float* sumsq;
};

// One CTA an adapter: its slots, kept with what their rounding leaves out,
// in a fixed order.
__global__ void __launch_bounds__(kThreads) sumsq_finish_kernel(const __grid_constant__ FinishArgs a) {
  __shared__ Pair32 sh[kThreads / 32];
  pdl_wait_then_release();
  const int e = blockIdx.x;
  const int ad = a.ids[e];
  Pair32 s{0.f, 0.f};
  for (int k = threadIdx.x; k < a.stride; k += kThreads) s = add_pair(s, Pair32{a.partial[(long long)e * a.stride + k], 0.f});
  int twice = 0;
  for (int k = threadIdx.x; k < e; k += kThreads) twice |= a.ids[k] == ad;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    s = add_pair(s, Pair32{__shfl_xor_sync(0xffffffffu, s.hi, d), __shfl_xor_sync(0xffffffffu, s.lo, d)});
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
  if (__syncthreads_or(twice) || ad < 0 || ad >= a.n_adapters || threadIdx.x != 0) return;
  s = sh[0];
  for (int k = 1; k < kThreads / 32; ++k) s = add_pair(s, sh[k]);
  if (a.accumulate) s = add_pair(s, Pair32{a.sumsq[ad], 0.f});
  a.sumsq[ad] = s.hi;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Chunks of `chunk` elements of a projection's A and of its B at max_rank.
long long chunks_of(long long max_rank, long long d, int chunk) { return (max_rank * d + chunk - 1) / chunk; }

lora_status_t check_list(const lora_train_proj_t* projs, int n_proj, const int32_t* ids, int n_ids) {
  if (projs == nullptr || n_proj < 1 || n_ids < 0) return LORA_ERR_INVALID_ARG;
  if (n_ids > LORA_MAX_ADAPTERS) return LORA_ERR_UNSUPPORTED;
  if (n_ids > 0 && ids == nullptr) return LORA_ERR_INVALID_ARG;
  for (int g = 0; g < n_proj; ++g) {
    const lora_status_t st = validate_view(&projs[g].view);
    if (st != LORA_OK) return st;
    if (projs[g].view.n_adapters != projs[0].view.n_adapters) return LORA_ERR_INVALID_ARG;
    if (projs[g].grad == nullptr || !aligned16(projs[g].grad)) return LORA_ERR_INVALID_ARG;
  }
  return LORA_OK;
}

bool overlap(const void* a, long long abytes, const void* b, long long bbytes) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && a0 < b0 + (uintptr_t)bbytes && b0 < a0 + (uintptr_t)abytes;
}

lora_status_t check_state(const lora_train_proj_t* projs, int n_proj, int state) {
  if (state != LORA_STATE_F32 && state != LORA_STATE_E4M3) return LORA_ERR_INVALID_ARG;
  for (int g = 0; g < n_proj; ++g) {
    const lora_train_proj_t& p = projs[g];
    if (p.m == nullptr || p.v == nullptr || !aligned16(p.m) || !aligned16(p.v) || !aligned16(p.master))
      return LORA_ERR_INVALID_ARG;
    const bool scales = p.m_scale != nullptr && p.v_scale != nullptr;
    if (state == LORA_STATE_E4M3 ? !scales || ((reinterpret_cast<uintptr_t>(p.m_scale) | reinterpret_cast<uintptr_t>(p.v_scale)) & 1u)
                                 : p.m_scale != nullptr || p.v_scale != nullptr)
      return LORA_ERR_INVALID_ARG;
    const long long n = p.view.n_pages * p.view.page_elems, mb = state == LORA_STATE_E4M3 ? n : 4 * n;
    const long long sb = n / LORA_ADAMW_BLOCK * 2;
    const struct {
      const void* at;
      long long bytes;
    } w[7] = {{p.view.pool, 2 * n}, {p.grad, 4 * n}, {p.master, 4 * n}, {p.m, mb}, {p.v, mb}, {p.m_scale, sb}, {p.v_scale, sb}};
    for (int i = 0; i < 7; ++i)
      for (int k = 0; k < i; ++k)
        if (overlap(w[i].at, w[i].bytes, w[k].at, w[k].bytes)) return LORA_ERR_INVALID_ARG;
  }
  return LORA_OK;
}

// Fill the projections [g0, g0 + n) of a launch; the number of its chunks, and in
// *slots that of the sum's slots.
long long fill(TrainArgs* a, const lora_train_proj_t* projs, int g0, int n, int chunk, int* slots) {
  long long at = 0, slot = 0;
  a->n_proj = n;
  for (int k = 0; k < n; ++k) {
    const lora_train_proj_t& s = projs[g0 + k];
    DevProj& d = a->p[k];
    make_dev_view(&s.view, &d.v);
    d.grad = s.grad;
    d.master = s.master;
    d.m = s.m;
    d.r = s.v;
    d.m_scale = static_cast<uint16_t*>(s.m_scale);
    d.r_scale = static_cast<uint16_t*>(s.v_scale);
    d.chunk0 = (int)at;
    d.chunks_a = (int)chunks_of(s.view.max_rank, s.view.d_in, chunk);
    at += d.chunks_a + chunks_of(s.view.max_rank, s.view.d_out, chunk);
    d.slot0 = (int)slot;
    d.slots_a = (int)chunks_of(s.view.max_rank, s.view.d_in, kSumGroups * kSpan);
    d.slots_b = (int)chunks_of(s.view.max_rank, s.view.d_out, kSumGroups * kSpan);
    slot += d.slots_a + d.slots_b;
    if (at > 0x7fffffffLL || slot > 0x7fffffffLL) return -1;
  }
  *slots = (int)slot;
  return at;
}

lora_status_t launch_over(const void* func, TrainArgs* a, const lora_train_proj_t* projs, int n_proj, int n_ids, int spans,
                          cudaStream_t s) {
  a->spans = spans;
  for (int g0 = 0; g0 < n_proj; g0 += kMaxProj) {
    int slots = 0;
    const long long chunks = fill(a, projs, g0, std::min(kMaxProj, n_proj - g0), spans * kSpan, &slots);
    if (chunks < 0) return LORA_ERR_UNSUPPORTED;
    if (launch_pdl(func, dim3((unsigned)chunks, (unsigned)n_ids), dim3(kThreads), 0, s, 0, a) != cudaSuccess)
      return LORA_ERR_CUDA;
    a->partial0 += slots;
  }
  return LORA_OK;
}

// Spans of a chunk of the sum: sixteen once the launch still has several CTAs for
// every place on the GPU, else four.
int sum_spans(const lora_train_proj_t* projs, int n_proj, int n_ids) {
  long long chunks = 0;
  for (int g = 0; g < n_proj; ++g)
    chunks += chunks_of(projs[g].view.max_rank, (long long)projs[g].view.d_in + projs[g].view.d_out, kSumMost * kSumGroups * kSpan);
  return chunks * n_ids >= 32LL * sm_count() ? kSumMost * kSumGroups : kSumGroups;
}

// Spans of a chunk of the step: four, which spreads a CTA's start over 4096 elements, once
// the launch still has several CTAs for every place on the GPU.  (Device times of one
// span and of four, us: 8-bit moments, 3.3 M elements 11.5 / 13.4, 9.1 M 28.4 / 23.0,
// 31.5 M with seven projections 98 / 69; fp32 moments and weights, 2.5 M 12.5 / 17.7,
// 62 M 293 / 280.)
int step_spans(const lora_train_proj_t* projs, int n_proj, int n_ids) {
  long long chunks = 0;
  for (int g = 0; g < n_proj; ++g)
    chunks += chunks_of(projs[g].view.max_rank, (long long)projs[g].view.d_in + projs[g].view.d_out, 4 * kSpan);
  return chunks * n_ids >= 16LL * sm_count() ? 4 : 1;
}

// Slots of an adapter in the sum's workspace, a function of the projections alone (so
// that a workspace made for many adapters serves fewer); -1 above what a launch can
// count.
long long sum_slots(const lora_train_proj_t* projs, int n_proj) {
  long long at = 0;
  for (int g = 0; g < n_proj; ++g)
    at += chunks_of(projs[g].view.max_rank, projs[g].view.d_in, kSumGroups * kSpan) +
          chunks_of(projs[g].view.max_rank, projs[g].view.d_out, kSumGroups * kSpan);
  return at > 0x7fffffffLL ? -1 : at;
}

}  // namespace

}  // namespace lora

using namespace lora;

extern "C" {

lora_status_t lora_adamw_init(const lora_train_proj_t* projs, int32_t n_proj, int32_t state, const int32_t* ids,
                              int32_t n_ids, int32_t* dev_err, lora_stream_t stream) {
  lora_status_t st = check_list(projs, n_proj, ids, n_ids);
  if (st != LORA_OK || (st = check_state(projs, n_proj, state)) != LORA_OK || n_ids == 0) return st;
  TrainArgs a;
  memset(&a, 0, sizeof(a));
  a.ids = ids;
  a.err = dev_err;
  return launch_over(state == LORA_STATE_E4M3 ? (const void*)adamw_init_kernel<true> : (const void*)adamw_init_kernel<false>,
                     &a, projs, n_proj, n_ids, step_spans(projs, n_proj, n_ids), (cudaStream_t)stream);
}

size_t lora_grad_sumsq_workspace_bytes(const lora_train_proj_t* projs, int32_t n_proj, int32_t n_ids) {
  if (projs == nullptr || n_proj < 1 || n_ids < 0 || n_ids > LORA_MAX_ADAPTERS) return 0;
  for (int g = 0; g < n_proj; ++g)
    if (validate_view(&projs[g].view) != LORA_OK) return 0;
  const long long n = sum_slots(projs, n_proj);
  return n < 0 ? 0 : (size_t)(((long long)n_ids * n * 4 + 16) / 16 * 16);
}

lora_status_t lora_grad_sumsq(const lora_train_proj_t* projs, int32_t n_proj, const int32_t* ids, int32_t n_ids,
                              int32_t accumulate, float* sumsq, void* workspace, size_t workspace_bytes,
                              int32_t* dev_err, lora_stream_t stream) {
  lora_status_t st = check_list(projs, n_proj, ids, n_ids);
  if (st != LORA_OK) return st;
  if (sumsq == nullptr || (reinterpret_cast<uintptr_t>(sumsq) & 3u) != 0) return LORA_ERR_INVALID_ARG;
  if (n_ids == 0) return LORA_OK;
  if (workspace == nullptr || !aligned16(workspace)) return LORA_ERR_INVALID_ARG;
  const long long n = sum_slots(projs, n_proj);
  if (n < 0) return LORA_ERR_UNSUPPORTED;
  if (workspace_bytes < lora_grad_sumsq_workspace_bytes(projs, n_proj, n_ids)) return LORA_ERR_WORKSPACE;
  TrainArgs a;
  memset(&a, 0, sizeof(a));
  a.ids = ids;
  a.err = dev_err;
  a.partial = static_cast<float*>(workspace);
  a.partial_stride = (int)n;
  st = launch_over((const void*)sumsq_kernel, &a, projs, n_proj, n_ids, sum_spans(projs, n_proj, n_ids),
                   (cudaStream_t)stream);
  if (st != LORA_OK) return st;
  FinishArgs f;
  memset(&f, 0, sizeof(f));
  f.ids = ids;
  f.n_adapters = projs[0].view.n_adapters;
  f.partial = a.partial;
  f.stride = (int)n;
  f.accumulate = accumulate ? 1 : 0;
  f.sumsq = sumsq;
  return launch_pdl((const void*)sumsq_finish_kernel, dim3((unsigned)n_ids), dim3(kThreads), 0, (cudaStream_t)stream, 0,
                    &f) == cudaSuccess
             ? LORA_OK
             : LORA_ERR_CUDA;
}

lora_status_t lora_adamw_step(const lora_train_proj_t* projs, int32_t n_proj, int32_t state, const int32_t* ids,
                              int32_t n_ids, const lora_adamw_hyper_t* hyper, const float* sumsq, uint32_t flags,
                              int32_t* dev_err, lora_stream_t stream) {
  if (flags & ~(uint32_t)LORA_ADAMW_ZERO_GRAD) return LORA_ERR_INVALID_ARG;
  lora_status_t st = check_list(projs, n_proj, ids, n_ids);
  if (st != LORA_OK || (st = check_state(projs, n_proj, state)) != LORA_OK) return st;
  if (hyper == nullptr || (reinterpret_cast<uintptr_t>(hyper) & 3u) != 0 || (reinterpret_cast<uintptr_t>(sumsq) & 3u) != 0)
    return LORA_ERR_INVALID_ARG;
  if (n_ids == 0) return LORA_OK;
  TrainArgs a;
  memset(&a, 0, sizeof(a));
  a.ids = ids;
  a.hyper = hyper;
  a.sumsq = sumsq;
  a.zero_grad = (flags & LORA_ADAMW_ZERO_GRAD) ? 1 : 0;
  a.reverse = sumsq != nullptr;  // the gradients that the norms read last are still in L2
  a.err = dev_err;
  return launch_over(state == LORA_STATE_E4M3 ? (const void*)adamw_kernel<true> : (const void*)adamw_kernel<false>, &a,
                     projs, n_proj, n_ids, step_spans(projs, n_proj, n_ids), (cudaStream_t)stream);
}

}  // extern "C"
