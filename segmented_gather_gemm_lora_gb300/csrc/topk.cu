// A teacher's top logits (lora_train.h): the k largest entries of each row, and the
// log of the sum of exponentials of the others.
//
// A row is read once, by one CTA or by the CTAs of a cluster, in chunks of four vectors
// a thread with the next chunk on its way.  Each warp keeps the 32 largest of its entries
// seen so far in order across its lanes.  With m = k / 8 rounded up, the least of the
// eight warps' m-th entries has k entries at or above it: what is below this threshold,
// which the warps exchange every few chunks, is not listed and goes into the sum at
// once.  The few others go to the warp's segment of a list in shared memory.  At the end
// the k-th largest of the CTA's 256 ranked entries is a threshold that passes few more
// than k; what it stops goes into the sum too, the rest is placed by counting.  A segment
// that would overflow (rising rows, ties by the thousand) is cut to the warp's k best,
// found bit by bit.  So the sum is of exactly the entries that are not listed, no
// difference of large sums; and every place and every sum's order is fixed.
//
// Keys are the values' bits made to order as integers; composite keys order as the
// listing does, no two alike.
//
// What bounds it: memory, one read of the logits.
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "lora_train.h"
#include "rows.cuh"

namespace lora {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kVec = 4;                           // vectors a thread takes at once
constexpr int kSeg = 320;                         // entries of a warp's segment: its k best and some more
constexpr int kSlots = kWarps * kSeg / kThreads;  // entries a thread looks after in a cut
static_assert(kSlots * kThreads >= kMaxCluster * LORA_TOPK_MAX, "the cluster's entries too");
constexpr int kKept = LORA_TOPK_MAX / kWarps;     // of a segment, after a cut
static_assert(kSeg >= LORA_TOPK_MAX, "a warp's k best");
constexpr int kResident = 3;                      // CTAs an SM
constexpr float kLowest = -3.402823466e38f;  // below it only -inf, which is not listed

struct TopkArgs {
  const void* logits;
  long long ld;
  const int32_t* labels;
  int T, V, k;
  float hi, lo;  // log2(e) / temperature in two parts
  float inv;     // 1 / temperature
  int32_t* ids;
  float* values;
  float* tail;
  int32_t* err;
  long long probe;
};

// Keys that order as the listing does: by value (a NaN first, -0 as +0).
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  if (key == 0xffffffffu) return __int_as_float(0x7fffffff);
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
// A threshold at or below the values of keys from `key` on.
__device__ __forceinline__ float threshold_of(uint32_t key) {
  if (key >= 0xff800000u) return INF_F;  // +inf's key, or a NaN's
  const float x = value_of(key);
  return x >= kLowest ? x : kLowest;
}

struct alignas(8) Entry {  // (read across the cluster in one piece)
  uint32_t key;
  int idx;
};
__device__ __forceinline__ unsigned long long composite(const Entry& e) {
  return (unsigned long long)e.key << 32 | (uint32_t)~e.idx;
}

__device__ __forceinline__ Entry entry_of(unsigned long long c) { return Entry{(uint32_t)(c >> 32), (int)~(uint32_t)c}; }

struct TopShared {
  uint64_t probe_bar;
  Entry list[kWarps * kSeg];
  int count[kWarps];  // entries of each segment
  uint32_t hist[2][256];
  int scan[kWarps];
  Sum part[kWarps];
  alignas(8) Sum sum;              // the CTA's
  uint32_t least[2][kWarps];       // the warps' m-th keys
  alignas(16) uint32_t ranked[kThreads];  // the warps' 32 largest
  uint32_t bound[kMaxCluster];     // the cluster's CTAs' thresholds
  int total;                       // entries in best
  alignas(16) unsigned long long best[kMaxCluster * LORA_TOPK_MAX + 2];  // composite keys, then two zeros
};

static_assert(offsetof(TopShared, best) % 16 == 0 && offsetof(TopShared, list) % 8 == 0 && offsetof(TopShared, sum) % 8 == 0,
              "eight bytes at a time");

// Terms exp((x - base) / temperature).
struct Terms {
  float hi, lo, inv;
  __device__ __forceinline__ Sum join(const Sum& x, const Sum& y) const {
    Sum r;
    r.m = fmaxf(x.m, y.m);
    const float base = base_of(r.m);
    r.s = x.s * expf((x.m - base) * inv) + y.s * expf((y.m - base) * inv);
    return r;
  }
  __device__ __forceinline__ Sum add(const Sum& t, float x) const {
    return join(t, Sum{x, x == x ? (x == -INF_F ? 0.f : x == INF_F ? x : 1.f) : x});
  }
  __device__ __forceinline__ Sum across(const Sum& t) const {  // the warp's lanes
    const float m = warp_max(t.m);
    return Sum{m, warp_add(t.s * expf((t.m - base_of(m)) * inv))};
  }
};

// Some vectors, whose largest element is top, joined to t.
template <typename E, int N>
__device__ __forceinline__ Sum add_vectors(const Terms& e, Sum t, const uint4 (&r)[N], float top) {
  constexpr int kPairs = Elem<E>::kPairs;
  const float m = fmaxf(t.m, top), base = base_of(m);
  const uint64_t hi = pair_of(e.hi, e.hi), lo = pair_of(e.lo, e.lo), nb = pair_of(-base, -base);
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
  if (m != t.m) t.s *= expf((t.m - base) * e.inv);
  return Sum{m, t.s + (a + b)};
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

// Which elements of a vector do not lie below `least`, and a vector without some.
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
__device__ __forceinline__ uint32_t without(uint32_t w, uint32_t which) {  // of a word's two
  if (which & 1) w = (w & 0xffff0000u) | 0xff80u;
  if (which & 2) w = (w & 0xffffu) | 0xff800000u;
  return w;
}
__device__ __forceinline__ uint4 without(const uint4& v, uint32_t m, uint16_t) {
  return make_uint4(without(v.x, m), without(v.y, m >> 2), without(v.z, m >> 4), without(v.w, m >> 6));
}
__device__ __forceinline__ uint4 without(const uint4& v, uint32_t m, float) {
  return make_uint4(m & 1 ? 0xff800000u : v.x, m & 2 ? 0xff800000u : v.y, m & 4 ? 0xff800000u : v.z, m & 8 ? 0xff800000u : v.w);
}

// The warp's keys in falling order (a bitonic network).
__device__ __forceinline__ uint32_t sort_lanes(uint32_t key, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int d = size >> 1; d > 0; d >>= 1) {
      const uint32_t o = __shfl_xor_sync(0xffffffffu, key, d);
      const bool up = (lane & size) != 0 && size < 32, low = (lane & d) == 0;
      key = low != up ? max(key, o) : min(key, o);
    }
  return key;
}

// The 32 largest of two lists of 32, both in falling order across the lanes.
__device__ __forceinline__ uint32_t merge_lanes(uint32_t a, uint32_t b, int lane) {
  uint32_t key = max(a, __shfl_sync(0xffffffffu, b, 31 - lane));  // rises and falls, or the other way round
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const uint32_t o = __shfl_xor_sync(0xffffffffu, key, d);
    key = (lane & d) == 0 ? max(key, o) : min(key, o);
  }
  return key;
}

// The least composite key (as many leading bits of it as needed, zeros after them) that
// exactly `want` of the CTA's keys reach; a thread's are c[i] where on(i).  At least
// `want` keys are on, and no two are alike, or alike in the bits from kLast on only by
// what the caller can bear.
template <int kN, int kFirst, int kLast, typename On>
__device__ __forceinline__ unsigned long long select_top(const unsigned long long (&c)[kN], On on, int want, TopShared* sh) {
  const int tid = threadIdx.x, lane = tid & 31;
  unsigned long long prefix = 0, mask = 0;
  int turn = 0;
  __syncthreads();
  sh->hist[0][tid] = 0;
  __syncthreads();
  for (int shift = kFirst; shift >= kLast; shift -= 8, turn ^= 1) {
    uint32_t* const h = sh->hist[turn];
    sh->hist[turn ^ 1][tid] = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (on(i) && (c[i] & mask) == prefix) atomicAdd(&h[(c[i] >> shift) & 255], 1u);
    __syncthreads();
    // every warp finds the bin of the want-th largest: lane l has bins 8 l .. 8 l + 7
    uint32_t bins[8], mine = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) mine += bins[i] = h[lane * 8 + i];
    uint32_t above = mine;  // of this lane's bins and the ones after them
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_down_sync(0xffffffffu, above, d);
      if (lane + d < 32) above += o;
    }
    above -= mine;
    const bool here = above < (uint32_t)want && (uint32_t)want <= above + mine;
    int bin = 0, inside = 0, left = 0;
    if (here) {
      uint32_t greater = above;
#pragma unroll
      for (int i = 7; i >= 0; --i) {
        if (greater < (uint32_t)want && (uint32_t)want <= greater + bins[i]) {
          bin = lane * 8 + i;
          inside = (int)bins[i];
          left = want - (int)greater;
        }
        greater += bins[i];
      }
    }
    const int from = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    bin = __shfl_sync(0xffffffffu, bin, from);
    inside = __shfl_sync(0xffffffffu, inside, from);
    want = __shfl_sync(0xffffffffu, left, from);
    prefix |= (unsigned long long)bin << shift;
    mask |= 255ull << shift;
    if (inside == want) break;
    __syncthreads();
  }
  return prefix;
}

// Bits of a composite key that tell entries apart: a bf16 value's lower half follows from
// its sign, so its digits there would be one bin.
template <typename E>
__device__ __forceinline__ unsigned long long digits(const Entry& e) {
  if (sizeof(E) == 2) return (unsigned long long)(e.key >> 16) << 32 | (uint32_t)~e.idx;
  return composite(e);
}
template <typename E>
constexpr int kFirstDigit = sizeof(E) == 2 ? 40 : 56;
template <typename E>
__device__ __forceinline__ uint32_t key_of_digits(unsigned long long d) {
  // (a negative bf16's key ends in ones: the zeros are below it)
  return sizeof(E) == 2 ? (uint32_t)(d >> 32) << 16 : (uint32_t)(d >> 32);
}

// Cut entries (a thread's e[i] where `on` has bit i; `total` in all) to the k best; what
// goes is added to *t, what stays is put(place, entry) in the order of (thread, i), with a
// barrier between the last read and the first put.  Returns the new threshold (or the old
// one, of no more than k).
template <typename E, typename Put>
__device__ __forceinline__ float cut(TopShared* sh, const Entry (&e)[kSlots], uint32_t on, int total, int k, float threshold,
                                     const Terms& terms, Sum* t, Put put) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (total > k) {
    unsigned long long c[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) c[i] = digits<E>(e[i]);
    const unsigned long long least = select_top<kSlots, kFirstDigit<E>, 0>(c, [&](int i) { return on >> i & 1; }, k, sh);
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
      if ((on >> i & 1) && c[i] < least) {
        on &= ~(1u << i);
        if (terms.inv > 0.f) *t = terms.add(*t, value_of(e[i].key));
      }
    threshold = fmaxf(threshold, threshold_of(key_of_digits<E>(least)));
  }
  const int mine = __popc(on);
  int before = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += o;
  }
  if (lane == 31) sh->scan[warp] = before;
  before -= mine;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before += sh->scan[w];
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (on >> i & 1) put(before++, e[i]);
  return threshold;
}

// The list cut to its k best: segment w then has entries 32 w .. of them.
template <typename E>
__device__ __noinline__ float cut_list(TopShared* sh, int k, float threshold, const Terms& terms, Sum* t) {
  const int tid = threadIdx.x;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += sh->count[w];
  Entry e[kSlots];
  uint32_t on = 0;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int slot = i * kThreads + tid, seg = slot / kSeg;
    e[i] = sh->list[slot];
    if (slot - seg * kSeg < sh->count[seg]) on |= 1u << i;
  }
  threshold = cut<E>(sh, e, on, total, k, threshold, terms, t,
                     [&](int at, const Entry& x) { sh->list[at / kKept * kSeg + at % kKept] = x; });
  if (tid < kWarps) sh->count[tid] = min(max(min(total, k) - tid * kKept, 0), kKept);
  __syncthreads();
  return threshold;
}

// The entries of best, N of them, cut to the k best.
template <typename E>
__device__ __noinline__ void cut_best(TopShared* sh, int N, int k, const Terms& terms, Sum* t) {
  Entry e[kSlots];
  uint32_t on = 0;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int at = i * kThreads + threadIdx.x;
    e[i] = at < N ? entry_of(sh->best[at]) : Entry{0, 0};
    if (at < N) on |= 1u << i;
  }
  cut<E>(sh, e, on, N, k, kLowest, terms, t, [&](int at, const Entry& x) { sh->best[at] = composite(x); });
  __syncthreads();
}

template <typename E>
__global__ void __launch_bounds__(kThreads, kResident) topk_kernel(const __grid_constant__ TopkArgs a) {
  constexpr int kN = Elem<E>::kN;
  __shared__ TopShared sh;
  const int n = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait_then_release();
  if (a.probe > 0) {
    if (tid == 0 && !wait_probe(&sh.probe_bar, a.probe)) report(a.err, LORA_DERR_TIMEOUT);
    return;
  }
  const int k = a.k, m = (k + kWarps - 1) / kWarps;
  const Terms terms{a.hi, a.lo, a.tail != nullptr ? a.inv : 0.f};
  auto cut_at = [&](int row) { return cut_row(static_cast<const E*>(a.logits) + (long long)row * a.ld, a.V, rank, n); };
  auto load = [&](const Cut<E>& c, int i, uint4 (&r)[kVec]) {
    const uint4* const mid = reinterpret_cast<const uint4*>(c.row + c.head);
#pragma unroll
    for (int u = 0; u < kVec; ++u) r[u] = i + u * kThreads < c.v1 ? mid[i + u * kThreads] : low_vector<E>();
  };
  uint4 r[kVec], next[kVec];
  int row = (int)cluster_id_x();
  {
    const Cut<E> c = cut_at(row);
    load(c, c.v0 + tid, r);
  }
  // (with clusters a row each, else rows in turn, each one's first chunk loaded before the
  // row before it is finished)
  for (;;) {
  const int next_row = n == 1 ? row + (int)gridDim.x : a.T;
  const long long out = (long long)row * k;
  const Cut<E> c = cut_at(row);
  auto load_next = [&] {
    if (next_row < a.T) {
      const Cut<E> d = cut_at(next_row);
      load(d, d.v0 + tid, r);
    }
  };
  if (a.labels != nullptr && a.labels[row] < 0) {  // the whole cluster agrees
    if (rank == 0) {
      if (tid < k) {
        a.ids[out + tid] = -1;
        a.values[out + tid] = -INF_F;
      }
      if (tid == 0 && a.tail != nullptr) a.tail[row] = -INF_F;
    }
    load_next();
    if (next_row >= a.T) return;
    row = next_row;
    continue;
  }
  Sum t{-INF_F, 0.f};
  float threshold = kLowest;
  int count = 0;  // of this warp's segment

  uint32_t ranked = 0;  // lane l: the warp's entry l from the top
  int turn = 0;
  // Entries of some vectors to the list or into the sum: element j of vector u is entry
  // first + u * kThreads * kN + j.  (The first chunk's are ranked before.)
  auto take = [&](uint4 (&r)[kVec], int first, bool rank_them) {
    auto place = [&](int b) { return first + b / kN * (kThreads * kN) + b % kN; };
    // to the list what `which` (bit u * kN + j) says, which fits, a lane's entries in rising
    // order; they are read again by their place (registers have no index)
    auto append = [&](uint32_t which) {
#pragma unroll
      for (int u = 0; u < kVec; ++u)
        if (which >> (u * kN) & ((1u << kN) - 1)) r[u] = without(r[u], which >> (u * kN) & ((1u << kN) - 1), E{});
      uint32_t some;
      while ((some = __ballot_sync(0xffffffffu, which != 0)) != 0) {
        uint32_t key = 0;
        if (which != 0) {
          const int idx = place(__ffs(which) - 1);
          which &= which - 1;
          key = key_of(Elem<E>::get(c.row[idx]));
          sh.list[warp * kSeg + count + __popc(some & ((1u << lane) - 1))] = Entry{key, idx};
        }
        count += __popc(some);
        if (!rank_them) continue;
        some &= __ballot_sync(0xffffffffu, key > __shfl_sync(0xffffffffu, ranked, 31));
        if (__popc(some) > 5) {
          ranked = merge_lanes(ranked, sort_lanes(key, lane), lane);
        } else {
          for (; some != 0; some &= some - 1) {
            const uint32_t x = __shfl_sync(0xffffffffu, key, __ffs(some) - 1);
            const int at = __popc(__ballot_sync(0xffffffffu, ranked >= x));
            const uint32_t up = __shfl_up_sync(0xffffffffu, ranked, 1);
            ranked = lane > at ? up : lane == at ? x : ranked;
          }
        }
      }
    };
    float top = top_nan(r[0], E{});
#pragma unroll
    for (int u = 1; u < kVec; ++u) top = max_nan(top, top_nan(r[u], E{}));
    if (__any_sync(0xffffffffu, !(top < threshold))) {
      uint32_t which = 0;
#pragma unroll
      for (int u = 0; u < kVec; ++u) which |= reaching(r[u], threshold, E{}) << (u * kN);
      if (count + __reduce_add_sync(0xffffffffu, __popc(which)) > kSeg) {
        // the warp's k best, of its segment and of these, bit by bit
        unsigned long long least = 0;
        auto some_reach = [&](unsigned long long higher) {
          int some = 0;
          for (uint32_t w = which; w != 0; w &= w - 1) {
            const int idx = place(__ffs(w) - 1);
            some += digits<E>(Entry{key_of(Elem<E>::get(c.row[idx])), idx}) >= higher;
          }
          for (int i = lane; i < count; i += 32) some += digits<E>(sh.list[warp * kSeg + i]) >= higher;
          return __reduce_add_sync(0xffffffffu, some);
        };
        __syncwarp();
        for (int bit = kFirstDigit<E> + 7; bit >= 0; --bit) {
          const unsigned long long higher = least | 1ull << bit;
          const int some = some_reach(higher);
          if (some >= k) least = higher;
          if (some == k) break;
        }
        int kept = 0;
        for (int i = lane; i - lane < count; i += 32) {
          const Entry e = i < count ? sh.list[warp * kSeg + i] : Entry{0, 0};
          const bool in = i < count && digits<E>(e) >= least;
          const uint32_t some = __ballot_sync(0xffffffffu, in);
          if (in) sh.list[warp * kSeg + kept + __popc(some & ((1u << lane) - 1))] = e;
          else if (i < count && terms.inv > 0.f) t = terms.add(t, value_of(e.key));
          kept += __popc(some);
        }
        count = kept;
        uint32_t best = 0;
        for (uint32_t w = which; w != 0; w &= w - 1) {
          const int idx = place(__ffs(w) - 1);
          if (digits<E>(Entry{key_of(Elem<E>::get(c.row[idx])), idx}) >= least) best |= w & -w;
        }
        which = best;
        threshold = fmaxf(threshold, threshold_of(key_of_digits<E>(least)));
      }
      append(which);
      top = -INF_F;
#pragma unroll
      for (int u = 0; u < kVec; ++u) top = fmaxf(top, top_nan(r[u], E{}));
    }
    if (terms.inv > 0.f) t = add_vectors<E>(terms, t, r, top);
  };
  // The least of the warps' m-th entries so far: a threshold for all of them.
  auto exchange = [&] {
    if (lane == m - 1) sh.least[turn][warp] = ranked;
    __syncthreads();
    uint32_t least = sh.least[turn][0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) least = min(least, sh.least[turn][w]);
    threshold = fmaxf(threshold, threshold_of(least));
    turn ^= 1;
  };

  for (int i0 = c.v0, turns = 0; i0 < c.v1; i0 += kVec * kThreads, ++turns) {
    const int i = i0 + tid;
    load(c, i + kVec * kThreads, next);
    if (turns == 0) {
      // the largest of the chunk's vectors' maxima are ranked, for a threshold to begin with
      uint32_t top[kVec];
#pragma unroll
      for (int u = 0; u < kVec; ++u) top[u] = sort_lanes(key_of(top_nan(r[u], E{})), lane);
      ranked = merge_lanes(merge_lanes(top[0], top[1], lane), merge_lanes(top[2], top[3], lane), lane);
      exchange();
    }
    take(r, c.head + i * kN, turns > 0);
    if (turns == 1 || (turns & 3) == 3) exchange();
#pragma unroll
    for (int u = 0; u < kVec; ++u) r[u] = next[u];
  }
  if ((c.first && c.head > 0) || (c.last && c.tail0 < a.V)) {
    const int e = edge_of(c, a.V, tid);
#pragma unroll
    for (int u = 0; u < kVec; ++u) r[u] = low_vector<E>();
    if (e >= 0) {
      const float x = Elem<E>::get(c.row[e]);
      if (sizeof(E) == 2) r[0].x = 0xff800000u | __float_as_uint(x) >> 16;
      else r[0].x = __float_as_uint(x);
    }
    take(r, e, true);
  }
  load_next();

  // The threshold at the end: the largest of the warps' first 2 m + 2 ranked entries that has
  // enough of them at or above it, k, or of each of a cluster's CTAs an equal share.
  const int tops = min(2 * m + 2, 32);
  if (lane < tops) sh.ranked[warp * tops + lane] = ranked;
  if (tid < n) sh.bound[tid] = 0;
  __syncthreads();
  if (tid < kWarps * tops) {
    const uint32_t ranked = sh.ranked[tid];
    int above = 0, same = 0;
#pragma unroll 4
    for (int j = 0; j < kWarps * tops; j += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(&sh.ranked[j]);
      above += (x.x > ranked) + (x.y > ranked) + (x.z > ranked) + (x.w > ranked);
      same += (x.x == ranked) + (x.y == ranked) + (x.z == ranked) + (x.w == ranked);
    }
    const int share = (k + n - 1) / n;
    if (above < share && share <= above + same) sh.least[0][0] = ranked;  // alike where several write
  }
  __syncthreads();
  uint32_t bound = sh.least[0][0];
  if (n > 1) {
    cluster_sync();  // every CTA's places are there
    if (tid < n) st_dsmem_u32(mapa(smem_u32(&sh.bound[rank]), tid), bound);
    cluster_sync();
    for (int i = 0; i < n; ++i) bound = min(bound, sh.bound[i]);
  }
  threshold = fmaxf(threshold, threshold_of(bound));
  // (a warp's own may be higher: its k best are above it)
  auto stays = [&](const Entry& e) { return !(value_of(e.key) < threshold); };
  int left = 0;
  for (int i = lane; i < count; i += 32) left += stays(sh.list[warp * kSeg + i]);
  left = __reduce_add_sync(0xffffffffu, left);
  if (lane == 0) sh.scan[warp] = left;
  __syncthreads();
  int total = 0, at = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    at += w < warp ? sh.scan[w] : 0;
    total += sh.scan[w];
  }
  if (total > LORA_TOPK_MAX * (n > 1 ? 1 : kMaxCluster)) {  // more than there is room for
    if (lane == 0) sh.count[warp] = count;
    cut_list<E>(&sh, k, threshold, terms, &t);
    total = 0, at = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      at += w < warp ? sh.count[w] : 0;
      total += sh.count[w];
    }
    count = sh.count[warp];
    for (int i = lane; i < count; i += 32) sh.best[at + i] = composite(sh.list[warp * kSeg + i]);
  } else {
    for (int i = lane; i - lane < count; i += 32) {
      const Entry e = i < count ? sh.list[warp * kSeg + i] : Entry{0, 0};
      const bool in = i < count && stays(e);
      const uint32_t some = __ballot_sync(0xffffffffu, in);
      if (in) sh.best[at + __popc(some & ((1u << lane) - 1))] = composite(e);
      else if (i < count && terms.inv > 0.f) t = terms.add(t, value_of(e.key));
      at += __popc(some);
    }
  }
  // A CTA's entries are in best.  The first CTA takes the others'.
  auto cta_sum = [&] {
    const Sum w = terms.across(t);
    if (lane == 0) sh.part[warp] = w;
    __syncthreads();
    return terms.across(lane < kWarps ? sh.part[lane] : Sum{-INF_F, 0.f});
  };
  if (n > 1) {
    if (terms.inv > 0.f && rank > 0) {
      const Sum all = cta_sum();
      if (tid == 0) sh.sum = all;
    }
    if (tid == 0) sh.total = total;
    cluster_sync();
    if (rank == 0) {
      int more = 0;  // of CTA `lane`, then of it and the ones before
      if (lane > 0 && lane < n)
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(more) : "r"(mapa(smem_u32(&sh.total), lane)) : "memory");
      const int own = more;
#pragma unroll
      for (int d = 1; d < kMaxCluster; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, more, d);
        if (lane >= d) more += o;
      }
      if (warp > 0 && warp < n) {  // a warp a CTA
        const int len = __shfl_sync(0xffffffffu, own, warp), to = total + __shfl_sync(0xffffffffu, more, warp) - len;
        const uint32_t src = mapa(smem_u32(sh.best), warp);
        for (int i = lane; i < len; i += 32) {
          unsigned long long x;
          asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(x) : "r"(src + 8 * i) : "memory");
          sh.best[to + i] = x;
        }
      }
      total += __shfl_sync(0xffffffffu, more, kMaxCluster - 1);
    }
  }
  Sum others[kMaxCluster];
  if (n > 1) {
    if (rank == 0 && tid == 0 && terms.inv > 0.f)
#pragma unroll
      for (int q = 1; q < kMaxCluster; ++q)
        if (q < n) {
          const uint32_t src = mapa(smem_u32(&sh.sum), q);
          asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(others[q].m), "=f"(others[q].s) : "r"(src) : "memory");
        }
    cluster_sync();  // nobody leaves before its entries are read
    if (rank > 0) return;
  }
  if (total > 2 * kThreads) {
    __syncthreads();
    cut_best<E>(&sh, total, k, terms, &t);
    total = min(total, k);
  }
  // an entry's place is the number of entries before it
  if (tid < 2) sh.best[total + tid] = 0;
  __syncthreads();
  for (int i = tid; i < total; i += kThreads) {
    const unsigned long long mine = sh.best[i];
    int place = 0;
#pragma unroll 4
    for (int j = 0; j < total; j += 2) {
      const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(&sh.best[j]);
      place += (two.x > mine) + (two.y > mine);
    }
    const Entry e = entry_of(mine);
    if (place < k) {
      a.ids[out + place] = e.idx;
      a.values[out + place] = value_of(e.key);
    } else if (terms.inv > 0.f) {
      t = terms.add(t, value_of(e.key));
    }
  }
  if (tid >= total && tid < k) {
    a.ids[out + tid] = -1;
    a.values[out + tid] = -INF_F;
  }
  if (a.tail != nullptr) {
  Sum all = cta_sum();
  if (tid == 0) {
#pragma unroll
    for (int q = 1; q < kMaxCluster; ++q)
      if (q < n) all = terms.join(all, others[q]);
    a.tail[row] = all.s == 0.f ? -INF_F : base_of(all.m) * a.inv + logf(all.s);
  }
  }
  if (next_row >= a.T) return;
  row = next_row;
  __syncthreads();  // the row's places in shared memory are free
  }
}

// CTAs a row: while the rows alone leave SMs idle and each CTA still has a chunk.
int ctas_of(int T, int V, int per) {
  int n = 1;
  while (n < kMaxCluster && (long long)T * n * 2 <= 2LL * sm_count() && V / (2 * n) >= per * kThreads * kVec / 2) n *= 2;
  return n;
}

}  // namespace

}  // namespace lora

using namespace lora;

extern "C" lora_status_t lora_topk_logits(const void* logits, int64_t ld, int32_t dtype, const int32_t* labels, int32_t T,
                                          int32_t V, int32_t k, float temperature, int32_t* ids, float* values, float* tail,
                                          int32_t* dev_err, lora_stream_t stream) {
  // without labels the ids' address stands for theirs in the check
  const lora_status_t st = check_logits(logits, ld, dtype, labels != nullptr ? labels : ids, T, V);
  if (st != LORA_OK) return st;
  if (k < 1 || k > V || !(temperature > 0.f) || temperature == INFINITY) return LORA_ERR_INVALID_ARG;
  if (k > LORA_TOPK_MAX) return LORA_ERR_UNSUPPORTED;
  if (T == 0) return LORA_OK;
  if (!f32_ok(ids) || !f32_ok(values) || !aligned_to(tail, 4)) return LORA_ERR_INVALID_ARG;
  TopkArgs a;
  memset(&a, 0, sizeof(a));
  a.logits = logits;
  a.ld = ld;
  a.labels = labels;
  a.T = T;
  a.V = V;
  a.k = k;
  const double per = 1.4426950408889634 / (double)temperature;
  a.hi = (float)per;
  if ((double)a.hi > per) a.hi = std::nextafter(a.hi, 0.f);
  a.lo = std::max((float)(per - (double)a.hi), 1e-30f);  // above 0: -inf times both parts is -inf
  a.inv = 1.f / temperature;
  a.ids = ids;
  a.values = values;
  a.tail = tail;
  a.err = dev_err;
  a.probe = wait_probe_cycles();
  const bool bf16 = dtype == LORA_LOGITS_BF16;
  const void* f = bf16 ? (const void*)topk_kernel<uint16_t> : (const void*)topk_kernel<float>;
  const int n = ctas_of(T, V, bf16 ? 8 : 4);
  const int ctas = n > 1 ? T * n : std::min(T, kResident * sm_count());
  return launch_pdl(f, dim3((unsigned)ctas), dim3(kThreads), 0, (cudaStream_t)stream, n, &a) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}
