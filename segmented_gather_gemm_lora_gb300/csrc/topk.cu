// A teacher's top logits (lora_train.h): the k largest entries of each row, and the
// log of the sum of exponentials of the others.
//
// A row is read by one CTA or by the CTAs of a cluster.  A thread reads its vectors in up
// to sixteen slots and leaves of each slot only its largest entry and its sum of
// exponentials over that: no entry is looked at by itself.  The k-th largest of the
// slots' maxima has k entries at or above it, so a slot below it has nothing to list and
// its sum stands; the others, k and those that tie with them, are read again and their
// entries below the threshold summed.  So the sum is of exactly the entries that are not
// listed, no difference of large sums.  What is listed is placed by counting.
// A row in which too many entries tie or crowd in few slots takes the slow way: a radix
// selection of the k best by passes over the row.
// Places and orders of sums are fixed: the same inputs give the same bits.
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
constexpr int kRows = 16;                         // slots of a thread; one more for the row's edges
constexpr int kListed = 512;                      // slots that are read again
constexpr int kBest = kMaxCluster * LORA_TOPK_MAX;  // entries that are placed
constexpr int kSlots = kBest / kThreads;          // of them, a thread's in a cut
constexpr int kResident = 3;                      // CTAs an SM
constexpr float kLowest = -3.402823466e38f;  // below it only -inf, which is not listed

struct TopkArgs {
  const void* logits;
  long long ld;
  const int32_t* labels;
  int T, V, k;
  Terms terms;
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
  float2 slot[kRows + 1][kThreads];  // the largest entry; sum of exponentials over it
  alignas(16) uint32_t key[kListed];  // of the slots that may be read again
  uint16_t which[kListed];
  uint32_t hist[2][256];
  int scan[kWarps];
  Sum part[kWarps];
  alignas(8) Sum sum;              // the CTA's
  uint32_t least[kWarps];          // the warps' m-th keys
  uint32_t bound[kMaxCluster];     // the cluster's CTAs' thresholds
  uint32_t threshold[2];           // of k entries, of a CTA's share of them
  int total;                       // entries in best
  alignas(16) unsigned long long best[kBest + 2];  // composite keys, then two zeros
};
static_assert(offsetof(TopShared, best) % 16 == 0 && offsetof(TopShared, key) % 16 == 0 && offsetof(TopShared, sum) % 8 == 0,
              "read in one piece");

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
// Where this thread's `mine` places begin among the CTA's, in the order of threads, and
// how many there are.  (Two barriers.)
__device__ __forceinline__ int places(int mine, TopShared* sh, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int before = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += o;
  }
  __syncthreads();
  if (lane == 31) sh->scan[warp] = before;
  __syncthreads();
  before -= mine;
  int all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? sh->scan[w] : 0;
    all += sh->scan[w];
  }
  *total = all;
  return before;
}

// The entries of best, `total` of them and more than k, cut to the k best; what goes is
// added to *t.
template <typename E>
__device__ __noinline__ void cut_best(TopShared* sh, int total, int k, const Terms& terms, Sum* t) {
  unsigned long long c[kSlots];
  Entry e[kSlots];
  int on = 0;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int at = i * kThreads + threadIdx.x;
    e[i] = entry_of(at < total ? sh->best[at] : 0);
    if (at < total) on |= 1 << i;
    c[i] = digits<E>(e[i]);
  }
  const unsigned long long least = select_top<kSlots, kFirstDigit<E>, 0>(c, [&](int i) { return on >> i & 1; }, k, sh);
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if ((on >> i & 1) && c[i] < least) {
      on &= ~(1 << i);
      if (terms.inv > 0.f) *t = terms.add(*t, value_of(e[i].key));
    }
  int at = places(__popc(on), sh, &total);
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (on >> i & 1) sh->best[at++] = composite(e[i]);
  __syncthreads();
}

// The slow way: the k best of this CTA's share of a row into best by passes over it, the
// others into *t.  Returns how many there are.
template <typename E>
__device__ __noinline__ int select_share(const Cut<E>& c, int V, int k, TopShared* sh, const Terms& terms, Sum* t) {
  constexpr int kN = Elem<E>::kN;
  const int tid = threadIdx.x, lane = tid & 31;
  // entries in rounds of a thread's one: the middle's, then the edges
  const int middle = (c.v1 - c.v0) * kN, rounds = (middle + kThreads - 1) / kThreads + 1;
  auto entry = [&](int round) {
    int idx = round * kThreads + tid;
    idx = round + 1 < rounds ? (idx < middle ? c.head + c.v0 * kN + idx : -1) : edge_of(c, V, tid);
    const float x = idx >= 0 ? Elem<E>::get(c.row[idx]) : -INF_F;
    return Entry{x < kLowest ? 0 : key_of(x), idx};  // key 0: nothing to list
  };
  int listed = 0;
  for (int i = 0; i < rounds; ++i) listed += entry(i).key != 0;
  int total;
  places(listed, sh, &total);
  const int n = min(total, k);
  unsigned long long least = 0, mask = 0;
  if (total > k) {
    int want = k;
    for (int shift = kFirstDigit<E>; shift >= 0; shift -= 8) {
      __syncthreads();
      sh->hist[0][tid] = 0;
      __syncthreads();
      for (int i = 0; i < rounds; ++i) {
        const Entry e = entry(i);
        const unsigned long long d = digits<E>(e);
        const bool in = e.key != 0 && (d & mask) == least;
        // lanes of one bin add once
        const uint32_t bin = in ? (uint32_t)(d >> shift) & 255 : 256;
        const uint32_t same = __match_any_sync(0xffffffffu, bin);
        if (in && lane == __ffs(same) - 1) atomicAdd(&sh->hist[0][bin], (uint32_t)__popc(same));
      }
      __syncthreads();
      int bin = 255;
      for (; bin > 0 && (int)sh->hist[0][bin] < want; --bin) want -= (int)sh->hist[0][bin];
      least |= (unsigned long long)bin << shift;
      mask |= 255ull << shift;
      if ((int)sh->hist[0][bin] == want) break;
    }
  }
  int at = 0;
  for (int i = 0; i < rounds; ++i) {
    const Entry e = entry(i);
    const bool in = e.key != 0 && digits<E>(e) >= least;
    int some;
    const int to = at + places(in, sh, &some);
    if (in) sh->best[to] = composite(e);
    else if (e.key != 0 && terms.inv > 0.f) *t = terms.add(*t, value_of(e.key));
    at += some;
  }
  return n;
}

template <typename E>
__global__ void __launch_bounds__(kThreads, kResident) topk_kernel(const __grid_constant__ TopkArgs a) {
  constexpr int kN = Elem<E>::kN;
  extern __shared__ __align__(16) uint8_t shared_bytes[];
  TopShared& sh = *reinterpret_cast<TopShared*>(shared_bytes);
  const int n = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait_then_release();
  if (a.probe > 0) {
    if (tid == 0 && !wait_probe(&sh.probe_bar, a.probe)) report(a.err, LORA_DERR_TIMEOUT);
    return;
  }
  const int k = a.k, m = (k + kWarps - 1) / kWarps;
  const Terms terms{a.terms.near, a.tail != nullptr ? a.terms.inv : 0.f};
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
    const int next_row = n == 1 && row < a.T - (int)gridDim.x ? row + (int)gridDim.x : a.T;
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
    int total = 0;
    const int chunks = (c.v1 - c.v0 + kVec * kThreads - 1) / (kVec * kThreads), group = (chunks + kRows - 1) / kRows;  // chunks of a slot
    const int slots = group > 0 ? (chunks + group - 1) / group : 0;
    for (int s = 0, chunk = 0; s < slots; ++s) {
      Sum w{-INF_F, 0.f};
      float top = -INF_F;  // w's maximum, or a NaN
      for (int g = 0; g < group && chunk < chunks; ++g, ++chunk) {
        load(c, c.v0 + tid + (chunk + 1) * kVec * kThreads, next);
        float m = top_nan(r[0], E{});
#pragma unroll
        for (int u = 1; u < kVec; ++u) m = max_nan(m, top_nan(r[u], E{}));
        top = max_nan(top, m);
        if (terms.inv > 0.f) w = add_vectors<E>(terms, w, r, m);
#pragma unroll
        for (int u = 0; u < kVec; ++u) r[u] = next[u];
      }
      sh.slot[s][tid] = make_float2(top, w.s);
    }
    {
      const int e = edge_of(c, a.V, tid);
      const float x = e >= 0 ? Elem<E>::get(c.row[e]) : -INF_F;
      sh.slot[slots][tid] = make_float2(x, x == -INF_F ? 0.f : x == INF_F ? x : 1.f);
    }
    load_next();

    // A threshold to begin with: the least of the warps' m-th lanes' largest entries, above
    // -inf; then the slots that reach it.
    float mine = -INF_F;
    for (int s = 0; s <= slots; ++s) mine = max_nan(mine, sh.slot[s][tid].x);
    const uint32_t sorted = sort_lanes(key_of(mine), lane);
    if (lane == m - 1) sh.least[warp] = sorted;
    __syncthreads();
    uint32_t floor_ = sh.least[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) floor_ = min(floor_, sh.least[w]);
    floor_ = max(floor_, key_of(kLowest));
    // x reaches key `least` (a NaN reaches every key, and only a NaN a NaN's)
    auto reaches = [](float x, float least) { return least == least ? !(x < least) : x != x; };
    auto slots_from = [&](uint32_t least) {
      const float v = value_of(least);
      int some = 0;
      for (int s = 0; s <= slots; ++s) some += reaches(sh.slot[s][tid].x, v);
      return some;
    };
    int n_listed;
    int at = places(slots_from(floor_), &sh, &n_listed);
    if (n_listed > kListed) {
      // bit by bit up to the k-th largest (its upper 16 bits)
      uint32_t step = 1u << 31;
      for (uint32_t high = 0; step >= 1u << 16; step >>= 1) {
        const uint32_t next_key = high | step;
        places(slots_from(next_key), &sh, &n_listed);
        if (n_listed >= k) high = next_key;
        if (step == 1u << 16) floor_ = max(floor_, high);
      }
      at = places(slots_from(floor_), &sh, &n_listed);
    }
    bool slow = n_listed > kListed;  // the same for all threads
    uint32_t bound = floor_;
    if (!slow) {
      const float least = value_of(floor_);
      for (int s = 0; s <= slots; ++s) {
        const float x = sh.slot[s][tid].x;
        if (reaches(x, least)) {
          sh.key[at] = key_of(x);
          sh.which[at++] = (uint16_t)(s * kThreads + tid);
        }
      }
      const int padded = (n_listed + 3) & ~3;
      if (tid < padded - n_listed) sh.key[n_listed + tid] = 0;
      if (tid < 2) sh.threshold[tid] = floor_;
      __syncthreads();
      const int share = (k + n - 1) / n;
      for (int i = tid; i < n_listed; i += kThreads) {
        const uint32_t own = sh.key[i];
        int above = 0, same = 0;
#pragma unroll 4
        for (int j = 0; j < padded; j += 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(&sh.key[j]);
          above += (x.x > own) + (x.y > own) + (x.z > own) + (x.w > own);
          same += (x.x == own) + (x.y == own) + (x.z == own) + (x.w == own);
        }
        if (above < k && k <= above + same) sh.threshold[0] = own;  // alike where several write
        if (above < share && share <= above + same) sh.threshold[1] = own;
      }
      __syncthreads();
      bound = sh.threshold[1];
    }
    if (n > 1) {  // entries of the whole row, a share of k from each CTA, that reach the least of the bounds
      cluster_sync();  // every CTA's places are there
      if (tid < n) st_dsmem_u32(mapa(smem_u32(&sh.bound[rank]), tid), bound);
      cluster_sync();
      for (int i = 0; i < n; ++i) bound = min(bound, sh.bound[i]);
    } else {
      bound = 0;
    }
    const uint32_t threshold = slow ? 0 : max(bound, sh.threshold[0]);
    if (!slow) {
      // The entries that reach it, of the slots that do; a slot's other entries into the sum.
      // A thread a slot; f(vectors, what reaches of them, the place of an element of them).
      const float least = value_of(threshold);
      const uint4* const mid = reinterpret_cast<const uint4*>(c.row + c.head);
      auto each = [&](int id, auto f) {
        const int s = id / kThreads, thread = id % kThreads;
        uint4 x[kVec];
        if (s == slots) {
          const int e = edge_of(c, a.V, thread);
#pragma unroll
          for (int u = 0; u < kVec; ++u) x[u] = low_vector<E>();
          const float v = e >= 0 ? Elem<E>::get(c.row[e]) : -INF_F;
          x[0].x = sizeof(E) == 2 ? 0xff800000u | __float_as_uint(v) >> 16 : __float_as_uint(v);
          f(x, reaches(v, least) ? 1u : 0u, [&](int) { return e; });
          return;
        }
        for (int chunk = s * group; chunk < min(chunks, (s + 1) * group); ++chunk) {
          const int i = c.v0 + chunk * kVec * kThreads + thread;
          uint32_t which = 0;
#pragma unroll
          for (int u = 0; u < kVec; ++u) x[u] = i + u * kThreads < c.v1 ? mid[i + u * kThreads] : low_vector<E>();
          if (least == least) {
#pragma unroll
            for (int u = 0; u < kVec; ++u) which |= reaching(x[u], least, E{}) << (u * kN);
          } else {  // NaNs alone: what is not below +inf, but +inf itself
#pragma unroll
            for (int u = 0; u < kVec; ++u)
#pragma unroll
              for (int j = 0; j < kN; ++j) {
                const float v = Elem<E>::get(Elem<E>::entry(x[u], j));
                which |= (v != v ? 1u : 0u) << (u * kN + j);
              }
          }
          f(x, which, [&](int b) { return c.head + (i + b / kN * kThreads) * kN + b % kN; });
        }
      };
      auto hide = [&](uint4 (&x)[kVec], uint32_t which) {
#pragma unroll
        for (int u = 0; u < kVec; ++u) x[u] = without(x[u], which >> (u * kN) & ((1u << kN) - 1), E{});
      };
      int some = 0;
      float top = -INF_F;  // of those below it
      for (int i = tid; i < n_listed; i += kThreads)
        if (sh.key[i] >= threshold)
          each(sh.which[i], [&](uint4 (&x)[kVec], uint32_t which, auto) {
            some += __popc(which);
            hide(x, which);
            top = fmaxf(top, Elem<E>::top(x));
          });
      at = places(some, &sh, &total);
      slow = total > kBest;
      if (!slow) {
        const float base = base_of(top);
        float rest = 0.f;
        for (int i = tid; i < n_listed; i += kThreads)
          if (sh.key[i] >= threshold)
            each(sh.which[i], [&](uint4 (&x)[kVec], uint32_t which, auto place) {
              for (uint32_t w = which; w != 0; w &= w - 1) {
                const int idx = place(__ffs(w) - 1);
                sh.best[at++] = composite(Entry{key_of(Elem<E>::get(c.row[idx])), idx});
              }
              hide(x, which);
              if (terms.inv > 0.f) rest += power_sum<E>(terms, x, base);
            });
        if (terms.inv > 0.f) {
          for (int s = 0; s <= slots; ++s) {
            const float x = sh.slot[s][tid].x;
            top = fmaxf(top, reaches(x, least) ? -INF_F : x);
          }
          t = Sum{top, rest == 0.f ? 0.f : rest * terms.power(base, base_of(top))};
          for (int s = 0; s <= slots; ++s) {
            const float2 w = sh.slot[s][tid];
            if (w.x != -INF_F && !reaches(w.x, least)) t.s += w.y * terms.power(base_of(w.x), base_of(top));
          }
        }
        __syncthreads();
        if (n > 1 && total > LORA_TOPK_MAX) {
          cut_best<E>(&sh, total, k, terms, &t);
          total = k;
        }
      }
    }
    if (slow) total = select_share<E>(c, a.V, k, &sh, terms, &t);
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
      total = k;
    }
    // an entry's place is the number of entries before it
    if (tid < 2) sh.best[total + tid] = 0;
    __syncthreads();
    const int parts = total <= kThreads / 4 ? 4 : total <= kThreads / 2 ? 2 : 1;  // threads that share an entry's counting
    for (int i = tid / parts; i - tid / parts < total; i += kThreads / parts) {
      const unsigned long long mine = i < total ? sh.best[i] : ~0ull;
      int place = 0;
#pragma unroll 4
      for (int j = 2 * (tid % parts); j < total; j += 2 * parts) {
        const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(&sh.best[j]);
        place += (two.x > mine) + (two.y > mine);
      }
      for (int d = 1; d < parts; d <<= 1) place += __shfl_xor_sync(0xffffffffu, place, d);
      if (i >= total || tid % parts != 0) continue;
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
        a.tail[row] = all.s == 0.f ? -INF_F : base_of(all.m) * a.terms.inv + logf(all.s);
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
  a.terms = terms_of(temperature);
  a.ids = ids;
  a.values = values;
  a.tail = tail;
  a.err = dev_err;
  a.probe = wait_probe_cycles();
  const bool bf16 = dtype == LORA_LOGITS_BF16;
  const void* f = bf16 ? (const void*)topk_kernel<uint16_t> : (const void*)topk_kernel<float>;
  const int n = ctas_of(T, V, bf16 ? 8 : 4);
  if (ensure_smem_attr(f, sizeof(TopShared)) != cudaSuccess) return LORA_ERR_CUDA;
  const int ctas = n > 1 ? T * n : std::min(T, kResident * sm_count());
  return launch_pdl(f, dim3((unsigned)ctas), dim3(kThreads), sizeof(TopShared), (cudaStream_t)stream, n, &a) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}
