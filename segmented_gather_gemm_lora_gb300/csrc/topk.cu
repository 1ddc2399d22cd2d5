// A teacher's top logits (lora_train.h): the k largest entries of each row, and the
// log of the sum of exponentials of the others.
//
// A row is read by one CTA of 32 to 512 threads.  A thread reads its vectors in up to sixteen
// slots and leaves of each slot only its largest entry and its sum of exponentials over that:
// no entry is looked at by itself.  A value that k of the slots' largest entries reach has k
// entries at or above it, so a slot below it has nothing to list and its sum stands; the
// others, k and some more, are read again (from L2), what reaches the value is listed and
// the rest of them summed.  So the sum is of exactly the entries that are not listed, no
// difference of large sums (but for ties, below).  What is listed is put in order in runs of 32;
// an entry's place is its place in its run and those that a search finds in the others.
// Where too many entries tie with the k-th largest (a mask's lowest value, say) those above it
// are listed so, then the first of the ties, which are taken out of the sum: at most half of it.
// A row in which too many crowd in few slots takes the slow way: a radix selection of the k best
// by passes over the row.  So do ordinary rows that are short for their list: with two or three
// vectors a thread, more entries than there is room for reach what k threads' largest do
// (8192 x 5000 bf16 with 250 listed 930 us, with 64 of 32000 94).
// Places and orders of sums are fixed: the same inputs give the same bits.
//
// Keys are the values' bits made to order as integers; composite keys order as the
// listing does, no two alike.
//
// What bounds it: of long rows latency (4096 x 128256 bf16, 64 listed: 236 us, 4.4 TB/s; without
// tail 211): half of the issue slots are used and warps wait for loads, of which only one or two chunks
// are on their way, and one of the next row while a row is finished; of short ones what is done once a
// row, about ten barriers.
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

constexpr int kVec = 4;       // vectors a thread takes at once
constexpr int kRows = 16;     // slots of a thread; one more for the row's edges
template <int kT>
constexpr int kListed = kT > 256 ? 2 * kT : 4 * kT;  // slots that are read again; entries that are placed at once
template <int kT>
constexpr int kAhead = kT > 256 ? 2 : 1;  // chunks under way: few rows wait for memory alone
constexpr int kResident = 896;  // threads an SM (4096 x 128256: 234 us; 640 258, 768 243, 1024, which spills, 310)
constexpr float kLowest = -3.402823466e38f;  // below it only -inf, which is not listed

constexpr int kMostEntries = 0x7fff0000;  // steps over a row end past it by less than 2^16, within 32 bits

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
struct Entry {
  uint32_t key;
  int idx;
};
__device__ __forceinline__ unsigned long long composite(const Entry& e) {
  return (unsigned long long)e.key << 32 | (uint32_t)~e.idx;
}

__device__ __forceinline__ Entry entry_of(unsigned long long c) { return Entry{(uint32_t)(c >> 32), (int)~(uint32_t)c}; }

template <int kT>
struct TopShared {
  static constexpr int kWarps = kT / 32;
  uint64_t probe_bar;
  float2 slot[kRows + 1][kT];  // the largest entry; sum of exponentials over it
  alignas(16) uint32_t key[kListed<kT>];  // of the slots that may be read again
  uint16_t which[kListed<kT>];
  uint32_t hist[256];
  int scan[kWarps];
  Sum part[kWarps];
  uint32_t least[kWarps], most[kWarps];  // the warps' m-th keys, and their first
  uint32_t threshold;              // of the slots
  int total;                       // entries in best
  alignas(16) unsigned long long best[kListed<kT>];  // composite keys
};
static_assert(offsetof(TopShared<256>, key) % 16 == 0 && offsetof(TopShared<32>, key) % 16 == 0, "read in one piece");

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

// The warp's composite keys in falling order, likewise.
__device__ __forceinline__ unsigned long long sort_lanes(unsigned long long c, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int d = size >> 1; d > 0; d >>= 1) {
      const unsigned long long o = __shfl_xor_sync(0xffffffffu, c, d);
      const bool up = (lane & size) != 0 && size < 32, low = (lane & d) == 0;
      c = (low != up) == (c > o) ? c : o;
    }
  return c;
}

// The bin of 256 that holds the want-th largest (every warp finds it; lane l looks at bins
// 8 l .. 8 l + 7).
__device__ __forceinline__ int find_bin(const uint32_t* h, uint32_t want) {
  const int lane = threadIdx.x & 31;
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
  const bool here = above < want && want <= above + mine;
  int bin = 0;
  if (here)
#pragma unroll
    for (int i = 7; i >= 0; --i) {
      if (above < want && want <= above + bins[i]) bin = lane * 8 + i;
      above += bins[i];
    }
  return __shfl_sync(0xffffffffu, bin, __ffs(__ballot_sync(0xffffffffu, here)) - 1);
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
// how many there are.  (Two barriers; kFree, one: a barrier has passed since the last call.)
template <bool kFree, int kT>
__device__ __forceinline__ int places(int mine, TopShared<kT>* sh, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int before = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += o;
  }
  if (!kFree) __syncthreads();
  if (lane == 31) sh->scan[warp] = before;
  __syncthreads();
  before -= mine;
  int all = 0;
#pragma unroll
  for (int w = 0; w < kT / 32; ++w) {
    before += w < warp ? sh->scan[w] : 0;
    all += sh->scan[w];
  }
  *total = all;
  return before;
}

// The slow way: the k best of a row into best by passes over it, the others into *t.  Returns
// how many there are.
template <typename E, int kT>
__device__ __noinline__ int select_row(const Cut<E>& c, int V, int k, TopShared<kT>* sh, const Terms& terms, Sum* t) {
  constexpr int kN = Elem<E>::kN;
  const int tid = threadIdx.x, lane = tid & 31;
  // entries in rounds of a thread's one: the middle's, then the edges
  const int middle = (c.v1 - c.v0) * kN, rounds = (middle + kT - 1) / kT + 1;
  auto entry = [&](int round) {
    int idx = round * kT + tid;
    idx = round + 1 < rounds ? (idx < middle ? c.head + c.v0 * kN + idx : -1) : edge_of(c, V, tid);
    const float x = idx >= 0 ? Elem<E>::get(c.row[idx]) : -INF_F;
    return Entry{x < kLowest ? 0 : key_of(x), idx};  // key 0: nothing to list
  };
  int listed = 0;
  for (int i = 0; i < rounds; ++i) listed += entry(i).key != 0;
  int total;
  places<false>(listed, sh, &total);
  const int n = min(total, k);
  unsigned long long least = 0, mask = 0;
  if (total > k) {
    int want = k;
    for (int shift = kFirstDigit<E>; shift >= 0; shift -= 8) {
      __syncthreads();
      for (int b = tid; b < 256; b += kT) sh->hist[b] = 0;
      __syncthreads();
      for (int i = 0; i < rounds; ++i) {
        const Entry e = entry(i);
        const unsigned long long d = digits<E>(e);
        const bool in = e.key != 0 && (d & mask) == least;
        // lanes of one bin add once
        const uint32_t bin = in ? (uint32_t)(d >> shift) & 255 : 256;
        const uint32_t same = __match_any_sync(0xffffffffu, bin);
        if (in && lane == __ffs(same) - 1) atomicAdd(&sh->hist[bin], (uint32_t)__popc(same));
      }
      __syncthreads();
      int bin = 255;
      for (; bin > 0 && (int)sh->hist[bin] < want; --bin) want -= (int)sh->hist[bin];
      least |= (unsigned long long)bin << shift;
      mask |= 255ull << shift;
      if ((int)sh->hist[bin] == want) break;
    }
  }
  int at = 0;
  for (int i = 0; i < rounds; ++i) {
    const Entry e = entry(i);
    const bool in = e.key != 0 && digits<E>(e) >= least;
    int some;
    const int to = at + places<false>(in, sh, &some);
    if (in) sh->best[to] = composite(e);
    else if (e.key != 0 && terms.inv > 0.f) *t = terms.add(*t, value_of(e.key));
    at += some;
  }
  __syncthreads();  // the last round's entries (the edges, one warp's) are there for the warps that sort them
  return n;
}

template <typename E, int kT>
__global__ void __launch_bounds__(kT, kT > kResident ? 1 : kResident / kT) topk_kernel(const __grid_constant__ TopkArgs a) {
  constexpr int kN = Elem<E>::kN;
  extern __shared__ __align__(16) uint8_t shared_bytes[];
  TopShared<kT>& sh = *reinterpret_cast<TopShared<kT>*>(shared_bytes);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait_then_release();
  if (a.probe > 0) {
    if (tid == 0 && !wait_probe(&sh.probe_bar, a.probe)) report(a.err, LORA_DERR_TIMEOUT);
    return;
  }
  const int k = a.k, m = (k + kT / 32 - 1) / (kT / 32);
  const Terms terms{a.terms.near, a.tail != nullptr ? a.terms.inv : 0.f};
  auto cut_at = [&](int row) { return cut_row(static_cast<const E*>(a.logits) + (long long)row * a.ld, a.V, 0, 1); };
  auto load = [&](const Cut<E>& c, int i, uint4 (&r)[kVec]) {
    const uint4* const mid = reinterpret_cast<const uint4*>(c.row + c.head);
#pragma unroll
    for (int u = 0; u < kVec; ++u) r[u] = i + u * kT < c.v1 ? mid[i + u * kT] : low_vector<E>();
  };
  uint4 r[kVec], ahead[kAhead<kT>][kVec];
  int row = (int)blockIdx.x;
  {
    const Cut<E> c = cut_at(row);
    load(c, c.v0 + tid, r);
  }
  // (each row's first chunk is loaded before the row before it is finished)
  for (;;) {
    const int next_row = row < a.T - (int)gridDim.x ? row + (int)gridDim.x : a.T;
    const long long out = (long long)row * k;
    const Cut<E> c = cut_at(row);
    auto load_next = [&] {
      if (next_row < a.T) {
        const Cut<E> d = cut_at(next_row);
        load(d, d.v0 + tid, r);
      }
    };
    if (a.labels != nullptr && a.labels[row] < 0) {
      for (int i = tid; i < k; i += kT) {
        a.ids[out + i] = -1;
        a.values[out + i] = -INF_F;
      }
      if (tid == 0 && a.tail != nullptr) a.tail[row] = -INF_F;
      load_next();
      if (next_row >= a.T) return;
      row = next_row;
      continue;
    }
    Sum t{-INF_F, 0.f};
    float mine = -INF_F;  // the thread's largest entry, or a NaN
    int total = 0;
    const int chunks = (c.v1 - c.v0 + kVec * kT - 1) / (kVec * kT), group = (chunks + kRows - 1) / kRows;  // chunks of a slot
    const int slots = group > 0 ? (chunks + group - 1) / group : 0;
#pragma unroll
    for (int i = 0; i + 1 < kAhead<kT>; ++i) load(c, c.v0 + tid + (i + 1) * kVec * kT, ahead[i]);
    for (int s = 0, chunk = 0; s < slots; ++s) {
      Sum w{-INF_F, 0.f};
      float top = -INF_F;  // w's maximum, or a NaN
      for (int g = 0; g < group && chunk < chunks; ++g, ++chunk) {
        load(c, c.v0 + tid + (chunk + kAhead<kT>) * kVec * kT, ahead[kAhead<kT> - 1]);
        float m = top_nan(r[0], E{});
#pragma unroll
        for (int u = 1; u < kVec; ++u) m = max_nan(m, top_nan(r[u], E{}));
        top = max_nan(top, m);
        if (terms.inv > 0.f) w = add_vectors<E>(terms, w, r, m);
#pragma unroll
        for (int u = 0; u < kVec; ++u) {
          r[u] = ahead[0][u];
          if constexpr (kAhead<kT> == 2) ahead[0][u] = ahead[1][u];
        }
      }
      sh.slot[s][tid] = make_float2(top, w.s);
      mine = max_nan(mine, top);
    }
    {
      const int e = edge_of(c, a.V, tid);
      const float x = e >= 0 ? Elem<E>::get(c.row[e]) : -INF_F;
      sh.slot[slots][tid] = make_float2(x, x == -INF_F ? 0.f : x == INF_F ? x : 1.f);
      mine = max_nan(mine, x);
    }
    load_next();

    // A threshold to begin with: the least of the warps' m-th lanes' largest entries, above
    // -inf; then the slots that reach it.
    const uint32_t sorted = sort_lanes(key_of(mine), lane);
    if (lane == m - 1) sh.least[warp] = sorted;
    if (lane == 0) sh.most[warp] = sorted;
    if (tid == 0) sh.total = 0;
    __syncthreads();
    uint32_t floor_ = sh.least[0];
#pragma unroll
    for (int w = 1; w < kT / 32; ++w) floor_ = min(floor_, sh.least[w]);
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
    int at = places<true>(slots_from(floor_), &sh, &n_listed);
    if (n_listed > kT) {
      // nearer to the k-th largest: the slots counted in 256 equal steps up to the row's largest
      uint32_t high = sh.most[0];
#pragma unroll
      for (int w = 1; w < kT / 32; ++w) high = max(high, sh.most[w]);
      const float lo = value_of(floor_), hi = value_of(high), step = (hi - lo) * (1.f / 256.f), per = 1.f / step;
      if (step > 0.f && step < INF_F && per < INF_F) {
        for (int b = tid; b < 256; b += kT) sh.hist[b] = 0;
        __syncthreads();
        for (int s = 0; s <= slots; ++s) {
          const float x = sh.slot[s][tid].x;
          if (reaches(x, lo)) atomicAdd(&sh.hist[min(255, (int)((x - lo) * per))], 1u);
        }
        __syncthreads();
        const float v = fmaf((float)find_bin(sh.hist, (uint32_t)k), step, lo);
        // (a little lower: no slot of that step or a later one is below it for the roundings)
        floor_ = max(floor_, key_of(v - 1e-6f * (fabsf(lo) + fabsf(hi))));
        at = places<true>(slots_from(floor_), &sh, &n_listed);
      }
    }
    // What is below these is one key to the row's values.
    constexpr uint32_t kUnit = sizeof(E) == 2 ? 0x10000u : 1u;
    auto above = [](uint32_t key) { return (key & ~(kUnit - 1)) + kUnit; };  // 0: nothing is
    bool ties = false;  // too much ties with the k-th largest: what is above it is listed, and the first that tie
    uint32_t kth = 0;
    if (n_listed > kListed<kT>) {
      // bit by bit up to the k-th largest
      for (uint32_t step = 1u << 31; step >= kUnit; step >>= 1) {
        places<false>(slots_from(kth | step), &sh, &n_listed);
        if (n_listed >= k) kth |= step;
      }
      floor_ = kth;
      at = places<false>(slots_from(floor_), &sh, &n_listed);
      if (n_listed > kListed<kT> && above(kth) != 0) {
        ties = true;
        floor_ = above(kth);
        at = places<false>(slots_from(floor_), &sh, &n_listed);
      }
    }
    bool slow = n_listed > kListed<kT>;  // the same for all threads
    uint32_t threshold = floor_;
    // Or of the slots' k-th largest.
    auto rank_slots = [&] {
      const int padded = (n_listed + 3) & ~3;
      if (tid < padded - n_listed) sh.key[n_listed + tid] = 0;
      if (tid == 0) sh.threshold = floor_;
      __syncthreads();
      for (int i = tid; i < n_listed; i += kT) {
        const uint32_t own = sh.key[i];
        int above = 0, same = 0;
#pragma unroll 4
        for (int j = 0; j < padded; j += 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(&sh.key[j]);
          above += (x.x > own) + (x.y > own) + (x.z > own) + (x.w > own);
          same += (x.x == own) + (x.y == own) + (x.z == own) + (x.w == own);
        }
        if (above < k && k <= above + same) sh.threshold = own;  // alike where several write
      }
      __syncthreads();
      threshold = sh.threshold;
    };
    // The entries that reach `threshold`, of the slots that do, to best in any order; a slot's
    // other entries into t.  A thread a slot.  Returns how many they are.
    const uint4* const mid = reinterpret_cast<const uint4*>(c.row + c.head);
    auto collect = [&](uint32_t threshold) {
      const float least = value_of(threshold);
      t = Sum{-INF_F, 0.f};
      for (int i = tid; i - lane < n_listed; i += kT) {
        const bool on = i < n_listed && sh.key[i] >= threshold;
        if (!__any_sync(0xffffffffu, on)) continue;
        const int s = on ? sh.which[i] / kT : 0, thread = on ? sh.which[i] % kT : 0;
        const bool edge = on && s == slots;
        for (int g = 0; g < max(group, 1); ++g) {
          const int chunk = s * group + g, from = c.v0 + chunk * kVec * kT + thread;
          const int e = edge_of(c, a.V, thread);
          uint4 x[kVec];
#pragma unroll
          for (int u = 0; u < kVec; ++u)
            x[u] = on && !edge && chunk < chunks && from + u * kT < c.v1 ? mid[from + u * kT] : low_vector<E>();
          if (edge && g == 0 && e >= 0) {
            const uint32_t v = __float_as_uint(Elem<E>::get(c.row[e]));
            x[0].x = sizeof(E) == 2 ? 0xff800000u | v >> 16 : v;
          }
          uint32_t which = 0;
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
          const int some = __popc(which);
          int to = some;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, to, d);
            if (lane >= d) to += o;
          }
          int first = 0;
          if (lane == 31 && to > 0) first = atomicAdd(&sh.total, to);
          to += __shfl_sync(0xffffffffu, first, 31) - some;
          for (uint32_t w = which; w != 0; w &= w - 1, ++to) {
            const int b = __ffs(w) - 1, u = b / kN;
            const uint4 v = u == 0 ? x[0] : u == 1 ? x[1] : u == 2 ? x[2] : x[3];
            const int idx = edge ? e : c.head + (from + u * kT) * kN + b % kN;
            if (to < kListed<kT>) sh.best[to] = composite(Entry{key_of(Elem<E>::get(Elem<E>::entry(v, b % kN))), idx});
          }
          if (terms.inv > 0.f && on) {
#pragma unroll
            for (int u = 0; u < kVec; ++u) x[u] = without(x[u], which >> (u * kN) & ((1u << kN) - 1), E{});
            t = add_vectors<E>(terms, t, x, Elem<E>::top(x));
          }
        }
      }
      __syncthreads();
      return sh.total;
    };
    if (!slow) {
      const float least = value_of(floor_);
      for (int s = 0; s <= slots; ++s) {
        const float x = sh.slot[s][tid].x;
        if (reaches(x, least)) {
          sh.key[at] = key_of(x);
          sh.which[at++] = (uint16_t)(s * kT + tid);
        }
      }
      __syncthreads();
      // (a threshold of nothing but the least value: fewer slots than it takes, so all their entries reach it)
      if (!ties && floor_ <= key_of(kLowest)) rank_slots();
      total = collect(threshold);
      if (total > kListed<kT> && !ties) {
        __syncthreads();
        if (tid == 0) sh.total = 0;
        rank_slots();
        total = collect(threshold);
        if (total > kListed<kT> && above(threshold) != 0) {
          __syncthreads();
          if (tid == 0) sh.total = 0;
          __syncthreads();
          ties = true;
          kth = threshold;
          threshold = above(kth);
          total = collect(threshold);
        }
      }
      slow = total > kListed<kT>;
      if (!slow) {
        if (terms.inv > 0.f) {
          const float least = value_of(threshold);
          float top = t.m;
          for (int s = 0; s <= slots; ++s) {
            const float x = sh.slot[s][tid].x;
            top = fmaxf(top, reaches(x, least) ? -INF_F : x);
          }
          t = Sum{top, t.s == 0.f ? 0.f : t.s * terms.power(base_of(t.m), base_of(top))};
          for (int s = 0; s <= slots; ++s) {
            const float2 w = sh.slot[s][tid];
            if (w.x != -INF_F && !reaches(w.x, least)) t.s += w.y * terms.power(base_of(w.x), base_of(top));
          }
        }
      }
    }
    // The first entries of the tied value, in the row's order, fill the list.  Their slots' sums
    // have them, so they are taken out of the row's: at least twice as many stay.
    int taken = 0;
    const float tied = sizeof(E) == 4 || (kth & 0x80000000u) ? value_of(kth & ~(kUnit - 1)) : value_of(kth | 0xffffu);
    if (!slow && ties && total < k) {
      taken = k - total;
      int found = 0;
      auto take = [&](uint32_t which, int from) {  // elements of this thread, in the order of threads
        int some;
        int to = found + places<false>(__popc(which), &sh, &some);
        for (; which != 0 && to < taken; which &= which - 1, ++to)
          sh.best[total + to] = composite(Entry{key_of(tied), from + __ffs(which) - 1});
        found += some;
      };
      if (c.head > 0) take(tid < c.head && Elem<E>::get(c.row[tid]) == tied, tid);
      for (int i0 = 0; i0 < c.nvec && found < taken; i0 += kT) {
        uint32_t which = 0;
        if (i0 + tid < c.nvec) {
          const uint4 x = mid[i0 + tid];
#pragma unroll
          for (int j = 0; j < kN; ++j) which |= (Elem<E>::get(Elem<E>::entry(x, j)) == tied ? 1u : 0u) << j;
        }
        take(which, c.head + (i0 + tid) * kN);
      }
      if (found < taken) take(tid < a.V - c.tail0 && Elem<E>::get(c.row[c.tail0 + tid]) == tied, c.tail0 + tid);
      total = k;
      __syncthreads();
    }
    if (slow) t = Sum{-INF_F, 0.f};
    if (slow) total = select_row<E, kT>(c, a.V, k, &sh, terms, &t);
    // An entry's place is the number of entries before it: runs of 32 are put in order, then each
    // entry is looked for in the other runs.
    const int runs = (total + 31) / 32;
    for (int r = warp; r < runs; r += kT / 32) {
      const int i = r * 32 + lane;
      sh.best[i] = sort_lanes(i < total ? sh.best[i] : 0ull, lane);
    }
    __syncthreads();
    for (int i = tid; i - lane < total; i += kT) {
      const unsigned long long own = sh.best[i];
      if (own == 0) continue;
      int place = lane;
#pragma unroll 4
      for (int r = 0; r < runs; ++r) {
        const unsigned long long* const run = sh.best + r * 32;
        int before = 0;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) before += run[before + d - 1] > own ? d : 0;
        before += run[before] > own;
        place += r == i / 32 ? 0 : before;
      }
      const Entry e = entry_of(own);
      if (place < k) {
        a.ids[out + place] = e.idx;
        a.values[out + place] = value_of(e.key);
      } else {
        sh.key[place - k] = __float_as_uint(value_of(e.key));  // by its place: the sum's order is fixed
      }
    }
    if (total > k && terms.inv > 0.f) {
      __syncthreads();
      for (int i = tid; i < total - k; i += kT) t = terms.add(t, __uint_as_float(sh.key[i]));
    }
    for (int i = total + tid; i < k; i += kT) {
      a.ids[out + i] = -1;
      a.values[out + i] = -INF_F;
    }
    if (a.tail != nullptr) {
      const Sum w = terms.across(t);
      if (lane == 0) sh.part[warp] = w;
      __syncthreads();
      Sum all = terms.across(lane < kT / 32 ? sh.part[lane] : Sum{-INF_F, 0.f});
      if (taken > 0 && all.m < INF_F) all.s -= (float)taken * terms.power(tied, base_of(all.m));
      if (tid == 0) a.tail[row] = all.s == 0.f ? -INF_F : base_of(all.m) * a.terms.inv + logf(all.s);
    }
    if (next_row >= a.T) return;
    row = next_row;
    __syncthreads();  // the row's places in shared memory are free
  }
}

template <typename E, int kT>
lora_status_t launch(TopkArgs& a, cudaStream_t s) {
  const void* const f = (const void*)topk_kernel<E, kT>;
  if (ensure_smem_attr(f, sizeof(TopShared<kT>)) != cudaSuccess) return LORA_ERR_CUDA;
  const int ctas = std::min(a.T, kResident / kT * sm_count());
  return launch_pdl(f, dim3((unsigned)ctas), dim3(kT), sizeof(TopShared<kT>), s, 0, &a) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

// The threads of a row (device times in us on a GB300, rows that fill the GPU unless
// said; measured with 768 threads an SM, kResident 896 since):
//  - the fewer, the more rows are under way and the less a row's fixed part costs: 8192 x 1000
//    bf16 with 20 listed and 32 / 64 / 128 / 256 threads 28 / 44 / 63 / 145; 4096 x 20000 with 60
//    listed - / 69 / 72 / 92;
//  - but a long row is at its threshold sooner with more: 4096 x 128256 with 64 listed - / 277 /
//    243 / 250, 2000 x 128256 fp32 - / 296 / 237 / 216;
//  - and few rows want all of the GPU: 200 x 5000 8.5 / 6.7 / 6.8 / 7.9, 300 x 128256 - / 55 / 34.5 /
//    28.7; 64 x 128256 with 256 / 512 threads 18.9 / 14.8, 300 x 128256 28.7 / 30.2. (Clusters of two to
//    eight CTAs of 256 a row: 64 x 128256 17.9 to 25.9, 16 x 32000 9.8 to 10.4, one CTA 7.7.)
//  - A list takes a lane's place in every warp, so k threads at least; where the row has few
//    vectors for it, more: 8192 x 1000 with 60 listed 105 with 64 threads, 81 with 128.
template <typename E>
lora_status_t launch_for(TopkArgs& a, cudaStream_t s) {
  const int sms = sm_count(), vectors = a.V / Elem<E>::kN;
  const long long bytes = (long long)a.V * (long long)sizeof(E);
  int threads = bytes <= 20000 ? 32 : bytes <= (a.k <= 32 ? 120000 : 60000) ? 64 : bytes <= 300000 ? 128 : 256;
  while (threads < a.k && threads < 256) threads *= 2;
  if (threads == 64 && a.k > 40 && vectors >= 64 && vectors < 5 * a.k) threads = 128;
  const long long rows = (bytes >= 32768 ? 2LL : 4LL) * a.T;
  while (threads < 256 && rows < (long long)kResident / threads * sms && bytes >= (threads < 128 ? 32 * threads : 16000)) threads *= 2;
  if (threads == 256 && a.T <= sms && bytes >= 100000) threads = 512;
  if (threads == 32) return launch<E, 32>(a, s);
  if (threads == 64) return launch<E, 64>(a, s);
  if (threads == 128) return launch<E, 128>(a, s);
  if (threads == 256) return launch<E, 256>(a, s);
  return launch<E, 512>(a, s);
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
  if (k < 1 || k > V || !temperature_ok(temperature)) return LORA_ERR_INVALID_ARG;
  if (k > LORA_TOPK_MAX || V > kMostEntries) return LORA_ERR_UNSUPPORTED;
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
  return dtype == LORA_LOGITS_BF16 ? launch_for<uint16_t>(a, (cudaStream_t)stream) : launch_for<float>(a, (cudaStream_t)stream);
}
