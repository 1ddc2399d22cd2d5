// The products of an 8-bit base (lora_f8.h): y = x W0^T and dx = dy W0 with a scale
// for each row's group of 128 of the one and for each 128 x 128 block of the other.
//
//     y[t, n] = sum_g xs[t, g] ws[n / 128, g] (sum over the 128 k of group g of xc[t, k] wc[n, k])
//
// The inner sums are tcgen05.mma.kind::f8f6f4 (four of K = 32) into tensor memory;
// between groups the scales change, so each group's sums are read back and added, times
// the product of the two scales, to fp32 sums in registers ("promotion").  Two
// accumulators in tensor memory alternate, so the next group's MMAs run meanwhile.
// dx = dy W0 sums over W0's rows: the same kernels with the operand from W0 MN-major,
// taken as it lies.  Ends inside a tile are the tensor maps' zero fill.
//
// Three forms:
//  - wide: 256 tokens x 256 outputs by a pair of CTAs that share their MMAs
//    (cta_group::2), tokens down the tile, so a thread's row has one factor a group and a
//    block of weights (a promotion is one FMA an element).  Each CTA holds half of the
//    tokens and half of the weights, and all the outputs of its tokens.  (With an MMA a
//    CTA, 128 x 256, each also reads the other half of the weights: 96 bytes a clock of
//    operands and as many of copies pass the shared memory's 128.)
//  - mid: 128 x 128 by a CTA, tokens down the tile, where wide tiles would leave SMs idle.
//  - split: few tokens.  128 outputs down the tile (so that every thread of a warpgroup has
//    work) and 16 to 64 tokens across.
// In the latter two a cluster of up to eight CTAs shares the sum over k and adds its parts
// up in rank order through distributed shared memory.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>

#include "internal.h"
#include "lora_f8.h"
#include "pairs.cuh"
#include "tc.cuh"

namespace lora {

namespace {

constexpr int kG = LORA_F8_BLOCK;

struct GemmArgs {
  CUtensorMap xmap;  // [T, inner], boxes of 128 columns
  CUtensorMap wmap;  // [N, K], boxes of 128 columns
  const float* xs;
  const float* ws;
  long long xs_t, xs_g;  // of a token, of a group
  long long ws_o, ws_g;  // of a block of outputs, of a group
  void* y;
  long long ldy;
  uint32_t idesc;
  int f32, wide_store;  // output type; rows of y on 16-byte boundaries
  int T, outer, nk;     // nk: groups of 128 of the sum
  int n_o, n_pairs;     // wide: tiles of outputs; pairs of tiles
  int32_t* err;
  long long probe;
};

// Every thread of a block learns whether the timeout probe's wait ran out.
__device__ __forceinline__ bool probe_passes(const GemmArgs& a) {
  if (a.probe <= 0) return true;
  __shared__ uint64_t probe_bar;
  __shared__ int probe_ok;
  if (threadIdx.x == 0) probe_ok = wait_probe(&probe_bar, a.probe) ? 1 : 0;
  __syncthreads();
  return probe_ok != 0;
}

// Sixteen bytes of outputs from fp32 values, one rounding each.
template <typename O>
__device__ __forceinline__ uint4 pack_out(const float* f);
template <>
__device__ __forceinline__ uint4 pack_out<uint16_t>(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
template <>
__device__ __forceinline__ uint4 pack_out<float>(const float* f) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// One lane of a warp, the same one each time.  Around an MMA inside code that the whole
// warp runs, it leaves addresses and descriptors in uniform registers, where MMAs want
// them: an issuing loop under `lane == 0` took about 700 cycles a group.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// A place in a ring of barriers and the parity of its turn.
template <int kN>
struct Turn {
  uint32_t at = 0, parity = 0;
  __device__ __forceinline__ void next() {
    if (++at == kN) {
      at = 0;
      parity ^= 1;
    }
  }
};

// The four MMAs of one group: descriptors step 32 bytes along a K-major operand, 32
// rows of 128 bytes along an MN-major one (which is one swizzle atom of 128 wide).
template <bool kPair, bool kAMn, bool kBMn>
__device__ __forceinline__ void group_mma(uint32_t d, uint32_t as, uint32_t bs, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < kG / 32; ++kk) {
    const uint64_t ad = kAMn ? sdesc_sw128(as + 4096 * kk, 0, 1024) : sdesc_sw128(as + 32 * kk, 16, 1024);
    const uint64_t bd = kBMn ? sdesc_sw128(bs + 4096 * kk, 0, 1024) : sdesc_sw128(bs + 32 * kk, 16, 1024);
    if (kPair) mma_f8_pair(d, ad, bd, idesc, kk != 0);
    else mma_f8(d, ad, bd, idesc, kk != 0);
  }
}

// Arrive on a barrier of a CTA of the cluster; nothing written is passed on with it.  The wide
// product's promoting warps free an accumulator so: their tcgen05.ld have completed (wait::ld, the
// sums are in registers) before tcgen05.fence::before_thread_sync, which orders them before the
// arrive, and the issuing warp has its after_thread_sync between its wait and the MMAs that write the
// columns again.  Nothing in memory goes with it, and a release would cost: with release and acquire
// between the two CTAs the product took 2.5 times as long.
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Wait (bounded) for the copies of the last `issued` stages that may be under way.
__device__ __forceinline__ void drain(uint64_t* full, uint32_t issued, int stages) {
  for (uint32_t g = issued > (uint32_t)stages ? issued - stages : 0; g < issued; ++g)
    mbar_wait(smem_u32(&full[g % stages]), (g / stages) & 1);
}

// --------------------------------------------------------------------- wide --

constexpr int kWM = 128, kWN = 256, kWStages = 6;
constexpr int kWEpiWarps = 8;
constexpr int kWThreads = 128 + 32 * kWEpiWarps;  // warp 0 copies, warp 1 issues MMAs, warps 4-11 promote
// Registers: 384 threads are launched with 168 each; the first warpgroup gives up 128 x 128
// of them, which the promoting ones' 128 sums a thread take (64 x 256): 64512 in all, as launched.
#define LORA_FEWER_REGISTERS() asm volatile("setmaxnreg.dec.sync.aligned.u32 40;" ::: "memory")
#define LORA_MORE_REGISTERS() asm volatile("setmaxnreg.inc.sync.aligned.u32 232;" ::: "memory")
constexpr int kWABytes = kWM * kG, kWStageBytes = kWABytes + kWN / 2 * kG;
constexpr size_t kWOffOut = (size_t)kWStages * kWStageBytes;  // a promoting warp's 32 rows of 128 bytes
constexpr size_t kWOffBars = kWOffOut + (size_t)kWEpiWarps * 4096;
constexpr size_t kWSmem = kWOffBars + (2 * kWStages + 5) * 8 + 16 + 1024;
static_assert(kWSmem <= 232448, "shared memory of one CTA");

// 32 rows x 128 bytes of a tile's outputs (this lane's row in v, 8 pieces of 16 bytes)
// through shared memory, so that a store covers whole lines.
template <typename O>
__device__ __forceinline__ void store_rows(const GemmArgs& a, uint8_t* st, const uint4 (&v)[8], int t0, int n0, int lane) {
  constexpr int kPer = 16 / sizeof(O);  // outputs of a piece
#pragma unroll
  for (int q = 0; q < 8; ++q) *reinterpret_cast<uint4*>(st + lane * 128 + ((q ^ (lane & 7)) << 4)) = v[q];
  __syncwarp();
  O* const y = static_cast<O*>(a.y);
  const int piece = lane & 7, n = n0 + piece * kPer;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3), t = t0 + r;
    if (t >= a.T || n >= a.outer) continue;
    const uint4 u = *reinterpret_cast<const uint4*>(st + r * 128 + ((piece ^ (r & 7)) << 4));
    O* const dst = y + (long long)t * a.ldy + n;
    if (a.wide_store && n + kPer <= a.outer) {
      *reinterpret_cast<uint4*>(dst) = u;
    } else {
      const O* e = reinterpret_cast<const O*>(&u);
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (n + j < a.outer) dst[j] = e[j];
    }
  }
  __syncwarp();
}

// Pair p of tiles: bands of kBand x 256 tokens, in a band outputs outermost, so that what
// runs at once is near square: 76 pairs of 256 x 256 read 8 x 256 rows of x and ten tiles of
// weights instead of all the weights.
constexpr int kBand = 8;
struct Tile {
  int m, o;  // in tiles of 2 kWM and kWN
};
__device__ __forceinline__ Tile tile_of(const GemmArgs& a, int p) {
  const int band = p / (kBand * a.n_o), in = p - band * kBand * a.n_o;
  const int rows = min(kBand, a.n_pairs / a.n_o - band * kBand);
  return Tile{band * kBand + in % rows, in / rows};
}

template <bool kBack>
__global__ void __launch_bounds__(kWThreads, 1) f8_wide_kernel(const __grid_constant__ GemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + kWOffBars);  // [stages] of the first CTA: both CTAs' copied bytes
  uint64_t* empty = full + kWStages;                             // [stages] MMA commit
  uint64_t* acc_full = empty + kWStages;                         // [2] MMA commit: a group's sums are complete
  uint64_t* acc_empty = acc_full + 2;                            // [2] of the first CTA: both CTAs' promoting warps have them
  uint64_t* mma_done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t crank = cluster_ctarank(), cid = cluster_id_x(), ncl = ncluster_x();
  if (tid == 0) {
    for (int s = 0; s < kWStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&acc_full[b]), 1);
      mbar_init(smem_u32(&acc_empty[b]), 2 * kWEpiWarps);
    }
    mbar_init(smem_u32(mma_done), 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(tmem_slot), 2 * kWN);
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers are there before the peer's copies and commits
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait_then_release();
  bool ok = probe_passes(a);
  if (warp < 4) {
    LORA_FEWER_REGISTERS();
    if (warp == 0 && lane == 0 && ok) {
      prefetch_tensormap(&a.xmap);
      prefetch_tensormap(&a.wmap);
      uint32_t g = 0;
      for (int p = (int)cid; p < a.n_pairs && ok; p += (int)ncl) {
        const Tile tile = tile_of(a, p);
        const int t0 = (2 * tile.m + (int)crank) * kWM, o0 = tile.o * kWN + (int)crank * kG;
        for (int kb = 0; kb < a.nk; ++kb, ++g) {
          const uint32_t st = g % kWStages;
          if (g >= kWStages && !mbar_wait(smem_u32(&empty[st]), ((g / kWStages) - 1) & 1)) {
            ok = false;
            break;
          }
          // this CTA's tokens and its half of the weights, counted by the first CTA, which
          // issues the MMAs (the other's bytes may come before it expects them)
          const uint32_t dst = smem_u32(sm + (size_t)st * kWStageBytes), bar = mapa(smem_u32(&full[st]), 0);
          if (crank == 0) mbar_arrive_expect_tx(smem_u32(&full[st]), 2 * kWStageBytes);
          tma_load_2d_pair(dst, &a.xmap, kb * kG, t0, bar);
          tma_load_2d_pair(dst + kWABytes, &a.wmap, kBack ? o0 : kb * kG, kBack ? kb * kG : o0, bar);
        }
      }
      // the last stages' commits have reached this CTA (so its copies have been read), or,
      // where a wait ran out, the copies under way have landed
      for (uint32_t i = g > kWStages ? g - kWStages : 0; i < g && ok; ++i) ok = mbar_wait(smem_u32(&empty[i % kWStages]), (i / kWStages) & 1);
      if (!ok) {
        report(a.err, LORA_DERR_TIMEOUT);
        if (crank == 0) drain(full, g, kWStages);
      }
    }
    if (warp == 1 && ok && crank == 0) {
      Turn<kWStages> st;
      Turn<2> ab;
      bool issued = false;
      const uint32_t stages = smem_u32(sm), fulls = smem_u32(full), empties = smem_u32(empty), accs = smem_u32(acc_full),
                     freed = smem_u32(acc_empty);
      for (int p = (int)cid; p < a.n_pairs && ok; p += (int)ncl) {
        for (int kb = 0; kb < a.nk; ++kb) {
          // (a barrier's first turn: the parity before it counts as complete)
          if (__any_sync(0xffffffffu, !mbar_wait(freed + 8 * ab.at, ab.parity ^ 1) || !mbar_wait(fulls + 8 * st.at, st.parity))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t as = stages + st.at * kWStageBytes;
          if (elected()) {
            group_mma<true, false, kBack>(tmem + ab.at * kWN, as, as + kWABytes, a.idesc);
            mma_commit_pair(accs + 8 * ab.at);
            mma_commit_pair(empties + 8 * st.at);
          }
          issued = true;
          st.next();
          ab.next();
        }
      }
      if (issued) {  // every MMA has completed before tensor memory is freed
        if (elected()) mma_commit_pair(smem_u32(mma_done), 1);
        mbar_wait(smem_u32(mma_done), 0);
      }
      if (!ok && lane == 0) report(a.err, LORA_DERR_TIMEOUT);
    }
    __syncwarp();
  } else {
    LORA_MORE_REGISTERS();
    const int quarter = warp & 3, half = (warp - 4) >> 2;  // tensor-memory lanes; the block of outputs
    uint8_t* const out = sm + kWOffOut + (size_t)(warp - 4) * 4096;
    uint32_t g = 0;
    for (int p = (int)cid; p < a.n_pairs && ok; p += (int)ncl) {
      const Tile tile = tile_of(a, p);
      const int t0 = (2 * tile.m + (int)crank) * kWM + quarter * 32, t = t0 + lane;
      const int n0 = tile.o * kWN + half * kG;
      const bool row_on = t < a.T, col_on = n0 < a.outer;
      const float* const xs = a.xs + (row_on ? t * a.xs_t : 0);
      const float* const ws = a.ws + (col_on ? n0 / kG * a.ws_o : 0);
      // the factors of the coming groups, two ahead
      float x1 = xs[0], w1 = ws[0], x2 = 0.f, w2 = 0.f;
      if (a.nk > 1) {
        x2 = xs[a.xs_g];
        w2 = ws[a.ws_g];
      }
      uint64_t acc[kG / 2];
#pragma unroll
      for (int i = 0; i < kG / 2; ++i) acc[i] = 0;
      for (int kb = 0; kb < a.nk; ++kb, ++g) {
        const float f = x1 * w1;
        x1 = x2;
        w1 = w2;
        if (kb + 2 < a.nk) {
          x2 = xs[(kb + 2) * a.xs_g];
          w2 = ws[(kb + 2) * a.ws_g];
        }
        const uint32_t ab = g & 1;
        if (__any_sync(0xffffffffu, !mbar_wait(smem_u32(&acc_full[ab]), (g >> 1) & 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t f2 = pair_of(f, f);
#pragma unroll
        for (int c = 0; c < kG / 32; ++c) {
          uint32_t r[32];
          tmem_ld32_nowait(tmem + ab * kWN + half * kG + c * 32 + ((uint32_t)(quarter * 32) << 16), r);
          tmem_wait_ld32(r);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            acc[c * 16 + i] = fma2(pair_of(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), f2, acc[c * 16 + i]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(mapa(smem_u32(&acc_empty[ab]), 0));
      }
      if (!ok) break;
      const int per = a.f32 ? 32 : 64;  // outputs of 128 bytes
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (a.f32) {
          uint4 v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float e[4];
            split(acc[c * 16 + 2 * q], e[0], e[1]);
            split(acc[c * 16 + 2 * q + 1], e[2], e[3]);
            v[q] = pack_out<float>(e);
          }
          if (n0 + c * per < a.outer) store_rows<float>(a, out, v, t0, n0 + c * per, lane);
        } else if (c < 2) {
          uint4 v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float e[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) split(acc[c * 32 + 4 * q + j], e[2 * j], e[2 * j + 1]);
            v[q] = pack_out<uint16_t>(e);
          }
          if (n0 + c * per < a.outer) store_rows<uint16_t>(a, out, v, t0, n0 + c * per, lane);
        }
      }
    }
    if (!ok && lane == 0) report(a.err, LORA_DERR_TIMEOUT);
  }
  tc_fence_before();
  cluster_sync();  // neither CTA leaves while the peer may still copy into it or arrive on its barriers
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 2 * kWN);
  }
}

// ------------------------------------------------------ a sum shared by a cluster --

constexpr int kSMaxSplit = 8;

// Where output o of a tile's token j is in its part of the sum: rows of 128, 16-byte
// pieces shuffled so that neither a token's nor an output's lanes meet in a bank.
__device__ __forceinline__ int part_at(int j, int o) { return j * kG + (((o >> 2) ^ (j & 7)) << 2) + (o & 3); }

__device__ __forceinline__ float4 ld_dsmem_v4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}

// The parts (of tokens t0 .. t0 + rows and outputs o0 .. o0 + 127, at `part` in each CTA)
// added up in rank order, by all threads: a warp a token, four outputs a lane.
template <int kThreads>
__device__ __forceinline__ void join_parts(const GemmArgs& a, const float* part, const int* failed, int n, int rank, int t0, int o0,
                                           int rows) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool whole = true;
#pragma unroll
  for (int q = 0; q < kSMaxSplit; ++q) {
    uint32_t bad = 0;
    if (q < n) asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(bad) : "r"(mapa(smem_u32(failed), q)) : "memory");
    whole = whole && bad == 0;
  }
  const int o = o0 + 4 * lane;
  if (!whole || o >= a.outer) return;
  for (int j = rank + n * warp; j < rows && t0 + j < a.T; j += n * (kThreads / 32)) {
    const uint32_t at = smem_u32(part + part_at(j, 4 * lane));
    float4 p[kSMaxSplit];
#pragma unroll
    for (int q = 0; q < kSMaxSplit; ++q)
      if (q < n) p[q] = ld_dsmem_v4(mapa(at, q));
    float e[4] = {p[0].x, p[0].y, p[0].z, p[0].w};
#pragma unroll
    for (int q = 1; q < kSMaxSplit; ++q)
      if (q < n) {
        e[0] += p[q].x;
        e[1] += p[q].y;
        e[2] += p[q].z;
        e[3] += p[q].w;
      }
    const long long dst = (long long)(t0 + j) * a.ldy + o;
    const bool whole4 = a.wide_store && o + 4 <= a.outer;
    if (a.f32) {
      float* const y = static_cast<float*>(a.y) + dst;
      if (whole4) *reinterpret_cast<float4*>(y) = make_float4(e[0], e[1], e[2], e[3]);
      else
        for (int i = 0; i < 4 && o + i < a.outer; ++i) y[i] = e[i];
    } else {
      uint16_t* const y = static_cast<uint16_t*>(a.y) + dst;
      if (whole4) *reinterpret_cast<uint2*>(y) = make_uint2(pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]));
      else
        for (int i = 0; i < 4 && o + i < a.outer; ++i) y[i] = __bfloat16_as_ushort(__float2bfloat16_rn(e[i]));
    }
  }
}

// A producer's loop over groups k0 .. k1 - 1 (one thread): per stage a box of weights and
// a box of tokens.
template <bool kBack, int kStages>
__device__ __forceinline__ bool copy_groups(const GemmArgs& a, uint8_t* sm, uint64_t* full, uint64_t* empty, int stage_bytes, int k0,
                                            int k1, int t0, int o0) {
  Turn<kStages> st;
  uint32_t g = 0;
  bool ok = true;
  for (int kb = k0; kb < k1 && ok; ++kb, ++g) {
    ok = mbar_wait(smem_u32(&empty[st.at]), st.parity ^ 1);
    if (!ok) break;
    const uint32_t dst = smem_u32(sm) + st.at * stage_bytes, bar = smem_u32(&full[st.at]);
    mbar_arrive_expect_tx(bar, stage_bytes);
    tma_load_2d(dst, &a.wmap, kBack ? o0 : kb * kG, kBack ? kb * kG : o0, bar);
    tma_load_2d(dst + kG * kG, &a.xmap, kb * kG, t0, bar);
    st.next();
  }
  drain(full, g, kStages);
  return ok;
}

// The MMAs of those groups (a whole warp): weights down the tile (kSwap) or tokens, kCols
// columns an accumulator.
template <bool kSwap, bool kBack, int kStages, int kAcc, int kCols>
__device__ __forceinline__ bool issue_groups(const GemmArgs& a, uint8_t* sm, uint64_t* full, uint64_t* empty, uint64_t* acc_full,
                                             uint64_t* acc_empty, uint64_t* mma_done, int stage_bytes, int k0, int k1, uint32_t tmem) {
  Turn<kStages> st;
  Turn<kAcc> ab;
  bool ok = true;
  const uint32_t stages = smem_u32(sm), fulls = smem_u32(full), empties = smem_u32(empty), accs = smem_u32(acc_full),
                 freed = smem_u32(acc_empty);
  for (int kb = k0; kb < k1; ++kb) {
    if (__any_sync(0xffffffffu, !mbar_wait(freed + 8 * ab.at, ab.parity ^ 1) || !mbar_wait(fulls + 8 * st.at, st.parity))) {
      ok = false;
      break;
    }
    tc_fence_after();
    const uint32_t ws = stages + st.at * stage_bytes, xs = ws + kG * kG;
    if (elected()) {
      if (kSwap) group_mma<false, kBack, false>(tmem + ab.at * kCols, ws, xs, a.idesc);
      else group_mma<false, false, kBack>(tmem + ab.at * kCols, xs, ws, a.idesc);
      mma_commit(accs + 8 * ab.at);
      mma_commit(empties + 8 * st.at);
    }
    st.next();
    ab.next();
  }
  if (elected()) mma_commit(smem_u32(mma_done));  // every MMA has completed before tensor memory is freed
  mbar_wait(smem_u32(mma_done), 0);
  return ok;
}

// ---------------------------------------------------------------------- mid --

constexpr int kMStages = 6, kMAcc = 4, kMEpiWarps = 8, kMCols = 64;
constexpr int kMThreads = 64 + 32 * kMEpiWarps;  // warp 0 copies, warp 1 issues MMAs, the others promote
constexpr int kMStageBytes = 2 * kG * kG;
constexpr size_t kMOffBars = (size_t)kMStages * kMStageBytes;
constexpr size_t kMSmem = kMOffBars + (2 * kMStages + 2 * kMAcc + 1) * 8 + 16 + 1024;

template <bool kBack>
__global__ void __launch_bounds__(kMThreads, 1) f8_mid_kernel(const __grid_constant__ GemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ int failed;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + kMOffBars);  // [stages] copied bytes
  uint64_t* empty = full + kMStages;                             // [stages] MMA commit
  uint64_t* acc_full = empty + kMStages;                         // [kMAcc] MMA commit: a group's sums are complete
  uint64_t* acc_empty = acc_full + kMAcc;                        // [kMAcc] the promoting warps have them
  uint64_t* mma_done = acc_empty + kMAcc;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  const int tile = (int)cluster_id_x(), o0 = tile % a.n_o * kG, t0 = tile / a.n_o * kG;
  // this CTA's groups of the sum
  const int k0 = (int)((long long)a.nk * rank / n), k1 = (int)((long long)a.nk * (rank + 1) / n);
  if (tid == 0) {
    prefetch_tensormap(&a.wmap);
    prefetch_tensormap(&a.xmap);
    for (int s = 0; s < kMStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < kMAcc; ++b) {
      mbar_init(smem_u32(&acc_full[b]), 1);
      mbar_init(smem_u32(&acc_empty[b]), kMEpiWarps);
    }
    mbar_init(smem_u32(mma_done), 1);
    failed = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), kMAcc * kG);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait_then_release();
  bool ok = probe_passes(a);
  if (warp == 0) {
    if (lane == 0 && ok) ok = copy_groups<kBack, kMStages>(a, sm, full, empty, kMStageBytes, k0, k1, t0, o0);
    if (!ok && lane == 0) report(a.err, LORA_DERR_TIMEOUT);
    __syncwarp();
  } else if (warp == 1) {
    if (ok) ok = issue_groups<false, kBack, kMStages, kMAcc, kG>(a, sm, full, empty, acc_full, acc_empty, mma_done, kMStageBytes, k0, k1, tmem);
    if (!ok && lane == 0) report(a.err, LORA_DERR_TIMEOUT);
    __syncwarp();
  } else {
    const int quarter = warp & 3, c0 = (warp - 2) / 4 * kMCols;  // tensor-memory lanes; first of 64 columns
    const int row = quarter * 32 + lane, t = t0 + row;
    const bool rows_on = t0 + quarter * 32 < a.T;  // some token of this warp's is there
    const float* const xs = a.xs + (t < a.T ? t * a.xs_t : 0);
    const float* const ws = a.ws + o0 / kG * a.ws_o;
    float x1 = xs[k0 * a.xs_g], w1 = ws[k0 * a.ws_g], x2 = 0.f, w2 = 0.f;  // two groups ahead
    if (k0 + 1 < k1) {
      x2 = xs[(k0 + 1) * a.xs_g];
      w2 = ws[(k0 + 1) * a.ws_g];
    }
    uint64_t acc[kMCols / 2];
#pragma unroll
    for (int i = 0; i < kMCols / 2; ++i) acc[i] = 0;
    Turn<kMAcc> ab;
    for (int kb = k0; kb < k1 && ok; ++kb) {
      const float f = x1 * w1;
      x1 = x2;
      w1 = w2;
      if (kb + 2 < k1) {
        x2 = xs[(kb + 2) * a.xs_g];
        w2 = ws[(kb + 2) * a.ws_g];
      }
      ok = !__any_sync(0xffffffffu, !mbar_wait(smem_u32(&acc_full[ab.at]), ab.parity));
      if (!ok) break;
      tc_fence_after();
      const uint64_t f2 = pair_of(f, f);
      const uint32_t at = tmem + ab.at * kG + c0 + ((uint32_t)(quarter * 32) << 16);
#pragma unroll
      for (int c = 0; c < kMCols / 32; ++c) {
        uint32_t r[32];
        if (rows_on) {
          tmem_ld32_nowait(at + c * 32, r);
          tmem_wait_ld32(r);
        }
        if (c == kMCols / 32 - 1) {  // these columns may be written again
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&acc_empty[ab.at]));
        }
        if (rows_on) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            acc[c * 16 + i] = fma2(pair_of(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), f2, acc[c * 16 + i]);
        }
      }
      ab.next();
    }
    if (!ok) {
      if (lane == 0) {
        report(a.err, LORA_DERR_TIMEOUT);
        failed = 1;
      }
    } else if (rows_on) {
      // this CTA's part of the sum where the stages were (their copies and MMAs are over:
      // the last group's sums are complete)
      float* const part = reinterpret_cast<float*>(sm);
#pragma unroll
      for (int i = 0; i < kMCols / 4; ++i) {
        float4 v;
        split(acc[2 * i], v.x, v.y);
        split(acc[2 * i + 1], v.z, v.w);
        *reinterpret_cast<float4*>(part + part_at(row, c0 + 4 * i)) = v;
      }
    }
  }
  tc_fence_before();
  if (n > 1) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kMAcc * kG);
  }
  join_parts<kMThreads>(a, reinterpret_cast<const float*>(sm), &failed, n, rank, t0, o0, kG);
  if (n > 1) cluster_sync();  // no CTA leaves while its part may be read
}

// -------------------------------------------------------------------- split --

template <int kNT>
struct Split {
  static constexpr int kStages = kNT == 16 ? 6 : kNT == 32 ? 5 : 4;
  static constexpr int kAcc = kNT <= 32 ? 8 : 4;  // accumulators: groups on their way to the sums
  static constexpr int kWarps = 4;                // promoting warps
  static constexpr int kThreads = 64 + 32 * kWarps;  // warp 0 copies, warp 1 issues MMAs
  static constexpr int kTable = 32;                  // groups whose factors are worked out at once
  static constexpr int kStageBytes = kG * kG + kNT * kG;
  static constexpr size_t kOffF = (size_t)kStages * kStageBytes;  // [kTable][kNT] factors
  static constexpr size_t kOffBars = kOffF + kTable * kNT * sizeof(float);
  static constexpr size_t kSmem = kOffBars + (2 * kStages + 2 * kAcc + 1) * 8 + 16 + 1024;
  static_assert((size_t)kStages * kStageBytes >= (size_t)kNT * kG * 4, "the parts of the sum take the stages' place");
  static_assert(2 * (kSmem + 1024) <= 233472, "two CTAs an SM");
};

// A barrier of the promoting threads.
template <int kThreads>
__device__ __forceinline__ void promoting_bar() {
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
}

template <int kNT, bool kBack>
__global__ void __launch_bounds__(Split<kNT>::kThreads, 2) f8_split_kernel(const __grid_constant__ GemmArgs a) {
  using S = Split<kNT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int failed;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  float* table = reinterpret_cast<float*>(sm + S::kOffF);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + S::kOffBars);  // [stages] copied bytes
  uint64_t* empty = full + S::kStages;                             // [stages] MMA commit
  uint64_t* acc_full = empty + S::kStages;                         // [kAcc] MMA commit: a group's sums are complete
  uint64_t* acc_empty = acc_full + S::kAcc;                        // [kAcc] the promoting warps have them
  uint64_t* mma_done = acc_empty + S::kAcc;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  const int tile = (int)cluster_id_x(), o0 = tile % a.n_o * kG, t0 = tile / a.n_o * kNT;
  // this CTA's groups of the sum
  const int k0 = (int)((long long)a.nk * rank / n), k1 = (int)((long long)a.nk * (rank + 1) / n);
  if (tid == 0) {
    prefetch_tensormap(&a.wmap);
    prefetch_tensormap(&a.xmap);
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < S::kAcc; ++b) {
      mbar_init(smem_u32(&acc_full[b]), 1);
      mbar_init(smem_u32(&acc_empty[b]), S::kWarps);
    }
    mbar_init(smem_u32(mma_done), 1);
    failed = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), S::kAcc * kNT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait_then_release();
  bool ok = probe_passes(a);
  if (warp == 0) {
    if (lane == 0 && ok) ok = copy_groups<kBack, S::kStages>(a, sm, full, empty, S::kStageBytes, k0, k1, t0, o0);
    if (!ok && lane == 0) report(a.err, LORA_DERR_TIMEOUT);
    __syncwarp();
  } else if (warp == 1) {
    if (ok) ok = issue_groups<true, kBack, S::kStages, S::kAcc, kNT>(a, sm, full, empty, acc_full, acc_empty, mma_done, S::kStageBytes, k0, k1, tmem);
    if (!ok && lane == 0) report(a.err, LORA_DERR_TIMEOUT);
    __syncwarp();
  } else {
    constexpr int kThreads = 32 * S::kWarps, kStep = kNT < 32 ? kNT : 32;
    const int id = tid - 64, quarter = warp & 3;  // tensor-memory lanes
    const float* const ws = a.ws + o0 / kG * a.ws_o;
    uint64_t acc[kNT / 2];
#pragma unroll
    for (int i = 0; i < kNT / 2; ++i) acc[i] = 0;
    // A warp whose wait ran out goes on through the barriers without waiting or reading.
    uint32_t g = 0;
    for (int kc = k0; kc < k1; kc += S::kTable) {
      const int groups = min(S::kTable, k1 - kc);
      if (kc > k0) promoting_bar<kThreads>();  // everyone is done with the factors before
      for (int i = id; i < groups * kNT; i += kThreads) {
        const int kb = kc + i / kNT, t = t0 + i % kNT;
        table[i] = t < a.T ? a.xs[t * a.xs_t + kb * a.xs_g] * ws[kb * a.ws_g] : 0.f;
      }
      promoting_bar<kThreads>();
      for (int j = 0; j < groups; ++j, ++g) {
        const uint32_t ab = g % S::kAcc;
        if (ok) ok = !__any_sync(0xffffffffu, !mbar_wait(smem_u32(&acc_full[ab]), (g / S::kAcc) & 1));
        if (!ok) continue;
        tc_fence_after();
        const float* const f = table + j * kNT;
#pragma unroll
        for (int c = 0; c < kNT / kStep; ++c) {
          uint32_t r[kStep];
          const uint32_t at = tmem + ab * kNT + c * kStep + ((uint32_t)(quarter * 32) << 16);
          if constexpr (kStep == 32) {
            tmem_ld32_nowait(at, r);
            tmem_wait_ld32(r);
          } else {
            tmem_ld16(at, reinterpret_cast<float*>(r));
          }
          if (c == kNT / kStep - 1) {  // these columns may be written again
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&acc_empty[ab]));
          }
#pragma unroll
          for (int i = 0; i < kStep / 4; ++i) {
            const float4 p = *reinterpret_cast<const float4*>(f + c * kStep + 4 * i);
            uint64_t* const s = acc + c * (kStep / 2) + 2 * i;
            s[0] = fma2(pair_of(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1])), pair_of(p.x, p.y), s[0]);
            s[1] = fma2(pair_of(__uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])), pair_of(p.z, p.w), s[1]);
          }
        }
      }
    }
    if (!ok) {
      if (lane == 0) {
        report(a.err, LORA_DERR_TIMEOUT);
        failed = 1;
      }
    } else {
      // this CTA's part of the sum, a token's outputs side by side, where the stages
      // were (their copies and MMAs are over: the last group's sums are complete)
      float* const part = reinterpret_cast<float*>(sm);
      const int o = quarter * 32 + lane;
#pragma unroll
      for (int i = 0; i < kNT / 2; ++i) {
        float u, v;
        split(acc[i], u, v);
        part[part_at(2 * i, o)] = u;
        part[part_at(2 * i + 1, o)] = v;
      }
    }
  }
  tc_fence_before();
  if (n > 1) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kAcc * kNT);
  }
  join_parts<S::kThreads>(a, reinterpret_cast<const float*>(sm), &failed, n, rank, t0, o0, kNT);
  if (n > 1) cluster_sync();  // no CTA leaves while its part may be read
}

// CTAs that share a tile's sum: up to `places` of them in all.
int splits_of(long long tiles, int nk, int places) {
  int splits = 1;
  while (splits < kSMaxSplit && tiles * splits * 2 <= places && nk >= 2 * splits) splits *= 2;
  return splits;
}

template <int kNT>
lora_status_t launch_split(GemmArgs* a, int back, int splits, long long tiles, cudaStream_t s) {
  const void* f = back ? (const void*)f8_split_kernel<kNT, true> : (const void*)f8_split_kernel<kNT, false>;
  if (ensure_smem_attr(f, Split<kNT>::kSmem) != cudaSuccess) return LORA_ERR_CUDA;
  if (tiles * splits > 0x7fffffffLL) return LORA_ERR_UNSUPPORTED;
  return launch_pdl(f, dim3((unsigned)(tiles * splits)), dim3(Split<kNT>::kThreads), Split<kNT>::kSmem, s, splits, a) == cudaSuccess
             ? LORA_OK
             : LORA_ERR_CUDA;
}

}  // namespace

lora_status_t launch_f8_product(const lora_f8_matrix_t* x, const lora_f8_matrix_t* w, void* y, long long ldy, int f32, int back,
                                int32_t* err, cudaStream_t s) {
  GemmArgs a;
  memset(&a, 0, sizeof(a));
  const int inner = back ? w->rows : w->cols;
  a.T = x->rows;
  a.outer = back ? w->cols : w->rows;
  a.nk = (inner + kG - 1) / kG;
  a.xs = x->scales;
  a.xs_t = x->scale_row;
  a.xs_g = x->scale_col;
  a.ws = w->scales;
  a.ws_o = back ? w->scale_col : w->scale_row;
  a.ws_g = back ? w->scale_row : w->scale_col;
  a.y = y;
  a.ldy = ldy;
  a.f32 = f32;
  const int size = f32 ? 4 : 2;
  a.wide_store = reinterpret_cast<uintptr_t>(y) % 16 == 0 && ldy * size % 16 == 0;
  a.err = err;
  a.probe = wait_probe_cycles();
  const int n_o = (a.outer + kG - 1) / kG;
  const long long m128 = (a.T + kWM - 1) / kWM;
  const int sms = sm_count();
  const long long tiles128 = n_o * m128;
  // The form and the CTAs that share a sum (times in us on a GB300, 4096 x 4096 weights
  // unless said, calls back to back; mid and split each with the splits that rule gives):
  //  - wide once mid tiles fill more than half of the SMs, so that they would not share sums:
  //    384 tokens 18.2 (mid 19.1), 512 18.5 (19.6), 1024 19.2 (39.6); 128 tokens x 13824
  //    outputs 22.6 (23.8).  Below: 256 tokens 17.8 (mid 12.4), 128 18.1 (9.3).
  //  - split up to 64 tokens: 8 tokens 6.3 (mid 8.3), 32 6.9 (7.8), 64 8.5 (8.3); 64 tokens
  //    x 13824 outputs 20.5 (22.3).
  if (a.T > 64 && 2 * tiles128 > sms) {
    if (!make_byte_map(&a.xmap, x->codes, a.T, inner, x->ld, kWM)) return LORA_ERR_UNSUPPORTED;
    if (!make_byte_map(&a.wmap, w->codes, w->rows, w->cols, w->ld, kG)) return LORA_ERR_UNSUPPORTED;
    a.n_o = (n_o + 1) / 2;
    if ((m128 + 1) / 2 * a.n_o > 0x7fffffffLL) return LORA_ERR_UNSUPPORTED;
    a.n_pairs = (int)((m128 + 1) / 2 * a.n_o);
    a.idesc = idesc_f8(2 * kWM, kWN, x->type, w->type, 0, back);
    const void* f = back ? (const void*)f8_wide_kernel<true> : (const void*)f8_wide_kernel<false>;
    if (ensure_smem_attr(f, kWSmem) != cudaSuccess) return LORA_ERR_CUDA;
    const int clusters = std::min(a.n_pairs, std::max(1, max_active_clusters(f, kWThreads, kWSmem, 2)));
    return launch_pdl(f, dim3((unsigned)(2 * clusters)), dim3(kWThreads), kWSmem, s, 2, &a) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
  }
  a.n_o = n_o;
  if (a.T > 64) {
    if (!make_byte_map(&a.xmap, x->codes, a.T, inner, x->ld, kG)) return LORA_ERR_UNSUPPORTED;
    if (!make_byte_map(&a.wmap, w->codes, w->rows, w->cols, w->ld, kG)) return LORA_ERR_UNSUPPORTED;
    a.idesc = idesc_f8(kG, kG, x->type, w->type, 0, back);
    const int splits = splits_of(tiles128, a.nk, sms);
    const void* f = back ? (const void*)f8_mid_kernel<true> : (const void*)f8_mid_kernel<false>;
    if (ensure_smem_attr(f, kMSmem) != cudaSuccess) return LORA_ERR_CUDA;
    return launch_pdl(f, dim3((unsigned)(tiles128 * splits)), dim3(kMThreads), kMSmem, s, splits, &a) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
  }
  const int nt = a.T <= 16 ? 16 : a.T <= 32 ? 32 : 64;
  if (!make_byte_map(&a.xmap, x->codes, a.T, inner, x->ld, nt)) return LORA_ERR_UNSUPPORTED;
  if (!make_byte_map(&a.wmap, w->codes, w->rows, w->cols, w->ld, kG)) return LORA_ERR_UNSUPPORTED;
  a.idesc = idesc_f8(kG, nt, w->type, x->type, back, 0);
  const long long tiles = (long long)n_o * ((a.T + nt - 1) / nt);
  // Two of these CTAs fit an SM.  8 tokens, 32 tiles of 32 groups: four CTAs a sum 6.3, eight
  // 6.5, two 7.7; 40 tiles of 108: four 14.7, two 18.3, eight 19.9; 108 tiles of 40: two 14.4,
  // one 14.9, four 18.3.
  const int splits = splits_of(tiles, a.nk, sms * 3 / 2);
  if (nt == 16) return launch_split<16>(&a, back, splits, tiles, s);
  if (nt == 32) return launch_split<32>(&a, back, splits, tiles, s);
  return launch_split<64>(&a, back, splits, tiles, s);
}

}  // namespace lora
