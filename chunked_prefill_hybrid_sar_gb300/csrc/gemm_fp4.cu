// Product of two microscaled 4-bit matrices on the 5th-generation tensor cores.
//
// C = epilogue(alpha * A . W^T), A = token rows [M, K], W = weight rows [N, K],
// both e2m1 codes with block scales (fp4.cu).  kind::mxf4nvf4 / kind::mxf4 MMAs
// take K = 64 codes a row from shared memory and the scales from tensor memory
// and accumulate in fp32; the scales never meet the codes in a register.
//
// Two tilings put the weight rows on the MMA's M side, so that a batch of any
// number of tokens pads to 16: a split one for few tokens, bound by the weight's
// bytes and, below about 30 MB, by the latencies of a launch; and a pair one for
// many, bound by the tensor pipe and by what the SMs can fetch from L2.
// pick_variant() chooses.
//
// Issuing is what both had to be made fast at: a 256-code slab is 8 to 12 scale
// copies, 4 MMAs and a commit, and issued under a test of the lane's number it
// took 910 clocks, under elect 344, from uniform registers 207.
#include <cuda.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <string>

#include "common.cuh"
#include "internal.h"
#include "tc05.cuh"

namespace sar {

namespace {

constexpr int kSlab = 256;                 // codes of a row per pipeline stage: 128 bytes, one swizzle span
constexpr int kOpTile = 128 * 128;         // 128 rows of a slab
constexpr int kTileBytes = 512;            // one scale tile
constexpr int kSmemPerSm = 233472;         // 228 KB
constexpr int kSmemLimit = 232448;         // 227 KB
constexpr int kBarBytes = 256;
constexpr int kPairThreads = 320;
// The pair tiling asks L2 for the residual ahead of the tile's MMAs up to this many
// slabs.  With and without, in us: 8192 x 7168, K = 4096 141 and 157, 6144 148 and
// 163, 7168 (28 slabs) 161 and 166, 7680 170 and 167, 8192 179 and 169, 20480 361
// and 344; 8192 x 14336, K = 7168 304 and 314, 7680 324 and 319; 2048 x 4096 within
// 3% either way from 6144 on.
constexpr int kPrefetchSlabs = 28;
// Staging of one epilogue warp of the pair tiling: two boxes of 2 KB, or (SwiGLU)
// 16 tokens x 32 columns of fp32 from its partner and two boxes of 1 KB.
constexpr int kWarpOut = 4096;

template <bool NV>
struct Fmt {
  static constexpr int kTiles = NV ? 4 : 2;  // scale tiles of a row block in a slab (64 or 128 columns each)
  static constexpr int kScaleBytes = kTiles * kTileBytes;
};

struct Params {
  int M, N, K;
  int slabs;      // of 256 columns
  int tiles;      // scale tiles per row block
  int bn;         // token rows per tile
  int splits, slabs_per_split;
  int stages, stage_bytes, tmem_cols;
  const uint8_t* sa;
  const uint8_t* sw;
  void* c;
  const float* r;
  float alpha;
  // pair tiling
  int m_full, n_tiles, last_bn, group, units;
  int pair_ranges;  // K ranges of a tile, a pair each (the pairs of a cluster)
  int tma_out;    // c is written (or, where it is r, added to) through a tensor map
  int vec;        // rows of c (and r) can be written four columns at a time
  int* err;
};

// Work unit u of the pair tiling.  Whole token tiles come first, in groups of
// `group` token tiles that share a weight tile one after the other (the pairs
// running at one time then cover a block of tiles, and what they fetch meets in
// L2); the narrow last token tile of each weight tile comes last.
struct Tile {
  int mt, nt, bn;
};
__device__ __forceinline__ Tile tile_of(const Params& p, int u) {
  Tile t;
  const int n_full = p.m_full * p.n_tiles;
  if (u < n_full) {
    const int g = u / (p.group * p.n_tiles), m0 = g * p.group;
    const int gs = min(p.group, p.m_full - m0), r = u - m0 * p.n_tiles;
    t.nt = r / gs;
    t.mt = m0 + r - t.nt * gs;
    t.bn = 256;
  } else {
    t.nt = u - n_full;
    t.mt = p.m_full;
    t.bn = p.last_bn;
  }
  return t;
}

// The whole warp waits; all its lanes get the same answer.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int* err, int site) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, err, site)) != 0;
}

// Whether the phase has completed, without waiting.
__device__ __forceinline__ uint32_t mbar_done(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}

// A warp's walk over the stages of a ring.  The barrier is asked one slab ahead,
// before the slab's instructions are issued, so that its answer's latency (about
// 100 clocks of the 430 that a slab took to issue) runs under them.
// flip: 1 for the warp that fills (a fresh barrier counts as passed).
struct Ring {
  uint32_t bars, stages, flip, s = 0, ph = 0, peek = 0;
  __device__ __forceinline__ bool next(int* err, int site, uint32_t& stage) {
    if (!__all_sync(0xffffffffu, peek) && !warp_wait(bars + s * 8, ph ^ flip, err, site)) return false;
    stage = s;
    if (++s == stages) {
      s = 0;
      ph ^= 1u;
    }
    peek = mbar_done(bars + s * 8, ph ^ flip);
    return true;
  }
};

__device__ __forceinline__ void st_shared(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
template <typename T>
__device__ __forceinline__ void st_shared16(uint32_t addr, T v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(*reinterpret_cast<const unsigned short*>(&v)) : "memory");
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Writes four neighbouring results of row m from column n on.
template <typename T, int EPI>
__device__ __forceinline__ void put4(const Params& p, size_t m, int n, int ncols, const float (&x)[4]) {
  const size_t at = m * (size_t)ncols + n;
  if constexpr (EPI == SAR_EPI_F32 || EPI == SAR_EPI_RESIDUAL) {
    float* c = reinterpret_cast<float*>(p.c) + at;
    if (p.vec) {
      float4 v = make_float4(x[0], x[1], x[2], x[3]);
      if constexpr (EPI == SAR_EPI_RESIDUAL) {
        const float4 r = *reinterpret_cast<const float4*>(p.r + at);
        v = make_float4(v.x + r.x, v.y + r.y, v.z + r.z, v.w + r.w);
      }
      *reinterpret_cast<float4*>(c) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < ncols) c[i] = EPI == SAR_EPI_RESIDUAL ? x[i] + p.r[at + i] : x[i];
    }
  } else {
    T* c = reinterpret_cast<T*>(p.c) + at;
    if (p.vec) {
      *reinterpret_cast<uint2*>(c) = make_uint2(Elem<T>::pack(x[0], x[1]), Elem<T>::pack(x[2], x[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < ncols) c[i] = Elem<T>::from(x[i]);
    }
  }
}

// Adds up a tile's partials, [token][128 weight rows] of fp32 at `part` in the
// shared memory of `ranges` CTAs (range k in the cluster's CTA k * stride +
// offset), for this CTA's share of the tokens (every ranges-th from `range` on),
// in the ranges' order, and writes them through the epilogue.  kThreads threads, a
// quarter warp's worth of columns each; block: which 128 weight rows.
template <typename T, int EPI, int kThreads>
__device__ __forceinline__ void join(const Params& p, uint32_t part, int ranges, int range, int stride, int offset, int t,
                                     int block, int m0, int rows) {
  constexpr int kLanes = EPI == SAR_EPI_SWIGLU ? 16 : 32;  // four columns each
  constexpr int kU = 8;  // tokens read at a time, so that the latency is paid once for all of them
  const int n4 = (t % kLanes) * 4;
  const int step = (kThreads / kLanes) * ranges;
  auto joined = [&](int tok0, int n, float4 (&x)[kU]) {
#pragma unroll
    for (int u = 0; u < kU; ++u) x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < ranges; ++s) {
      const uint32_t at = cluster_addr(part, (uint32_t)(s * stride + offset)) + (uint32_t)n * 4;
      float4 v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u)
        v[u] = tok0 + u * step < rows ? ld_cluster_f4(at + (uint32_t)(tok0 + u * step) * 512) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        x[u].x += v[u].x;
        x[u].y += v[u].y;
        x[u].z += v[u].z;
        x[u].w += v[u].w;
      }
    }
  };
  for (int tok0 = (t / kLanes) * ranges + range; tok0 < rows; tok0 += kU * step) {
    float4 x[kU], y[kU];
    joined(tok0, n4, x);
    if constexpr (EPI == SAR_EPI_SWIGLU) joined(tok0, 64 + n4, y);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int tok = tok0 + u * step;
      if (tok >= rows) continue;
      float o[4] = {x[u].x * p.alpha, x[u].y * p.alpha, x[u].z * p.alpha, x[u].w * p.alpha};
      if constexpr (EPI == SAR_EPI_SWIGLU) {
        o[0] = silu(o[0]) * (y[u].x * p.alpha);
        o[1] = silu(o[1]) * (y[u].y * p.alpha);
        o[2] = silu(o[2]) * (y[u].z * p.alpha);
        o[3] = silu(o[3]) * (y[u].w * p.alpha);
        if (block * 64 + n4 < p.N >> 1) put4<T, EPI>(p, (size_t)(m0 + tok), block * 64 + n4, p.N >> 1, o);
      } else if (block * 128 + n4 < p.N) {
        put4<T, EPI>(p, (size_t)(m0 + tok), block * 128 + n4, p.N, o);
      }
    }
  }
}

// Split tiling: 128 weight rows on the MMA's M side x bn <= 128 tokens on its N
// side (one tile of all tokens, or tiles of 64 or 128), the K range cut over the
// `splits` CTAs of a cluster.  Each CTA leaves its fp32 partial tile in its own
// shared memory; after a cluster barrier each adds up every CTA's partials (in
// rank order) for its share of the tokens and writes them: no workspace, no
// atomics, one launch, the same sums each time.  Two CTAs to an SM, each with
// half of its shared memory and tensor memory: one starts or joins while the
// other streams.
//
// 16 x 28672 x 4096 (66 MB): 13.1 us, 5.1 TB/s; 16 x 28672 x 14336: 36.8 us, 6.3
// TB/s (93% of the copy rate): what is lost is about 3.3 us of launch, first
// loads and join.  16 x 4096 x 4096 as four ranges 5.8 us, as one 6.6.
//   warp 0      TMA producer: 256-code slabs of both operands and their scale tiles
//   warp 1      tensor memory; lane 0 copies scale tiles there and issues the MMAs
//   warps 2..5  partial tile to shared memory, join, epilogue
template <typename T, int EPI, bool NV>
__global__ void __launch_bounds__(192)
    gemm_fp4_split_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a, const Params p) {
  using F = Fmt<NV>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + p.stages * p.stage_bytes);
  uint64_t* empty_bar = full_bar + p.stages;
  uint64_t* acc_bar = empty_bar + p.stages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_bar + 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    mbar_init(smem_u32(acc_bar), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc<false>(smem_u32(tmem_slot), (uint32_t)p.tmem_cols);
    tmem_relinquish<false>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // (addresses that the compiler cannot tell to be the same in all lanes are made
  // so by a shuffle: the MMA loop then runs on uniform registers, without a move
  // per operand and instruction)
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
  const uint32_t bars = __shfl_sync(0xffffffffu, smem_u32(full_bar), 0);

  const int rank = p.splits > 1 ? (int)cluster_ctarank() : 0;
  const int mt = blockIdx.y, nt = blockIdx.z;
  const int kb0 = rank * p.slabs_per_split;
  const int n_slabs = min(p.slabs - kb0, p.slabs_per_split);
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_a);
  }
  pdl_wait();
  pdl_launch_dependents();

  if (warp == 0) {
    bool ok = true;
    int i = 0;
    Ring ring{bars + (uint32_t)p.stages * 8, (uint32_t)p.stages, 1};
    const uint8_t* sw = p.sw + (size_t)nt * p.tiles * kTileBytes;
    const uint8_t* sa = p.sa + (size_t)(mt * p.bn >> 7) * p.tiles * kTileBytes;
    for (; i < n_slabs; ++i) {
      uint32_t s;
      ok = ring.next(p.err, SITE_FP4_PRODUCER, s);
      if (!ok) break;
      const int kb = kb0 + i;
      const uint32_t st = base + s * (uint32_t)p.stage_bytes;
      const uint32_t fb = bars + s * 8;
      const uint32_t tile0 = (uint32_t)kb * F::kTiles;
      const uint32_t sb = (uint32_t)min(F::kTiles, p.tiles - (int)tile0) * kTileBytes;
      const uint32_t a_at = st + kOpTile, s_at = a_at + (uint32_t)p.bn * 128;
      if (elect_one()) {
        mbar_expect_tx(fb, (uint32_t)kOpTile + (uint32_t)p.bn * 128 + 2 * sb);
        tma_load_2d(st, &tm_w, kb * 128, nt * 128, fb);
        tma_load_2d(a_at, &tm_a, kb * 128, mt * p.bn, fb);
        bulk_g2s(s_at, sw + (size_t)tile0 * kTileBytes, sb, fb);
        bulk_g2s(s_at + F::kScaleBytes, sa + (size_t)tile0 * kTileBytes, sb, fb);
      }
    }
    // after a failure: no copy is in flight when the CTA leaves
    for (int j = max(0, i - p.stages); !ok && j < i; ++j)
      mbar_wait(smem_u32(&full_bar[j % p.stages]), (uint32_t)(j / p.stages) & 1u, p.err, SITE_FP4_PRODUCER);
    __syncwarp();
  } else if (warp == 1) {
    // a scale buffer per stage (16 columns of W, 16 of A): a stage that is full
    // was emptied, so the MMAs that read its scale buffer before have completed
    const uint32_t sf0 = tmem + (uint32_t)p.tmem_cols - (uint32_t)p.stages * 32;
    const uint32_t stage_step = (uint32_t)p.stage_bytes >> 4;  // in a descriptor's 16-byte units
    const uint64_t wd0 = sw128_desc(base), ad0 = sw128_desc(base + kOpTile);
    const uint64_t swd0 = scale_desc(base + kOpTile + (uint32_t)p.bn * 128);
    // the odd 64-token tiles' scales are the last two of their row block's four columns
    const uint32_t half = (uint32_t)(mt * p.bn >> 5) & 2u;
    const uint32_t idesc0 = idesc_fp4(128, p.bn, NV, 0), idesc1 = idesc_fp4(128, p.bn, NV, NV ? 0 : 2);
    Ring ring{bars, (uint32_t)p.stages, 0};
    // one slab: nt_s scale tiles of each operand to tensor memory, n_mma MMAs
    auto slab = [&](uint32_t acc, int nt_s, int n_mma) {
      uint32_t s;
      if (!ring.next(p.err, SITE_FP4_MMA, s)) return false;
      const uint32_t off = s * stage_step;
      const uint64_t wd = wd0 + off, ad = ad0 + off, swd = swd0 + off;
      const uint32_t sf = sf0 + s * 32;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int t = 0; t < F::kTiles; ++t) {
          if (t < nt_s) {
            tmem_cp_scales<false>(sf + 4 * t, swd + (uint64_t)(t * (kTileBytes >> 4)));
            tmem_cp_scales<false>(sf + 16 + 4 * t, swd + (uint64_t)((F::kScaleBytes + t * kTileBytes) >> 4));
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j < n_mma) {
            const int t = NV ? j : j >> 1;
            mma_fp4<NV, false>(tmem, wd + (uint64_t)(2 * j), ad + (uint64_t)(2 * j), (j & 1) ? idesc1 : idesc0, sf + 4 * t,
                        sf + 16 + 4 * t + half, j != 0 ? 1u : acc);
          }
        }
        mma_commit(bars + (p.stages + s) * 8);
      }
      return true;
    };
    // whole slabs, then the row's ragged end
    const int whole = min(n_slabs, p.K / kSlab - kb0);
    bool ok = true;
    for (int i = 0; ok && i < whole; ++i) ok = slab(i != 0 ? 1u : 0u, F::kTiles, 4);
    if (ok && whole < n_slabs)
      ok = slab(whole != 0 ? 1u : 0u, p.tiles - (kb0 + whole) * F::kTiles, (p.K - (kb0 + whole) * kSlab + 63) >> 6);
    if (ok && elect_one()) mma_commit(smem_u32(acc_bar));
    __syncwarp();
  } else {
    const bool ok = warp_wait(smem_u32(acc_bar), 0, p.err, SITE_FP4_EPILOGUE);
    tc_fence_after();
    // every MMA has completed, and with it every copy into the stages: they hold
    // the partial tile now, [token][128 weight rows]
    const int q = warp & 3;
    float* part = reinterpret_cast<float*>(smem) + q * 32 + lane;
    const uint32_t t0 = tmem + ((uint32_t)(q * 32) << 16);
    for (int j = 0; ok && j < p.bn; j += 32) {
      uint32_t v[32];
      tmem_ld32(t0 + j, v);  // (past bn: columns of the tile's own allocation)
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (j + e < p.bn) part[(j + e) * 128] = __uint_as_float(v[e]);
    }
    tc_fence_before();
  }
  if (p.splits > 1)
    cluster_sync();
  else
    __syncthreads();

  if (warp >= 2)
    join<T, EPI, 128>(p, smem_u32(smem), p.splits, rank, 1, 0, threadIdx.x - 64, nt, mt * p.bn, min(p.bn, p.M - mt * p.bn));
  __syncwarp();
  if (p.splits > 1)
    cluster_sync();  // the partials are read by the whole cluster
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<false>(tmem, (uint32_t)p.tmem_cols);
  }
}

// Pair tiling: 256 weight rows x up to 256 tokens per tile over a CTA pair
// (cta_group::2).  Each CTA of the pair holds 128 weight rows and half of the
// tile's tokens in shared memory; the leader's MMAs (M = 256) read both, so an
// SM fetches (128 + 128) rows per 128 x 256 results where one CTA alone would
// fetch (128 + 256).  Tokens lie on the MMA's N side, so the last token tile is
// as narrow as the batch leaves it (multiples of 16), not a whole tile.
// Persistent: the pairs walk the tiles, whole ones first.
//
// Where the tiles are too few for the SMs, a cluster of two pairs shares one: each
// pair takes a K range, and the partial tiles are joined as in the split tiling
// (512 x 4096 x 14336: 16.6 us, against 21.8 with one range; four ranges, in
// clusters of 8 whole SMs of which few fit at a time, took 40.7).
//
// 8192 x 7168 x 20480: 316 us, 7.6 PFLOP/s; the power cap leaves 1560 MHz there, at
// which the MMAs alone take 309 us.  8192 x 14336 x 4096: 143 us, 6.7 PFLOP/s: a
// slab takes 640 clocks instead of the MMAs' 512, as its 39 KB per SM come from L2
// at 15.6 TB/s (asking for them earlier, by prefetches into L2, made it 157 us).
// With 128 x 128 tiles of one CTA each it took 277 us.
//   warp 0      TMA producer (both CTAs), completion counted on the leader's barrier
//   warp 1      tensor memory; the leader's copies the scale tiles and issues the MMAs
//   warps 2..9  epilogue: a lane quarter (32 weight rows) x half of the tokens each,
//               held in registers, so that the next tile's MMAs start once the
//               accumulator has been read and run under the stores
// Tensor memory: 256 accumulator columns, then a scale buffer of 48 (NV; 24)
// columns per stage.
template <typename T, int EPI, bool NV>
__global__ void __launch_bounds__(kPairThreads, 1)
    gemm_fp4_pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a,
                         const __grid_constant__ CUtensorMap tm_last, const __grid_constant__ CUtensorMap tm_sw,
                         const __grid_constant__ CUtensorMap tm_sa, const __grid_constant__ CUtensorMap tm_c,
                         const Params p) {
  using F = Fmt<NV>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + p.stages * p.stage_bytes);
  uint64_t* empty_bar = full_bar + p.stages;
  uint64_t* acc_bar = empty_bar + p.stages;  // [0] full, [1] empty
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_bar + 2);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    mbar_init(smem_u32(&acc_bar[0]), 1);
    mbar_init(smem_u32(&acc_bar[1]), 16);  // the epilogue warps of both CTAs
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc<true>(smem_u32(tmem_slot), 512);
    tmem_relinquish<true>();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
  const uint32_t bars = __shfl_sync(0xffffffffu, smem_u32(full_bar), 0);
  const uint32_t accb = __shfl_sync(0xffffffffu, smem_u32(acc_bar), 0);
  const uint32_t stage_end = base + (uint32_t)(p.stages * p.stage_bytes + kBarBytes);  // the epilogue's staging
  // this CTA's place in its pair, the pair's K range, the pair's leader
  const int crank = (int)cluster_ctarank(), rank = crank & 1, kr = crank >> 1;
  const uint32_t leader = (uint32_t)crank & ~1u;
  const int cid = blockIdx.x / (2 * p.pair_ranges), pairs = gridDim.x / (2 * p.pair_ranges);
  const int kb0 = kr * p.slabs_per_split, kb1 = min(p.slabs, kb0 + p.slabs_per_split);
  if (warp == 0 && elect_one()) {
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_sw);
    tma_prefetch_desc(&tm_sa);
  }
  pdl_wait();
  pdl_launch_dependents();

  if (warp == 0) {
    Ring ring{bars + (uint32_t)p.stages * 8, (uint32_t)p.stages, 1};
    bool ok = true;
    for (int u = cid; ok && u < p.units; u += pairs) {
      const Tile w = tile_of(p, u);
      const int blocks = w.bn > 128 ? 2 : 1;
      const uint32_t bytes = (uint32_t)(kOpTile + (w.bn >> 1) * 128 + (1 + blocks) * F::kScaleBytes);
      const void* ma = w.bn == 256 ? &tm_a : &tm_last;
      const int w_row = w.nt * 256 + rank * 128, a_row = w.mt * 256 + rank * (w.bn >> 1);
      const int sw_row = (w.nt * 2 + rank) * p.tiles, sa_row = w.mt * 2 * p.tiles;
      for (int kb = kb0; kb < kb1; ++kb) {
        uint32_t s;
        ok = ring.next(p.err, SITE_FP4_PRODUCER, s);
        if (!ok) break;
        const uint32_t st = base + s * (uint32_t)p.stage_bytes;
        if (elect_one()) {
          const uint32_t fb = bars + s * 8, lead = cluster_addr(fb, leader);
          if (rank == 0) mbar_expect_tx(fb, 2 * bytes);
          tma_load_2d_pair(st, &tm_w, kb * 128, w_row, lead);
          tma_load_2d_pair(st + kOpTile, ma, kb * 128, a_row, lead);
          tma_load_2d_pair(st + 2 * kOpTile, &tm_sw, 0, sw_row + kb * F::kTiles, lead);
          tma_load_2d_pair(st + 2 * kOpTile + F::kScaleBytes, &tm_sa, 0, sa_row + kb * F::kTiles, lead);
          if (blocks == 2)
            tma_load_2d_pair(st + 2 * kOpTile + 2 * F::kScaleBytes, &tm_sa, 0, sa_row + p.tiles + kb * F::kTiles, lead);
        }
      }
    }
    // the leader's MMAs have released every fill, so that neither a copy nor a
    // commit is still on its way to this CTA when it leaves (after a failure:
    // waited for once more, for a shorter time)
    for (int i = 0; i < p.stages; ++i) {
      mbar_wait(ring.bars + ring.s * 8, ring.ph ^ 1u, p.err, SITE_FP4_PRODUCER, ok ? kWaitLimitNs : kWaitLimitNs / 16);
      if (++ring.s == ring.stages) {
        ring.s = 0;
        ring.ph ^= 1u;
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      constexpr uint32_t kScaleCols = NV ? 48 : 24;
      const uint32_t stage_step = (uint32_t)p.stage_bytes >> 4;
      const uint64_t wd0 = sw128_desc(base), ad0 = sw128_desc(base + kOpTile);
      const uint64_t sd0 = scale_desc(base + 2 * kOpTile);
      const uint16_t both = (uint16_t)(3u << leader);
      Ring ring{bars, (uint32_t)p.stages, 0};
      int n = 0;
      bool ok = true;
      for (int u = cid; ok && u < p.units; u += pairs, ++n) {
        const Tile w = tile_of(p, u);
        const bool two = w.bn > 128;
        const uint32_t idesc0 = idesc_fp4(256, w.bn, NV, 0), idesc1 = idesc_fp4(256, w.bn, NV, NV ? 0 : 2);
        // The accumulator has to have been read (by both CTAs' epilogues) before
        // the tile's first MMA; its first scale tiles are copied ahead of that wait
        auto slab = [&](bool first, int nt_s, int n_mma) {
          uint32_t s;
          if (!ring.next(p.err, SITE_FP4_MMA, s)) return false;
          const uint32_t off = s * stage_step;
          const uint64_t wd = wd0 + off, ad = ad0 + off, sd = sd0 + off;
          const uint32_t sf = tmem + 256 + s * kScaleCols;
          tc_fence_after();
          auto scales = [&]() {
            // columns: W tile t at 4 t; token tile t at 4 kTiles + 8 t, its two row blocks side by side
#pragma unroll
            for (int t = 0; t < F::kTiles; ++t) {
              if (t < nt_s) {
                tmem_cp_scales<true>(sf + 4 * t, sd + (uint64_t)(t * (kTileBytes >> 4)));
                tmem_cp_scales<true>(sf + 4 * F::kTiles + 8 * t, sd + (uint64_t)((F::kScaleBytes + t * kTileBytes) >> 4));
                if (two)
                  tmem_cp_scales<true>(sf + 4 * F::kTiles + 8 * t + 4,
                                       sd + (uint64_t)((2 * F::kScaleBytes + t * kTileBytes) >> 4));
              }
            }
          };
          if (first) {
            if (elect_one()) scales();
            __syncwarp();
            if (n > 0 && !warp_wait(accb + 8, (uint32_t)(n - 1) & 1u, p.err, SITE_FP4_MMA)) return false;
            tc_fence_after();
          }
          if (elect_one()) {
            if (!first) scales();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (j < n_mma) {
                const int t = NV ? j : j >> 1;
                mma_fp4<NV, true>(tmem, wd + (uint64_t)(2 * j), ad + (uint64_t)(2 * j), (j & 1) ? idesc1 : idesc0,
                                  sf + 4 * t, sf + 4 * F::kTiles + 8 * t, (j != 0 || !first) ? 1u : 0u);
              }
            }
            mma_commit_pair(bars + (p.stages + s) * 8, both);
          }
          return true;
        };
        const int whole = min(kb1, p.K / kSlab);
        if (whole > kb0) ok = slab(true, F::kTiles, 4);
        for (int i = kb0 + 1; ok && i < whole; ++i) ok = slab(false, F::kTiles, 4);
        if (ok && whole < kb1)
          ok = slab(whole == kb0, p.tiles - whole * F::kTiles, (p.K - whole * kSlab + 63) >> 6);
        if (ok && elect_one()) mma_commit_pair(accb, both);
        __syncwarp();
      }
    }
    __syncwarp();
  } else {
    const int q = warp & 3, h = (warp - 2) >> 2;
    const uint32_t mine = stage_end + (uint32_t)(warp - 2) * kWarpOut;  // this warp's staging
    int n = 0, boxes = 0;
    bool alive = true;  // false once a wait gave up: no more loads and stores, but the named barriers stay matched
    for (int u = cid; u < p.units; u += pairs, ++n) {
      const Tile w = tile_of(p, u);
      const int m0 = w.mt * 256 + h * 128;
      const int n0 = w.nt * 256 + rank * 128 + q * 32;  // this warp's first weight row
      const int row = n0 + lane;
      const bool adds = EPI == SAR_EPI_RESIDUAL && p.tma_out && p.c == p.r;  // added in L2
      if (EPI == SAR_EPI_RESIDUAL && !adds && p.slabs <= kPrefetchSlabs) {
        // the residual's lines are on their way to L2 while the MMAs run; over a long
        // K they come so early that some have left L2 again when they are read
        for (int e = lane; e < min(128, p.M - m0); e += 32)
          if (n0 < p.N) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.r + (size_t)(m0 + e) * p.N + n0));
      }
      if (alive) alive = warp_wait(accb, (uint32_t)n & 1u, p.err, SITE_FP4_EPILOGUE);
      if (!alive && EPI != SAR_EPI_SWIGLU && p.pair_ranges == 1) break;
      tc_fence_after();
      uint32_t v[128];
      const uint32_t t0 = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(h * 128);
#pragma unroll
      for (int j = 0; j < 4; ++j) tmem_ld32(t0 + j * 32, v + j * 32);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (alive && elect_one()) mbar_arrive_cluster_relaxed(cluster_addr(accb + 8, leader));
      const int rows = alive ? min(128, p.M - m0) : 0;  // (may be negative: the half is empty)
      if (p.pair_ranges > 1) {
        // One tile to a cluster: this CTA's MMAs are done, its stages are free for
        // the partial tile; every warp of the cluster passes this barrier once
#pragma unroll
        for (int e = 0; e < 128; ++e) st_shared(base + (uint32_t)((h * 128 + e) * 512 + (q * 32 + lane) * 4), v[e]);
        __syncwarp();
        cluster_sync();
        if (alive)
          join<T, EPI, 256>(p, base, p.pair_ranges, kr, 2, rank, threadIdx.x - 64, w.nt * 2 + rank, w.mt * 256,
                            min(256, p.M - w.mt * 256));
        break;
      }
      // One box of `cnt` tokens x 32 columns leaves from the warp's staging
      // (rows behind M and columns behind N are clipped); the other box of the two
      // may still be read meanwhile.
      auto box_begin = [&](uint32_t bytes) {
        if (lane == 0) bulk_wait_read_all_but_one();
        __syncwarp();
        return mine + (EPI == SAR_EPI_SWIGLU ? kWarpOut / 2 : 0) + (uint32_t)(boxes & 1) * bytes;
      };
      auto box_end = [&](uint32_t at, int col, int m) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // visible to the TMA unit
        __syncwarp();
        if (lane == 0) {
          if (adds)
            tma_reduce_add_2d(&tm_c, col, m, at);
          else
            tma_store_2d(&tm_c, col, m, at);
          bulk_commit();
        }
        ++boxes;
      };
      if constexpr (EPI == SAR_EPI_SWIGLU) {
        // The CTA's lanes 0..63 hold gate rows, 64..127 the matching up rows.  Of
        // every 32 tokens the gate warp finishes the first 16 and the warp with
        // its up rows the others: each hands over the half that the other needs.
        const int F2 = p.N >> 1;
        const int col0 = (w.nt * 2 + rank) * 64 + (q & 1) * 32;
        const bool gate = q < 2;
        const uint32_t theirs = stage_end + (uint32_t)((warp - 2) ^ 2) * kWarpOut;
        const int bar = 1 + h * 2 + (q & 1);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");  // the partner has read the last ones
#pragma unroll
          for (int e = 0; e < 16; ++e)
            st_shared(theirs + (uint32_t)(e * 32 + lane) * 4, gate ? v[32 * g + 16 + e] : v[32 * g + e]);
          asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");
          const int m = m0 + 32 * g + (gate ? 0 : 16), cnt = m0 + rows - m;
          if (cnt <= 0 || col0 >= F2) continue;
          const uint32_t at = p.tma_out ? box_begin(1024) : 0;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float mineval = __uint_as_float(gate ? v[32 * g + e] : v[32 * g + 16 + e]) * p.alpha;
            const float other = __uint_as_float(ld_shared(mine + (uint32_t)(e * 32 + lane) * 4)) * p.alpha;
            const T o = Elem<T>::from(gate ? silu(mineval) * other : silu(other) * mineval);
            if (p.tma_out)
              st_shared16(at + (uint32_t)(e * 32 + lane) * 2, o);
            else if (e < cnt)
              reinterpret_cast<T*>(p.c)[(size_t)(m + e) * F2 + col0 + lane] = o;
          }
          if (p.tma_out) box_end(at, col0, m);
        }
      } else if constexpr (EPI == SAR_EPI_STORE) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (32 * g >= rows || n0 >= p.N) continue;
          const uint32_t at = p.tma_out ? box_begin(2048) : 0;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const T o = Elem<T>::from(__uint_as_float(v[32 * g + e]) * p.alpha);
            if (p.tma_out)
              st_shared16(at + (uint32_t)(e * 32 + lane) * 2, o);
            else if (32 * g + e < rows && row < p.N)
              reinterpret_cast<T*>(p.c)[(size_t)(m0 + 32 * g + e) * p.N + row] = o;
          }
          if (p.tma_out) box_end(at, n0, m0 + 32 * g);
        }
      } else {
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          if (16 * g >= rows || n0 >= p.N) continue;
          float x[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(v[16 * g + e]) * p.alpha;
          if (EPI == SAR_EPI_RESIDUAL && !adds) {
            // (all loads first: C may be R)
            float r[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              r[e] = 16 * g + e < rows && row < p.N ? p.r[(size_t)(m0 + 16 * g + e) * p.N + row] : 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] += r[e];
          }
          const uint32_t at = p.tma_out ? box_begin(2048) : 0;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if (p.tma_out)
              st_shared(at + (uint32_t)(e * 32 + lane) * 4, __float_as_uint(x[e]));
            else if (16 * g + e < rows && row < p.N)
              reinterpret_cast<float*>(p.c)[(size_t)(m0 + 16 * g + e) * p.N + row] = x[e];
          }
          if (p.tma_out) box_end(at, n0, m0 + 16 * g);
        }
      }
    }
    // the boxes are in C before the CTA (and its shared memory) goes
    if (lane == 0 && boxes > 0) bulk_wait_all();
    __syncwarp();
  }
  if (warp < 2 && p.pair_ranges > 1) cluster_sync();  // (the epilogue's)
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA of a pair leaves while the other may still address it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<true>(tmem, 512);
  }
}

template <typename T, bool NV>
const void* pick_split(int epi) {
  switch (epi) {
    case SAR_EPI_STORE: return reinterpret_cast<const void*>(&gemm_fp4_split_kernel<T, SAR_EPI_STORE, NV>);
    case SAR_EPI_RESIDUAL: return reinterpret_cast<const void*>(&gemm_fp4_split_kernel<T, SAR_EPI_RESIDUAL, NV>);
    case SAR_EPI_SWIGLU: return reinterpret_cast<const void*>(&gemm_fp4_split_kernel<T, SAR_EPI_SWIGLU, NV>);
    default: return reinterpret_cast<const void*>(&gemm_fp4_split_kernel<T, SAR_EPI_F32, NV>);
  }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct Call {
  const void *a, *w;
  int epi, format, storage, variant;
  cudaStream_t s;
};

// ---- choice of the tiling ----------------------------------------------------
//
// Microseconds of a launch, from its tiles: fitted to 2300 timed runs (1 to 2048
// tokens, N 1024 to 28672, K 1024 to 14336, every tiling and number of K ranges).
// Taking the smallest estimate costs 1.3% over the fastest measured tiling on
// average and 15% at worst.  What it weighs: few tokens want many CTAs on the
// weight (K ranges, until their join costs more than the shorter ranges save: 16
// x 4096 x 14336 15.8 us as one range, 10.1 as four, 12.4 as eight); a middling
// number wants 64-token tiles (128 x 4096 x 4096: 7.5 us, against 9.2 with 128);
// many want the pair tiling (2048 x 28672 x 4096: 74 us, against 147), with two K
// ranges where its tiles would leave half of the SMs idle (512 x 4096 x 14336: 16.6
// us, against 21.8).
constexpr double kSlabOne = 0.28, kSlabOneToken = 0.0006;  // a slab of a CTA alone on its SM; per token of the tile
constexpr double kSlabTwo = 0.44, kSlabTwoToken = 0.0003;  // of a CTA that shares its SM
constexpr double kSplitBase = -1.65, kSplitWave = 3.77, kSplitToken = 0.025, kSplitJoin = 0.54;
constexpr double kPairSlab = 0.338, kPairSlabMin = 0.27, kPairBase = 2.6, kPairTile = 2.1;
constexpr double kPairsSlab = 0.28, kPairsBase = 0.3, kPairsTile = 7.0;  // two K ranges to a tile

double split_us(const Params& p, int width, int splits, int sms) {
  const int m_tiles = (p.M + width - 1) / width, per = (p.slabs + splits - 1) / splits;
  const int ranges = (p.slabs + per - 1) / per;
  const int bn = m_tiles > 1 ? width : (p.M + 15) / 16 * 16;
  const double ctas = (double)m_tiles * ((p.N + 127) / 128) * ranges;
  const double slab = ctas <= sms ? kSlabOne + kSlabOneToken * bn : kSlabTwo + kSlabTwoToken * bn;
  return kSplitBase + std::ceil(ctas / (2.0 * sms)) * (per * slab + kSplitWave + kSplitToken * bn) +
         kSplitJoin * (ranges - 1) * std::cbrt(bn / 16.0);
}

double pair_us(const Params& p, int sms) {
  const int last = (p.M % 256 + 15) / 16 * 16, full = p.M / 256 + (last == 256), pairs = std::max(1, sms / 2);
  const long n_tiles = (p.N + 255) / 256, units = n_tiles * (full + (last != 0 && last != 256));
  const long whole = (full * n_tiles + pairs - 1) / pairs, narrow = std::max(0l, (units + pairs - 1) / pairs - whole);
  return kPairBase + whole * (p.slabs * kPairSlab + kPairTile) +
         narrow * (p.slabs * std::max(kPairSlabMin, kPairSlab * last / 256) + kPairTile);
}

// Two K ranges: a cluster of four whole SMs to a tile (a GPC's SMs do not divide
// into fours: about two clusters fewer than a quarter of the SMs fit).
double pairs_us(const Params& p, int sms) {
  const long units = (long)((p.N + 255) / 256) * ((p.M + 255) / 256), fit = std::max(1, sms / 4 - 2);
  return kPairsBase + (units + fit - 1) / fit * ((p.slabs + 1) / 2 * kPairsSlab + kPairsTile);
}

// The split tiling's tiles lie on a grid's y and z (the pair tiling's on x).
constexpr int kMaxGridYz = 65535;
bool split_fits(const Params& p, int width) {
  return (p.M + width - 1) / width <= kMaxGridYz && (p.N + 127) / 128 <= kMaxGridYz;
}

int pick_variant(const Params& p) {
  const int sms = num_sms();
  int best = SAR_FP4_GEMM_PAIR;
  double us = pair_us(p, sms);
  if (p.slabs > 1 && pairs_us(p, sms) < us) {
    us = pairs_us(p, sms);
    best = SAR_FP4_GEMM_PAIR | 2 << 8;
  }
  for (int width : {128, 64}) {
    if (width == 64 && p.M <= 64) break;  // one tile either way
    if (!split_fits(p, width)) continue;
    for (int splits : {1, 2, 3, 4, 6, 8}) {
      if (splits > p.slabs) break;
      const double t = split_us(p, width, splits, sms);
      if (t < us) {
        us = t;
        best = SAR_FP4_GEMM_SPLIT | splits << 8 | (width == 64 ? SAR_FP4_GEMM_TOKENS64 : 0);
      }
    }
  }
  return best;
}

int launch_split(const Call& g, Params p) {
  const bool nv = g.format == SAR_FP4_NV;
  const int width = g.variant & SAR_FP4_GEMM_TOKENS64 ? 64 : 128;
  const int m_tiles = (p.M + width - 1) / width, n_tiles = (p.N + 127) / 128;
  if (!split_fits(p, width)) return set_error(SAR_ERR_UNSUPPORTED, "gemm_fp4: too many tiles for the split tiling");
  p.bn = m_tiles > 1 ? width : (p.M + 15) / 16 * 16;
  const int splits = std::max(1, g.variant >> 8 & 0xf);
  if (splits > 8 || splits > p.slabs) return set_error(SAR_ERR_UNSUPPORTED, "gemm_fp4: too many K ranges");
  p.slabs_per_split = (p.slabs + splits - 1) / splits;
  p.splits = (p.slabs + p.slabs_per_split - 1) / p.slabs_per_split;  // no empty range
  p.stage_bytes = kOpTile + p.bn * 128 + 2 * (nv ? Fmt<true>::kScaleBytes : Fmt<false>::kScaleBytes);
  p.tmem_cols = 256;  // two CTAs to an SM share its 512 columns
  // two CTAs to an SM, each with half of its shared memory
  const int extra = kBarBytes + 1024;
  p.stages = std::min((p.tmem_cols - p.bn) / 32, (kSmemPerSm / 2 - 1024 - extra) / p.stage_bytes);
  const int smem = p.stages * p.stage_bytes + extra;
  const bool bf = g.storage == SAR_STORAGE_BF16;
  const void* fn = nv ? (bf ? pick_split<__nv_bfloat16, true>(g.epi) : pick_split<__half, true>(g.epi))
                      : (bf ? pick_split<__nv_bfloat16, false>(g.epi) : pick_split<__half, false>(g.epi));
  CUtensorMap tw, ta;
  SAR_TRY(make_tmap_bytes(&tw, g.w, (uint64_t)p.N, (uint64_t)p.K / 2, 128));
  SAR_TRY(make_tmap_bytes(&ta, g.a, (uint64_t)p.M, (uint64_t)p.K / 2, (uint32_t)p.bn));
  SAR_TRY(ensure_smem_attr(fn, kSmemLimit, "gemm_fp4: set smem attribute"));
  void* args[] = {&tw, &ta, &p};
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[2];
  lc.gridDim = dim3((unsigned)p.splits, (unsigned)m_tiles, (unsigned)n_tiles);
  lc.blockDim = dim3(192);
  lc.dynamicSmemBytes = (size_t)smem;
  lc.stream = g.s;
  lc.attrs = attr;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  lc.numAttrs = 1;
  if (p.splits > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    lc.numAttrs = 2;
  }
  const cudaError_t e = cudaLaunchKernelExC(&lc, fn, args);
  if (e != cudaSuccess) return cuda_error(e, "gemm_fp4 launch");
  count_launches(1);
  return SAR_OK;
}

template <typename T, bool NV>
const void* pick_pair(int epi) {
  switch (epi) {
    case SAR_EPI_STORE: return reinterpret_cast<const void*>(&gemm_fp4_pair_kernel<T, SAR_EPI_STORE, NV>);
    case SAR_EPI_RESIDUAL: return reinterpret_cast<const void*>(&gemm_fp4_pair_kernel<T, SAR_EPI_RESIDUAL, NV>);
    case SAR_EPI_SWIGLU: return reinterpret_cast<const void*>(&gemm_fp4_pair_kernel<T, SAR_EPI_SWIGLU, NV>);
    default: return reinterpret_cast<const void*>(&gemm_fp4_pair_kernel<T, SAR_EPI_F32, NV>);
  }
}

int launch_pair(const Call& g, Params p) {
  const bool nv = g.format == SAR_FP4_NV;
  const int rem = p.M % 256;
  p.m_full = p.M / 256;
  p.last_bn = (rem + 15) / 16 * 16;
  if (p.last_bn == 256) {  // the last tile is as good as whole
    ++p.m_full;
    p.last_bn = 0;
  }
  p.n_tiles = (p.N + 255) / 256;
  p.group = std::max(1, std::min(8, p.m_full));
  const long units = (long)p.n_tiles * (p.m_full + (p.last_bn ? 1 : 0));
  if (units > (1l << 30)) return set_error(SAR_ERR_UNSUPPORTED, "gemm_fp4: too many tiles");
  p.units = (int)units;
  int ranges = std::max(1, g.variant >> 8 & 0xf);
  if (ranges > 2) return set_error(SAR_ERR_UNSUPPORTED, "gemm_fp4: the pair tiling takes one or two K ranges");
  if (ranges > p.slabs) return set_error(SAR_ERR_UNSUPPORTED, "gemm_fp4: too many K ranges");
  p.slabs_per_split = (p.slabs + ranges - 1) / ranges;
  if ((p.slabs + p.slabs_per_split - 1) / p.slabs_per_split != ranges)
    return set_error(SAR_ERR_UNSUPPORTED, "gemm_fp4: the K ranges leave one empty");
  p.pair_ranges = ranges;
  const int sb = nv ? Fmt<true>::kScaleBytes : Fmt<false>::kScaleBytes;
  p.stage_bytes = 2 * kOpTile + 3 * sb;  // (a multiple of 1024)
  const int extra = kBarBytes + 1024 + 8 * kWarpOut;
  p.stages = std::min(256 / (nv ? 48 : 24), (kSmemLimit - extra) / p.stage_bytes);
  const int smem = p.stages * p.stage_bytes + extra;
  const bool bf = g.storage == SAR_STORAGE_BF16;
  const void* fn = nv ? (bf ? pick_pair<__nv_bfloat16, true>(g.epi) : pick_pair<__half, true>(g.epi))
                      : (bf ? pick_pair<__nv_bfloat16, false>(g.epi) : pick_pair<__half, false>(g.epi));
  CUtensorMap tw, ta, tl, tsw, tsa, tc;
  std::memset(&tc, 0, sizeof(tc));
  const uint64_t kb = (uint64_t)p.K / 2;
  SAR_TRY(make_tmap_bytes(&tw, g.w, (uint64_t)p.N, kb, 128));
  SAR_TRY(make_tmap_bytes(&ta, g.a, (uint64_t)p.M, kb, 128));
  SAR_TRY(make_tmap_bytes(&tl, g.a, (uint64_t)p.M, kb, p.last_bn ? (uint32_t)p.last_bn / 2 : 128));
  SAR_TRY(make_tmap_words(&tsw, p.sw, (uint64_t)((p.N + 127) / 128) * p.tiles, kTileBytes / 4, sb / kTileBytes));
  SAR_TRY(make_tmap_words(&tsa, p.sa, (uint64_t)((p.M + 127) / 128) * p.tiles, kTileBytes / 4, sb / kTileBytes));
  const bool wide = g.epi == SAR_EPI_F32 || g.epi == SAR_EPI_RESIDUAL;
  const int cols = g.epi == SAR_EPI_SWIGLU ? p.N / 2 : p.N;
  p.tma_out = cols % (wide ? 4 : 8) == 0 && aligned(p.c, 16);
  if (p.tma_out)
    SAR_TRY(make_tmap_out(&tc, p.c, (uint64_t)p.M, (uint64_t)cols, g.epi == SAR_EPI_STORE ? 32 : 16, 32,
                          wide ? SAR_TYPE_F32 : g.storage));
  SAR_TRY(ensure_smem_attr(fn, kSmemLimit, "gemm_fp4: set smem attribute"));
  void* args[] = {&tw, &ta, &tl, &tsw, &tsa, &tc, &p};
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[2];
  lc.blockDim = dim3(kPairThreads);
  lc.dynamicSmemBytes = (size_t)smem;
  lc.stream = g.s;
  lc.attrs = attr;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2 * (unsigned)ranges;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  int clusters = p.units;  // (several ranges: one tile to a cluster)
  if (ranges == 1) {
    cudaLaunchConfig_t qc = lc;  // the cluster shape alone
    qc.gridDim = dim3(128);
    qc.attrs = &attr[1];
    qc.numAttrs = 1;
    int pairs = 0;
    SAR_TRY(max_active_clusters(fn, qc, 2, &pairs, "gemm_fp4: cluster occupancy"));
    clusters = std::min(pairs, p.units);
  }
  lc.numAttrs = 2;
  lc.gridDim = dim3(2u * (unsigned)(ranges * clusters));
  const cudaError_t e = cudaLaunchKernelExC(&lc, fn, args);
  if (e != cudaSuccess) return cuda_error(e, "gemm_fp4 launch");
  count_launches(1);
  return SAR_OK;
}

}  // namespace

}  // namespace sar

using sar::set_error;

extern "C" {

int sar_op_gemm_fp4(const void* a, const void* a_scales, const void* w, const void* w_scales, void* c,
                    const void* residual, int32_t M, int32_t N, int32_t K, float alpha, int32_t epilogue, int32_t format,
                    int32_t variant, int32_t storage, void* stream) try {
  if (M < 0 || N < 1 || K < 1) return set_error(SAR_ERR_INVALID_ARG, "gemm_fp4: bad shape");
  if (epilogue < SAR_EPI_STORE || epilogue > SAR_EPI_F32) return set_error(SAR_ERR_INVALID_ARG, "gemm_fp4: bad epilogue");
  if (format != SAR_FP4_NV && format != SAR_FP4_MX) return set_error(SAR_ERR_INVALID_ARG, "gemm_fp4: bad format");
  if (storage != SAR_STORAGE_F16 && storage != SAR_STORAGE_BF16) return set_error(SAR_ERR_INVALID_ARG, "gemm_fp4: bad storage");
  if (variant < 0 || (variant & 0xff) > SAR_FP4_GEMM_PAIR || variant > 0x1fff ||
      ((variant & 0xf00) && (variant & 0xff) == SAR_FP4_GEMM_AUTO) ||
      ((variant & SAR_FP4_GEMM_TOKENS64) && (variant & 0xff) != SAR_FP4_GEMM_SPLIT))
    return set_error(SAR_ERR_INVALID_ARG, "gemm_fp4: unknown variant");
  // (sizes are rounded up to whole tiles in 32 bits)
  if (M > 1 << 30 || N > 1 << 30 || K > 1 << 30) return set_error(SAR_ERR_UNSUPPORTED, "gemm_fp4: a side above 2^30");
  if (K % 32) return set_error(SAR_ERR_UNSUPPORTED, "gemm_fp4: K must be a multiple of 32");
  if (epilogue == SAR_EPI_SWIGLU && N % 128)
    return set_error(SAR_ERR_UNSUPPORTED, "gemm_fp4: SwiGLU needs whole 64-row gate/up block pairs");
  if (M == 0) return SAR_OK;
  if (!a || !a_scales || !w || !w_scales || !c) return set_error(SAR_ERR_INVALID_ARG, "gemm_fp4: null pointer");
  if (epilogue == SAR_EPI_RESIDUAL && !residual)
    return set_error(SAR_ERR_INVALID_ARG, "gemm_fp4: residual epilogue without residual");
  if (!sar::aligned(a, 16) || !sar::aligned(a_scales, 16) || !sar::aligned(w, 16) || !sar::aligned(w_scales, 16))
    return set_error(SAR_ERR_INVALID_ARG, "gemm_fp4: codes and scales must be 16-byte aligned");
  const bool wide_out = epilogue == SAR_EPI_F32 || epilogue == SAR_EPI_RESIDUAL;
  const uintptr_t elem = wide_out ? 4 : 2;
  if (!sar::aligned(c, elem) || (epilogue == SAR_EPI_RESIDUAL && !sar::aligned(residual, 4)))
    return set_error(SAR_ERR_INVALID_ARG, "gemm_fp4: output not aligned to its element");
  sar::Params p = {};
  p.M = M;
  p.N = N;
  p.K = K;
  p.slabs = (K + sar::kSlab - 1) / sar::kSlab;
  p.tiles = sar::fp4_tiles(K, format);
  p.sa = static_cast<const uint8_t*>(a_scales);
  p.sw = static_cast<const uint8_t*>(w_scales);
  p.c = c;
  p.r = static_cast<const float*>(residual);
  p.alpha = alpha;
  p.vec = N % 4 == 0 && sar::aligned(c, 4 * elem) && (epilogue != SAR_EPI_RESIDUAL || sar::aligned(residual, 16));
  SAR_TRY(sar::op_flags(&p.err));
  if (variant == SAR_FP4_GEMM_AUTO) variant = sar::pick_variant(p);
  const sar::Call g = {a, w, epilogue, format, storage, variant, static_cast<cudaStream_t>(stream)};
  return (variant & 0xff) == SAR_FP4_GEMM_PAIR ? sar::launch_pair(g, p) : sar::launch_split(g, p);
} catch (...) {
  return sar::entry_failed("gemm_fp4");
}

}  // extern "C"
