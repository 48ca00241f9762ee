// Attention of sequences with several rows over the 8-bit paged cache, on the
// 5th-generation tensor cores.
//
// A unit is 256 (row, query head) pairs of one sequence and KV head, packed row by
// row, so that a chunk of a few tokens wastes no tensor rows on absent ones and every
// key is converted once for the whole group; pairs [0, 128) are tile A, the rest B.
//   warps 0..15  softmax: eight per tile (row quarter = the lanes of tensor memory that
//                a warp may touch, key half); scores S from tensor memory, running
//                maximum and sum, P (fp16) back over S; O rescaled where a row's
//                maximum has grown by more than 2^8; at the end O / sum.
//   warps 16..19 convert: 128 keys' codes by 16-byte loads, a block ahead in registers,
//                e4m3 -> fp16 (exact) into the 128-byte swizzled K and V tiles of two
//                stages each.
//   warp 20      one thread issues S_x(j) = Q_x K_j^T and O_x += P_x(j) V_j, the tiles in
//                turn, so that one tile's products run under the other's softmax.
// The queries are fp16 too (bf16 rows scaled by a power of two, undone in the scores'
// factor).  Page scales act as in the single-token kernel: with raw scores S and
// t = S k_scale scale + log2(v_scale), 2^(t - m) weighs V's codes and its sum takes it
// times 1 / v_scale, 16 keys (which lie in one page) at a time: one multiplication
// more per 16 keys and row.
//
// NaN codes of V count as zero in the product, where they would reach rows that do not
// see their key; if any came by, the rows look through their own keys at the end.
//
// Units' blocks of 128 keys form one line.  Where there are few units, every CTA (one
// per SM) takes an equal stretch of it, and pieces of a unit are joined by a second
// kernel; where there are four or more to an SM, a CTA takes a whole unit, the longest
// of a sequence first: a stretch's two pieces cost 256 KB of partial results more.
#include <algorithm>

#include "kv8.cuh"
#include "tc05.cuh"

namespace sar {

namespace {

constexpr int kKeys = 128;               // keys of a block
constexpr int kSoftWarps = 16, kConvWarps = 4;
constexpr int kChunkThreads = (kSoftWarps + kConvWarps + 1) * 32;
constexpr int kTileRegion = 128 * 128;   // [128 rows][128 bytes]: 64 dims of 128 rows
constexpr int kScaleRing = 4;
constexpr int kMostTiles = 640;          // of a call whose CTAs take stretches
constexpr int kLeastBlocks = 4;          // of a stretch
constexpr float kGrowth = 8.f;           // log2 of a maximum's growth that O tolerates
constexpr uint32_t kColsS = 128;         // S_x at x * 128; P over its first 64 columns
constexpr uint32_t kColsO = 256;         // O_x at 256 + x * 128

struct ChunkBars {
  uint64_t k_full[2], v_full[2], k_free[2], v_free[2];
  uint64_t s_full[2], p_full[2];
  uint64_t q_ready, mma_done;
  uint32_t tmem;
  int nan;  // a NaN code of V came by
};

// The plan, in the workspace, for the joining kernel.
struct ChunkPlan {
  int64_t all;    // blocks on the line; 0: nothing to join
  int64_t ctas;
  int32_t tiles;
  int32_t seq[kMostTiles], u[kMostTiles];
  int64_t before[kMostTiles + 1];
};

struct ChunkArgs8 {
  Kv8Attn a;
  ChunkPlan* plan;
  float* parts;      // [2 * SMs][256][D]
  float2* parts_ml;  // [2 * SMs][256]
  int sms, vec_q, vec_o;
};

template <int D>
struct ChunkSmem {
  static constexpr int kOperand = (D / 64) * kTileRegion;  // Q_x, K or V of a block
  static constexpr int kK = 2 * kOperand, kV = kK + 2 * kOperand, kBars = kV + 2 * kOperand;
  static constexpr int kScales = kBars + 256;                       // [ring][3][8] floats
  static constexpr int kRed = kScales + kScaleRing * 3 * 8 * 4;     // [2 tiles][2 parities][2 halves][128]
  static constexpr int kTable = kRed + 2 * 2 * 2 * 128 * 4;         // before [640 + 1], seq, u
  static constexpr int kBytes = 1024 + kTable + (kMostTiles + 1) * 8 + 2 * kMostTiles * 4;
};
static_assert(sizeof(ChunkBars) <= 256, "barrier area");
static_assert(ChunkSmem<128>::kBytes <= 226 * 1024, "shared memory per CTA");

__device__ __forceinline__ uint32_t idesc_f16(int n, uint32_t b_mn) {
  return (1u << 4) | (b_mn << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* err) {
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(smem_u32(bar), parity, err, SITE_KV8_PIPE) ? 1 : 0;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();
  return ok != 0;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void sts_u4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ int tiles_of(int rows, int G) { return rows < 2 ? 0 : (int)(((int64_t)rows * G + 255) / 256); }

// Tile u of a sequence: its pairs, and the blocks of 128 keys that they see.
struct Tile {
  int64_t pair0;       // its first pair
  int pairs;           // up to 256
  int j0, j1, j1a;     // blocks [j0, j1), of which tile A's pairs end at j1a
  int lo;              // the oldest key that any row sees
};
__device__ __forceinline__ Tile tile_of(const Kv8Attn& a, int rows, int len, int u) {
  Tile t;
  t.pair0 = (int64_t)u * 256;
  t.pairs = (int)min((int64_t)256, (int64_t)rows * a.G - t.pair0);
  const int first = len - rows + (int)(t.pair0 / a.G);
  const int last = len - rows + (int)((t.pair0 + t.pairs - 1) / a.G);
  const int last_a = len - rows + (int)((t.pair0 + min(t.pairs, 128) - 1) / a.G);
  t.lo = a.window > 0 ? max(0, first - a.window + 1) : 0;
  t.j0 = t.lo / kKeys;
  t.j1 = max(last, 0) / kKeys + 1;
  t.j1a = max(last_a, 0) / kKeys + 1;
  return t;
}

template <typename T, int D>
__global__ void __launch_bounds__(kChunkThreads, 1) kv8_chunk_kernel(const __grid_constant__ ChunkArgs8 args) {
  using M = ChunkSmem<D>;
  constexpr int REGIONS = D / 64;
  constexpr int CHUNKS = D / 16;                // 16-byte loads of a key
  constexpr int PASS = kConvWarps * 32 / CHUNKS;  // keys of a pass of the converting warps
  constexpr int PASSES = kKeys / PASS;
  const Kv8Attn& a = args.a;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto q_reg = [&](int x) { return sbase + (uint32_t)(x * M::kOperand); };
  auto k_reg = [&](int s) { return sbase + (uint32_t)(M::kK + s * M::kOperand); };
  auto v_reg = [&](int s) { return sbase + (uint32_t)(M::kV + s * M::kOperand); };
  ChunkBars* bars = reinterpret_cast<ChunkBars*>(smem + M::kBars);
  float* scales = reinterpret_cast<float*>(smem + M::kScales);
  int64_t* before = reinterpret_cast<int64_t*>(smem + M::kTable);
  int32_t* t_seq = reinterpret_cast<int32_t*>(before + kMostTiles + 1);
  int32_t* t_u = t_seq + kMostTiles;
  __shared__ int64_t sums[kChunkThreads / 32];
  __shared__ int first_s[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&bars->k_full[s]), kConvWarps);
      mbar_init(smem_u32(&bars->v_full[s]), kConvWarps);
      mbar_init(smem_u32(&bars->k_free[s]), 1);
      mbar_init(smem_u32(&bars->v_free[s]), 1);
      mbar_init(smem_u32(&bars->s_full[s]), 1);
      mbar_init(smem_u32(&bars->p_full[s]), kSoftWarps / 2);
    }
    mbar_init(smem_u32(&bars->q_ready), kSoftWarps);
    mbar_init(smem_u32(&bars->mma_done), 1);
    bars->nan = 0;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();

  // ---- the plan: tiles of every sequence, then this CTA's stretch or unit ----
  auto block_sum = [&](int64_t v, int64_t& total) -> int64_t {  // exclusive
    int64_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kChunkThreads / 32; ++w) {
      if (w < warp) incl += sums[w];
      total += sums[w];
    }
    return incl - v;
  };
  auto seq_tiles = [&](int i) -> int {
    int r0, rows, len;
    return kv8_sequence(a, i, r0, rows, len) ? tiles_of(rows, a.G) : 0;
  };
  const int per = (a.n + kChunkThreads - 1) / kChunkThreads;
  const int i0 = min(a.n, (int)threadIdx.x * per), i1 = min(a.n, i0 + per);
  int64_t mine = 0, nt;
  for (int i = i0; i < i1; ++i) mine += seq_tiles(i);
  const int64_t at0 = block_sum(mine, nt);
  const bool stretches = nt <= kMostTiles && nt * a.kvh < 4 * args.sms;
  int64_t b0, b1, all = 0, C = 0;
  int whole_seq = 0, whole_u = 0;
  if (stretches) {
    int64_t t = at0;
    for (int i = i0; i < i1; ++i) {
      const int k = seq_tiles(i);
      for (int u = 0; u < k; ++u, ++t) t_seq[t] = i, t_u[t] = u;
    }
    __syncthreads();
    int64_t blocks = 0;
    if (threadIdx.x < nt) {
      int r0, rows, len;
      kv8_sequence(a, t_seq[threadIdx.x], r0, rows, len);
      const Tile tl = tile_of(a, rows, len, t_u[threadIdx.x]);
      blocks = tl.j1 - tl.j0;
    }
    const int64_t at = block_sum(blocks, all);
    if (threadIdx.x < nt) before[threadIdx.x] = at;
    if (threadIdx.x == 0) before[nt] = all;
    all *= a.kvh;
    C = max((int64_t)1, min((int64_t)min(args.sms, (int)gridDim.x), all / kLeastBlocks));
    __syncthreads();
    if (blockIdx.x == 0) {
      for (int k = threadIdx.x; k < nt; k += kChunkThreads) {
        args.plan->seq[k] = t_seq[k];
        args.plan->u[k] = t_u[k];
        args.plan->before[k] = before[k];
      }
      if (threadIdx.x == 0) {
        args.plan->before[nt] = before[nt];
        args.plan->all = all;
        args.plan->ctas = C;
        args.plan->tiles = (int)nt;
      }
    }
    if (all == 0 || blockIdx.x >= C) return;
    b0 = all * blockIdx.x / C;
    b1 = all * (blockIdx.x + 1) / C;
  } else {
    if (blockIdx.x == 0 && threadIdx.x == 0) args.plan->all = 0;
    if (blockIdx.x >= nt * a.kvh) return;
    const int64_t t = blockIdx.x / a.kvh;
    if (t >= at0 && t < at0 + mine) {
      int64_t at = at0;
      int i = i0;
      while (t >= at + seq_tiles(i)) at += seq_tiles(i++);
      first_s[0] = i;
      first_s[1] = seq_tiles(i) - 1 - (int)(t - at);
    }
    __syncthreads();
    whole_seq = first_s[0];
    whole_u = first_s[1];
    b0 = 0;
    b1 = 1;
  }

  // A piece: blocks [ja, jb) of one unit.
  struct Piece {
    int seq, kh, row0, rows, len, ja, jb, na;  // na: blocks of tile A
    Tile t;
    int64_t next;
    bool whole;
  };
  auto piece_at = [&](int64_t b) -> Piece {
    Piece p;
    int u;
    if (stretches) {
      int lo = 0, hi = (int)nt;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before[mid] * a.kvh <= b)
          lo = mid;
        else
          hi = mid;
      }
      p.seq = t_seq[lo];
      u = t_u[lo];
      const int64_t nb = before[lo + 1] - before[lo], o = b - before[lo] * a.kvh;
      p.kh = (int)(o / nb);
      p.ja = (int)(o - p.kh * nb);
      p.jb = (int)min(nb, p.ja + (b1 - b));
      p.whole = p.ja == 0 && p.jb == nb;
    } else {
      p.seq = whole_seq;
      u = whole_u;
      p.kh = (int)(blockIdx.x % a.kvh);
      p.whole = true;
    }
    kv8_sequence(a, p.seq, p.row0, p.rows, p.len);
    p.t = tile_of(a, p.rows, p.len, u);
    if (stretches) {
      p.ja += p.t.j0;
      p.jb += p.t.j0;
      p.next = b + (p.jb - p.ja);
    } else {
      p.ja = p.t.j0;
      p.jb = p.t.j1;
      p.next = b1;
    }
    p.na = max(0, min(p.jb, p.t.j1a) - p.ja);
    return p;
  };

  if (warp == kSoftWarps + kConvWarps) {
    tmem_alloc<false>(smem_u32(&bars->tmem), 512);
    tmem_relinquish<false>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;

  if (warp == kSoftWarps + kConvWarps) {
    // ---------------- products ----------------
    if (lane == 0) {
      const uint32_t id_s = idesc_f16(kKeys, 0), id_pv = idesc_f16(D, 1);
      const uint64_t dqa = sw128_desc(q_reg(0)), dqb = sw128_desc(q_reg(1));
      const uint64_t dk0 = sw128_desc(k_reg(0)), dk1 = sw128_desc(k_reg(1));
      const uint64_t dv0 = sw128_desc_mn(v_reg(0), kTileRegion, 1024), dv1 = sw128_desc_mn(v_reg(1), kTileRegion, 1024);
      bool ok = true;
      uint32_t base = 0, done_a = 0, done_b = 0, pieces = 0;  // blocks so far: of the stages, of each tile
      for (int64_t b = b0; b < b1; ++pieces) {
        const Piece p = piece_at(b);
        const int nb = p.jb - p.ja;
        const bool has_b = p.t.pairs > 128;
        if (ok) ok = mbar_wait(smem_u32(&bars->q_ready), pieces & 1, a.err, SITE_KV8_PIPE);
        tc_fence_after();
        // S_x(j); the last tile to read the block frees its K stage
        auto issue_s = [&](int x, int j) -> bool {
          const uint32_t jt = base + j, s = jt & 1;
          const bool first = x == 0 || j >= p.na, last = x == 1 || !has_b;
          if (first && !mbar_wait(smem_u32(&bars->k_full[s]), (jt >> 1) & 1, a.err, SITE_KV8_PIPE)) return false;
          tc_fence_after();
          const uint32_t d = tmem + kColsS * (uint32_t)x;
          const uint64_t db = s ? dk1 : dk0, dq = x ? dqb : dqa;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t o = (uint64_t)(((kk >> 2) * kTileRegion + (kk & 3) * 32) >> 4);
            mma_f16<false>(d, dq + o, db + o, id_s, kk != 0);
          }
          mma_commit(smem_u32(&bars->s_full[x]));
          if (last) mma_commit(smem_u32(&bars->k_free[s]));
          return true;
        };
        auto issue_pv = [&](int x, int j) -> bool {
          const uint32_t jt = base + j, s = jt & 1, jx = (x ? done_b : done_a) + j;
          const bool first = x == 0 || j >= p.na, last = x == 1 || !has_b;
          if (!mbar_wait(smem_u32(&bars->p_full[x]), jx & 1, a.err, SITE_KV8_PIPE)) return false;
          if (first && !mbar_wait(smem_u32(&bars->v_full[s]), (jt >> 1) & 1, a.err, SITE_KV8_PIPE)) return false;
          tc_fence_after();
          const uint32_t pcol = tmem + kColsS * (uint32_t)x, dO = tmem + kColsO + kColsS * (uint32_t)x;
          const uint64_t dv = s ? dv1 : dv0;
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            mma_f16_ts(dO, pcol + kk * 8, dv + (uint64_t)(kk * (16 * 128 / 16)), id_pv, (j > 0 || kk > 0) ? 1u : 0u);
          if (last) mma_commit(smem_u32(&bars->v_free[s]));
          return true;
        };
        if (ok && p.na > 0) ok = issue_s(0, 0);
        if (ok && has_b) ok = issue_s(1, 0);
        for (int j = 0; j < nb && ok; ++j) {
          if (j < p.na) {
            if (!(ok = issue_pv(0, j))) break;
            if (j + 1 < p.na && !(ok = issue_s(0, j + 1))) break;
          }
          if (has_b) {
            if (!(ok = issue_pv(1, j))) break;
            if (j + 1 < nb && !(ok = issue_s(1, j + 1))) break;
          }
        }
        mma_commit(smem_u32(&bars->mma_done));
        base += nb;
        done_a += p.na;
        if (has_b) done_b += nb;
        b = p.next;
        // (the next piece's queries wait for it too; after a wait that gave up nothing is in flight)
        mbar_wait(smem_u32(&bars->mma_done), pieces & 1, a.err, SITE_KV8_PIPE);
      }
    }
    __syncwarp();
  } else if (warp >= kSoftWarps) {
    // ---------------- codes to fp16 ----------------
    const int t = threadIdx.x - kSoftWarps * 32;
    const int c4 = t & 3, rin = (t >> 2) % PASS, half = (t >> 2) / PASS;
    const int ps = 1 << a.shift;
    bool ok = true;
    uint32_t jt = 0;
    for (int64_t b = b0; b < b1;) {
      const Piece p = piece_at(b);
      const int nb = p.jb - p.ja;
      uint4 kr[PASSES], vr[PASSES];
      float ks = 1.f, vs = 1.f;  // lanes 0..7: run lane's scales
      int page = -1, page_next = -1;
      // lanes 0..7: the page of run `lane` of block j; -1 where the call reads none, -2 out of range
      auto look_up = [&](int j) -> int {
        const int key = (p.ja + j) * kKeys + (lane & 7) * 16;
        if (j >= nb || key >= p.len || key + 16 <= p.t.lo) return -1;
        const int g = a.bt[(int64_t)p.seq * a.bt_stride + (key >> a.shift)];
        if (g >= 0 && g < a.num_pages) return g;
        if (lane < 8 && t < 32) report(a.err, SAR_ERR_BOUNDS, SITE_KV8_PAGE, g);
        return -2;
      };
      auto fetch = [&](const uint8_t* codes, uint4 (&r)[PASSES], int j) {
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
          const int row = i * PASS + rin, key = (p.ja + j) * kKeys + row;
          const int g = __shfl_sync(0xffffffffu, page, row >> 4);
          r[i] = make_uint4(0, 0, 0, 0);
          if (g >= 0 && key < p.len)
            r[i] = *reinterpret_cast<const uint4*>(
                codes + ((((int64_t)g * a.kvh + p.kh) << a.shift) + (key & (ps - 1))) * D + half * 64 + c4 * 16);
        }
      };
      auto put = [&](uint32_t dst, const uint4 (&r)[PASSES]) {
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
          const int row = i * PASS + rin;
          const uint32_t at = dst + (uint32_t)(half * kTileRegion + row * 128);
          const uint32_t c0 = at + (uint32_t)(((2 * c4) ^ (row & 7)) << 4), c1 = at + (uint32_t)(((2 * c4 + 1) ^ (row & 7)) << 4);
          sts_u4(c0, from_e4m3x2(r[i].x), from_e4m3x2(r[i].x >> 16), from_e4m3x2(r[i].y), from_e4m3x2(r[i].y >> 16));
          sts_u4(c1, from_e4m3x2(r[i].z), from_e4m3x2(r[i].z >> 16), from_e4m3x2(r[i].w), from_e4m3x2(r[i].w >> 16));
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // visible to the tensor core
        __syncwarp();
      };
      page = look_up(0);
      fetch(a.k_codes, kr, 0);
      fetch(a.v_codes, vr, 0);
      auto fetch_scales = [&]() {
        ks = page == -2 ? -1.f : 1.f, vs = 1.f;
        if (t < 8 && page >= 0) {
          const int64_t unit = (int64_t)page * a.kvh + p.kh;
          ks = a.k_scales[unit];
          vs = a.v_scales[unit];
        }
      };
      fetch_scales();
      page_next = look_up(1);
      for (int j = 0; j < nb; ++j, ++jt) {
        const uint32_t s = jt & 1, par = ((jt >> 1) & 1) ^ 1;
        if (ok) ok = warp_wait(&bars->k_free[s], par, a.err);
        if (!ok) break;
        if (t < 8) {
          float* sc = scales + (jt % kScaleRing) * 24 + t;
          sc[0] = ks;  // negative: keys that are passed over
          sc[8] = log2f(vs);
          sc[16] = 1.f / vs;
        }
        put(k_reg(s), kr);
        if (lane == 0) mbar_arrive(smem_u32(&bars->k_full[s]));
        page = page_next;
        if (j + 1 < nb) {
          fetch(a.k_codes, kr, j + 1);
          fetch_scales();
        }
        page_next = look_up(j + 2);
        // V's NaN codes: zero, and known to have been there
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
          const uint32_t w[4] = {vr[i].x, vr[i].y, vr[i].z, vr[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) bad |= (w[k] & 0x7f7f7f7fu) + 0x01010101u;
        }
        if (bad & 0x80808080u) {
          bars->nan = 1;
#pragma unroll
          for (int i = 0; i < PASSES; ++i) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&vr[i]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t m = (((w[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
              w[k] &= ~(m * 0xffu);
            }
          }
        }
        ok = warp_wait(&bars->v_free[s], par, a.err);
        if (!ok) break;
        put(v_reg(s), vr);
        if (lane == 0) mbar_arrive(smem_u32(&bars->v_full[s]));
        if (j + 1 < nb) fetch(a.v_codes, vr, j + 1);
      }
      if (!ok) break;
      b = p.next;
    }
    __syncwarp();
  } else {
    // ---------------- softmax ----------------
    const int x = warp >> 3, qq = warp & 3, hf = (warp >> 2) & 1;
    const int r = qq * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(qq * 32) << 16);
    const uint32_t scol = lane_base + kColsS * (uint32_t)x, ocol = lane_base + kColsO + kColsS * (uint32_t)x + hf * (D / 2);
    float* red = reinterpret_cast<float*>(smem + M::kRed) + x * 4 * 128;  // [parity][half][128]
    auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + x * 4 + qq) : "memory"); };
    bool alive = true;  // false once a wait gave up: work stops, the barriers stay matched
    uint32_t base = 0, mine_done = 0, pieces = 0;
    bool first_piece = true;
    for (int64_t b = b0; b < b1; ++pieces) {
      const Piece p = piece_at(b);
      const int nb = x == 0 ? p.na : p.t.pairs > 128 ? p.jb - p.ja : 0;
      const int64_t pair = p.t.pair0 + x * 128 + r;
      const bool valid = x * 128 + r < p.t.pairs;
      const int token = valid ? (int)(pair / a.G) : 0, head = p.kh * a.G + (valid ? (int)(pair % a.G) : 0);
      const int pos = valid ? p.len - p.rows + token : -1;  // keys (pos - window, pos] are seen
      const int lo = a.window > 0 ? pos - a.window + 1 : 0;
      float fac = a.scale;
      {
        // this half of the query -> fp16, swizzled as the product reads it
        uint32_t w[D / 4];
        const T* qp = static_cast<const T*>(a.q) + (int64_t)(p.row0 + token) * a.ldq + (int64_t)head * D + hf * (D / 2);
#pragma unroll
        for (int k = 0; k < D / 4; k += 4) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (valid) {
            if (args.vec_q) {
              v = *reinterpret_cast<const uint4*>(qp + 2 * k);
            } else {
              const unsigned short* h = reinterpret_cast<const unsigned short*>(qp + 2 * k);
              v = make_uint4(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16, h[4] | (uint32_t)h[5] << 16,
                             h[6] | (uint32_t)h[7] << 16);
            }
          }
          w[k] = v.x, w[k + 1] = v.y, w[k + 2] = v.z, w[k + 3] = v.w;
        }
        if constexpr (Elem<T>::kMmaFormat == 1) {
          // by a power of two into [1, 2) (both halves by the same): bf16's range into fp16's
          float m = 0.f;
#pragma unroll
          for (int k = 0; k < D / 4; ++k) m = fmaxf(m, fmaxf(fabsf(Elem<T>::lo(w[k])), fabsf(Elem<T>::hi(w[k]))));
          red[hf * 128 + r] = m;
          pair_sync();
          m = fmaxf(m, red[(hf ^ 1) * 128 + r]);
          pair_sync();
          const uint32_t ex = min(max(__float_as_uint(m) >> 23, 1u), 253u);
          fac *= __uint_as_float(ex << 23);
          const float inv = __uint_as_float((254u - ex) << 23);
#pragma unroll
          for (int k = 0; k < D / 4; ++k) w[k] = pack_f16(Elem<T>::lo(w[k]) * inv, Elem<T>::hi(w[k]) * inv);
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int c = REGIONS == 2 ? k : hf * 4 + k;  // 16-byte chunk of the row's 128 bytes
          sts_u4(q_reg(x) + (uint32_t)((REGIONS == 2 ? hf * kTileRegion : 0) + r * 128 + ((c ^ (r & 7)) << 4)), w[4 * k],
                 w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();  // (the piece before's O has been read)
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->q_ready));
      }

      float m_used = -INFINITY, l = 0.f;
      for (int j = 0; j < nb; ++j) {
        const uint32_t jx = mine_done + j;
        if (alive) alive = warp_wait(&bars->s_full[x], jx & 1, a.err);
        tc_fence_after();
        // Scores 32 keys at a time: those of the half's first 32 are read twice, so
        // that a thread holds 32 of them (64 took the registers of half the warps).
        // P goes over S's first 64 columns: this half's first 32 are read again before
        // it writes there, and no one else's are after the exchange of the maxima.
        float sv[32];
        auto load = [&](int h) {
          if (alive) {
            tmem_ld32(scol + hf * 64 + h * 32, reinterpret_cast<uint32_t*>(sv));
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) sv[c] = 0.f;
          }
        };
        const int key0 = (p.ja + j) * kKeys + hf * 64;
        const float* sc = scales + ((base + j) % kScaleRing) * 24 + hf * 4;
        const bool edge = key0 + 63 > pos || key0 < lo;
        // keys that this row does not see, and pages out of range: raw score times factor is -inf
        auto mask = [&](int h) {
          if (edge) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (key0 + h * 32 + c > pos || key0 + h * 32 + c < lo) sv[c] = -INFINITY;
          }
#pragma unroll
          for (int g = 0; g < 2; ++g)
            if (sc[2 * h + g] < 0.f) {
#pragma unroll
              for (int c = 0; c < 16; ++c) sv[16 * g + c] = -INFINITY;
            }
        };
        // (above zero, where -inf times it would be NaN)
        auto factor = [&](int g) { return fmaxf(fabsf(sc[g]) * fac, 1.2e-38f); };
        auto most = [&](int h) -> float {
          float m = -INFINITY;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float m4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) m4[e] = sv[g * 16 + e];
#pragma unroll
            for (int c = 4; c < 16; ++c) m4[c & 3] = fmaxf(m4[c & 3], sv[g * 16 + c]);
            m = fmaxf(m, fmaf(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), factor(2 * h + g), sc[8 + 2 * h + g]));
          }
          return m;
        };
        load(0);
        mask(0);
        float pm = most(0);
        load(1);
        mask(1);
        pm = fmaxf(pm, most(1));
        red[((jx & 1) * 2 + hf) * 128 + r] = pm;
        pair_sync();
        const float m_new = fmaxf(m_used, fmaxf(pm, red[((jx & 1) * 2 + (hf ^ 1)) * 128 + r]));
        const bool need = m_new > m_used + kGrowth;
        uint32_t u[16];
        // P_x(j - 1) V has landed before S_x(j), which was issued behind it
        if (__any_sync(0xffffffffu, need)) {
          const float rs = need ? exp2_fast(m_used - m_new) : 1.f;  // 0 while m_used is -inf
          if (alive && __any_sync(0xffffffffu, need && m_used != -INFINITY)) {
#pragma unroll 1
            for (int c = 0; c < D / 2; c += 16) {
              tmem_ld16(ocol + c, u);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * rs);
              tmem_st16(ocol + c, u);
            }
            tmem_wait_st();
          }
          l *= rs;
          if (need) m_used = m_new;
        }
        const float ref = m_used == -INFINITY ? 0.f : m_used;
        auto weigh = [&](int h) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float f = factor(2 * h + g), off = sc[8 + 2 * h + g] - ref;
            float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float p0 = exp2_fast(fmaf(sv[g * 16 + 2 * e], f, off));
              const float p1 = exp2_fast(fmaf(sv[g * 16 + 2 * e + 1], f, off));
              ls[e & 3] += p0 + p1;
              u[g * 8 + e] = pack_f16(p0, p1);
            }
            l = fmaf((ls[0] + ls[1]) + (ls[2] + ls[3]), sc[16 + 2 * h + g], l);
          }
        };
        weigh(1);
        load(0);
        if (alive) tmem_st16(scol + hf * 32 + 16, u);
        mask(0);
        weigh(0);
        if (alive) tmem_st16(scol + hf * 32, u);
        if (alive) tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (alive && lane == 0) mbar_arrive(smem_u32(&bars->p_full[x]));
      }
      // ---- O / sum, or the piece as it is ----
      pair_sync();  // (red's last maxima have been read)
      red[hf * 128 + r] = l;
      pair_sync();
      const float lt = l + red[(hf ^ 1) * 128 + r];
      pair_sync();
      if (alive) alive = warp_wait(&bars->mma_done, pieces & 1, a.err);
      if (alive && x * 128 < p.t.pairs) {
        tc_fence_after();
        uint32_t nan[D / 64] = {};  // dims whose value is NaN under a key that this row sees
        if (*reinterpret_cast<volatile int*>(&bars->nan)) {
          const int k0 = max(max(lo, 0), p.ja * kKeys), k1 = min(pos, p.jb * kKeys - 1);
          for (int key = k0; key <= k1; ++key) {
            const int g = a.bt[(int64_t)p.seq * a.bt_stride + (key >> a.shift)];
            if (g < 0 || g >= a.num_pages) continue;
            const uint8_t* c = a.v_codes + ((((int64_t)g * a.kvh + p.kh) << a.shift) + (key & ((1 << a.shift) - 1))) * D + hf * (D / 2);
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
              const uint32_t w = *reinterpret_cast<const uint32_t*>(c + 4 * k);
              const uint32_t m = (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
              nan[k >> 3] |= ((m & 1) | (m >> 7 & 2) | (m >> 14 & 4) | (m >> 21 & 8)) << ((k & 7) * 4);
            }
          }
        }
        __syncwarp();
        const int64_t slot = 2 * (int64_t)blockIdx.x + (first_piece ? 0 : 1);
        // (a row that sees keys and has no sum is NaN)
        const float inv = p.whole ? (pos < 0 ? 0.f : 1.f / lt) : 1.f;
        if (!p.whole && hf == 0) args.parts_ml[slot * 256 + x * 128 + r] = make_float2(m_used, lt);
#pragma unroll 1
        for (int c = 0; c < D / 2; c += 16) {
          uint32_t u[16];
          tmem_ld16(ocol + c, u);
          tmem_wait_ld();
          float o[16];
          const uint32_t bits = nan[c >> 5] >> (c & 31);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = bits >> e & 1 ? NAN : __uint_as_float(u[e]) * inv;
          if (p.whole) {
            if (valid) {
              T* op = static_cast<T*>(a.out) + (int64_t)(p.row0 + token) * a.ldo + (int64_t)head * D + hf * (D / 2) + c;
              if (args.vec_o) {
                uint32_t h[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = Elem<T>::pack(o[2 * e], o[2 * e + 1]);
                reinterpret_cast<uint4*>(op)[0] = make_uint4(h[0], h[1], h[2], h[3]);
                reinterpret_cast<uint4*>(op)[1] = make_uint4(h[4], h[5], h[6], h[7]);
              } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) op[e] = Elem<T>::from(o[e]);
              }
            }
          } else if (nb > 0) {
            float4* pp = reinterpret_cast<float4*>(args.parts + (slot * 256 + x * 128 + r) * D + hf * (D / 2) + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) pp[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
      }
      first_piece = false;
      base += p.jb - p.ja;
      mine_done += nb;
      b = p.next;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps + kConvWarps) {
    tc_fence_after();
    tmem_dealloc<false>(tmem, 512);
  }
}

// Joins the pieces of units that several CTAs share, in their order: a CTA per 16
// pairs of a unit.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv8_chunk_join_kernel(const __grid_constant__ ChunkArgs8 args) {
  const Kv8Attn& a = args.a;
  pdl_wait();
  pdl_launch_dependents();
  const ChunkPlan& plan = *args.plan;
  const int64_t all = plan.all, C = plan.ctas;
  if (all == 0) return;
  const int64_t work = (int64_t)plan.tiles * a.kvh * 16;
  for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
    const int t = (int)(w / (a.kvh * 16)), kh = (int)(w / 16 % a.kvh), sub = (int)(w % 16);
    const int64_t nb = plan.before[t + 1] - plan.before[t];
    const int64_t u0 = plan.before[t] * a.kvh + kh * nb, u1 = u0 + nb;
    const int64_t c0 = ((u0 + 1) * C - 1) / all, c1 = (u1 * C - 1) / all;  // the CTAs of its first and last block
    if (c0 == c1) continue;
    const bool starts = all * c0 / C == u0;
    int row0, rows, len;
    kv8_sequence(a, plan.seq[t], row0, rows, len);
    const Tile tl = tile_of(a, rows, len, plan.u[t]);
    for (int k = threadIdx.x; k < 16 * (D / 4); k += 256) {
      const int r = sub * 16 + k / (D / 4), dim = k % (D / 4) * 4;
      if (r >= tl.pairs) continue;
      const int64_t pair = tl.pair0 + r;
      const int token = (int)(pair / a.G), head = kh * a.G + (int)(pair % a.G);
      float Mx = -INFINITY, L = 0.f;
      float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int64_t c = c0; c <= c1; ++c) {
        const int64_t slot = 2 * c + (c == c0 && !starts ? 1 : 0);
        const float2 ml = args.parts_ml[slot * 256 + r];
        if (ml.x == -INFINITY) {
          L += ml.y;  // (zero, or NaN)
          continue;
        }
        const float4 v = *reinterpret_cast<const float4*>(args.parts + (slot * 256 + r) * D + dim);
        const float mn = fmaxf(Mx, ml.x);
        const float f = Mx == -INFINITY ? 0.f : exp2_fast(Mx - mn), g = exp2_fast(ml.x - mn);
        L = fmaf(ml.y, g, L * f);
        A.x = fmaf(v.x, g, A.x * f);
        A.y = fmaf(v.y, g, A.y * f);
        A.z = fmaf(v.z, g, A.z * f);
        A.w = fmaf(v.w, g, A.w * f);
        Mx = mn;
      }
      const float inv = len - rows + token < 0 ? 0.f : 1.f / L;
      T* op = static_cast<T*>(a.out) + (int64_t)(row0 + token) * a.ldo + (int64_t)head * D + dim;
      if (args.vec_o) {
        *reinterpret_cast<uint2*>(op) = make_uint2(Elem<T>::pack(A.x * inv, A.y * inv), Elem<T>::pack(A.z * inv, A.w * inv));
      } else {
        op[0] = Elem<T>::from(A.x * inv), op[1] = Elem<T>::from(A.y * inv);
        op[2] = Elem<T>::from(A.z * inv), op[3] = Elem<T>::from(A.w * inv);
      }
    }
  }
}

template <typename T, int D>
int launch_chunk8(const ChunkArgs8& c, cudaStream_t s) {
  const int smem = ChunkSmem<D>::kBytes;
  SAR_TRY(ensure_smem_attr(reinterpret_cast<const void*>(&kv8_chunk_kernel<T, D>), smem, "kv8 chunk: set smem attribute"));
  // as many CTAs as units can come to, one per SM at least
  const int64_t pairs = (int64_t)c.a.rows * c.a.G;
  const int64_t tiles = pairs / 256 + std::min(c.a.n, c.a.rows / 2);
  const int64_t grid = std::max(tiles * c.a.kvh, (int64_t)c.sms);
  if (grid > INT32_MAX) return set_error(SAR_ERR_UNSUPPORTED, "kv8_attention: more than 2^31 units");
  cudaError_t e = launch_pdl(kv8_chunk_kernel<T, D>, dim3((unsigned)grid), dim3(kChunkThreads), (size_t)smem, s, c);
  if (e != cudaSuccess) return cuda_error(e, "kv8 chunk launch");
  e = launch_pdl(kv8_chunk_join_kernel<T, D>, dim3((unsigned)std::min(grid * 16, (int64_t)8 * c.sms)), dim3(256), 0, s, c);
  if (e != cudaSuccess) return cuda_error(e, "kv8 chunk join launch");
  count_launches(2);
  return SAR_OK;
}

int64_t up256(int64_t x) { return (x + 255) & ~int64_t(255); }

}  // namespace

int64_t kv8_chunk_space(int head_dim) {
  const int64_t slots = 2ll * num_sms() * 256;
  return up256(sizeof(ChunkPlan)) + up256(slots * 8) + slots * head_dim * 4;
}

int launch_kv8_chunks(const Kv8Attn& a, int head_dim, int storage, void* space, cudaStream_t s) {
  ChunkArgs8 c = {};
  c.a = a;
  c.sms = num_sms();
  uint8_t* w = static_cast<uint8_t*>(space);
  c.plan = reinterpret_cast<ChunkPlan*>(w);
  w += up256(sizeof(ChunkPlan));
  c.parts_ml = reinterpret_cast<float2*>(w);
  c.parts = reinterpret_cast<float*>(w + up256(2ll * c.sms * 256 * 8));
  c.vec_q = aligned_to(a.q, 16) && a.ldq % 8 == 0;
  c.vec_o = aligned_to(a.out, 16) && a.ldo % 8 == 0;
  if (head_dim == 128)
    return storage == SAR_STORAGE_BF16 ? launch_chunk8<__nv_bfloat16, 128>(c, s) : launch_chunk8<__half, 128>(c, s);
  return storage == SAR_STORAGE_BF16 ? launch_chunk8<__nv_bfloat16, 64>(c, s) : launch_chunk8<__half, 64>(c, s);
}

}  // namespace sar
