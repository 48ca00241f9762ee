// Attention of single tokens over the 8-bit paged cache.
//
// Bound by the cache's bytes: 2 D of them per key and KV head, for 4 D G flops.  128
// sequences of up to 8192 keys (1.09 GB): 174.5 us with the join, 6.2 TB/s (170 without it);
// four of up to 131072: 117 us, 5.8 TB/s; one of 500 keys: 10.3 us, latencies.
//
// All (sequence, KV head) units' keys, in blocks of 32, form one line, of which every
// CTA takes a stretch, whatever the lengths.  Where a stretch begins or ends
// inside a unit, the CTA writes that piece unnormalised, and a second kernel joins a
// unit's pieces; so a call of a few long sequences and one of many short ones both
// fill the machine.  The plan is three prefix sums' worth of arithmetic on the
// lengths, formed by every CTA itself.
//
// Inside a CTA four warps take the stretch's blocks in turn, each with a ring of
// blocks of its own, filled by TMA with the 128-byte swizzle across unit ends, so
// the stream does not stop where a unit does.  Keys are the rows of the products:
// S^T = K Q^T has 16 keys x 8 heads a tile and O^T = V^T P^T 16 dims x 8 heads, so a
// group of up to eight heads wastes half as much as it would as the rows.  Codes
// turn to fp16 in registers, exactly, on their way into the products (an e4m3 mma.sync
// does the same, and with the queries too, at every use: 139 us against 127 when it was
// tried); the order of the dims inside a step is free, and taken so that a lane's 16 bytes
// of a key are its operands.  V's bytes are transposed by ldmatrix over pairs of dims.
//
// Scales cost nothing: with t = S k_scale scale + log2(v_scale) in base 2 and m the
// running maximum of t, 2^(t - m) weighs V's codes, and the sum takes it times
// 1 / v_scale.  Pages of value scales far below others' have weights too small for fp16: 16 keys
// of such a page get a product of their own against their own maximum (a context of 200000 keys
// 67 us, 75 where pages differ so; the test alone costs nothing that was measured).
#include <algorithm>

#include "kv8.cuh"
#include "tc05.cuh"

namespace sar {

namespace {

constexpr int kDecWarps = 4;
constexpr int kDecKeys = 32;    // keys of a block
constexpr int kDecStages = 2;   // blocks of a warp's ring
constexpr int kDecPerSm = 3;
// A CTA takes a unit where the longest sequence has few blocks (six requests of up to 300
// keys 8.9 us; 13 cut), or some more and there are many units (16 requests of up to 1000
// keys, 128 units: 15.9 us, 18.5 cut; 32: 18 and 26; but eight 15.5 and 12.3, one 16.5 and
// 10.9); else the line is cut, for a second kernel to join; so it is where chunks,
// whose CTAs take whole SMs, wait for the last (42.4 and 39.3 us).
constexpr int kDecFew = 16, kDecUnit = 32, kDecUnits = 96;

struct DecArgs {
  Kv8Attn a;
  DecLine* line;
  DecStart* starts;  // [CTAs]
  float* parts;      // [2 * CTAs][8][D]: a CTA's first and last piece
  float2* parts_ml;  // [2 * CTAs][8] maximum and sum
  int resident;  // CTAs that stay on the SMs at once
  int units;     // a unit to a CTA, and nothing to join
  int vec_q, vec_o;
};

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// The transpose of an 8 x 8 matrix of 16-bit elements, a row's pair to a lane.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// A sequence of one row, as the decode kernel sees it.
struct DecSeq {
  int row, len, lo;  // its row, its length, the oldest key it sees
  int blocks;        // of 32 keys, from the one that holds lo; one (without keys) where it is empty; 0: not this kernel's
};
__device__ __forceinline__ DecSeq dec_sequence(const Kv8Attn& a, int i) {
  DecSeq s;
  int rows;
  const bool ok = kv8_sequence(a, i, s.row, rows, s.len);
  s.lo = a.window > 0 ? max(0, s.len - a.window) : 0;
  s.blocks = ok && rows == 1 ? max(1, (s.len + kDecKeys - 1) / kDecKeys - s.lo / kDecKeys) : 0;
  return s;
}

template <typename T, int D>
__global__ void __launch_bounds__(kDecWarps * 32, kDecPerSm)
    kv8_decode_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                      const __grid_constant__ DecArgs d) {
  constexpr int BLK = kDecKeys * D;          // bytes of a block's keys
  constexpr int STAGE = 2 * BLK;
  constexpr int NT = D / 16;                 // tiles of 16 dims
  constexpr int JOINERS = NT / 2;            // warps that join pieces: a tile each in each of two rounds
  constexpr int HALVES = D / 64;
  constexpr int kThreads = kDecWarps * 32;
  const Kv8Attn& a = d.a;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ float rec[kDecWarps][JOINERS][4][32];  // half a piece's tiles, for the joining warps
  __shared__ float ml_s[kDecWarps][kDecHeads][2];
  __shared__ float scale_s[kDecWarps][kDecStages][2][2];  // a block's two pages: key, value scale; key < 0: no page
  __shared__ uint64_t bars_s[kDecWarps][kDecStages];
  __shared__ int64_t sums_s[kDecWarps];
  __shared__ int64_t first_s[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c4 = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * kDecStages * STAGE;
  if (lane == 0) {
    for (int s = 0; s < kDecStages; ++s) mbar_init(smem_u32(&bars_s[warp][s]), 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
  }
  pdl_wait();

  auto check = [&](int i) {  // (once for the call)
    int r0, rows, len;
    if (!kv8_sequence(a, i, r0, rows, len)) report(a.err, SAR_ERR_BOUNDS, SITE_KV8_SEQUENCE, i);
  };
  // ---- this CTA's stretch ----
  struct Place {  // block j of KV head kh of sequence seq
    int seq, kh, j;
    DecSeq s;
  };
  Place here;
  int count;  // this CTA's blocks, counted from 0 below
  if (d.units) {
    here.seq = (int)(blockIdx.x / (unsigned)a.kvh);
    here.kh = (int)(blockIdx.x - (unsigned)here.seq * a.kvh);
    here.j = 0;
    here.s = dec_sequence(a, here.seq);
    count = here.s.blocks;
    if (here.kh == 0 && threadIdx.x == 0) check(here.seq);
    pdl_launch_dependents();
    if (count == 0) return;
  } else {
    const int per = (a.n + kThreads - 1) / kThreads;
    const int i0 = min(a.n, (int)threadIdx.x * per), i1 = min(a.n, i0 + per);
    int64_t mine = 0;
    for (int i = i0; i < i1; ++i) {
      mine += dec_sequence(a, i).blocks;
      if (blockIdx.x == 0) check(i);
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) sums_s[warp] = incl;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      if (w < warp) incl += sums_s[w];
      total += sums_s[w];
    }
    const int64_t excl = incl - mine;
    const int64_t all = total * a.kvh;
    const DecLine line = DecLine::of(all, d.resident, gridDim.x);
    // (a CTA counts its blocks in 32 bits: 2^36 keys)
    const bool fits = all <= (int64_t)line.first * 0x7fffff00;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      *d.line = line;
      if (!fits) {
        d.line->all = 0;  // nothing to join
        report(a.err, SAR_ERR_BOUNDS, SITE_KV8_SEQUENCE, -1);
      }
    }
    if (all == 0 || !fits || blockIdx.x >= line.ctas) return;
    pdl_launch_dependents();
    const int64_t b0 = line.at(blockIdx.x), b1 = line.at(blockIdx.x + 1);
    if (b0 >= excl * a.kvh && b0 < incl * a.kvh) {
      int64_t at = excl;
      int i = i0;
      while (true) {
        const int nb = dec_sequence(a, i).blocks;
        if (b0 < (at + nb) * a.kvh) break;
        at += nb;
        ++i;
      }
      first_s[0] = i;
      first_s[1] = at * a.kvh;
    }
    __syncthreads();
    count = (int)(b1 - b0);
    here.seq = (int)first_s[0];
    here.s = dec_sequence(a, here.seq);
    const int64_t o = b0 - first_s[1];
    here.kh = (int)DecLine::quotient(o, here.s.blocks);
    here.j = (int)(o - (int64_t)here.kh * here.s.blocks);
    if (threadIdx.x == 0)
      d.starts[blockIdx.x] = {b0 - here.j, here.s.blocks, here.j > 0 ? here.seq : -1, here.kh, here.s.row};
  }

  // n blocks on; the caller knows that the line is that long
  auto advance = [&](Place& p, int n) {
    p.j += n;
    while (p.j >= p.s.blocks) {
      p.j -= p.s.blocks;
      if (++p.kh < a.kvh) continue;
      p.kh = 0;
      do p.s = dec_sequence(a, ++p.seq);
      while (p.s.blocks == 0);
    }
  };

  // ---- loads: a warp's blocks are warp, warp + 4, ... ----
  Place ahead = here;
  int at = warp;  // the next block to fetch
  if (at < count) advance(ahead, warp);
  int kh_a = 0, key_a = 0, page_a = -1;
  bool want_a = false;
  // the page of the next block's 16 keys (lane 0: the first, lane 1: the second); looked at
  // when the block is fetched, a block later: a test here would wait for the load
  auto look_up = [&]() {
    if (at >= count) return;
    kh_a = ahead.kh;
    key_a = (ahead.s.lo / kDecKeys + ahead.j) * kDecKeys;
    const int key = key_a + 16 * lane;
    want_a = lane < 2 && key < ahead.s.len && key + (a.shift > 4 ? kDecKeys : 16) > ahead.s.lo;  // (pages behind a window may be gone)
    if (want_a) page_a = a.bt[(int64_t)ahead.seq * a.bt_stride + (key >> a.shift)];
  };
  auto issue = [&](int s) {  // that block into stage s, and the look-up of the one after
    if (want_a && (page_a < 0 || page_a >= a.num_pages)) {
      report(a.err, SAR_ERR_BOUNDS, SITE_KV8_PAGE, page_a);
      page_a = -1;
    }
    if (!want_a) page_a = -1;
    const uint32_t bar = smem_u32(&bars_s[warp][s]), dst = ring + s * STAGE;
    // pages of 32 keys and up: one box holds the block
    const bool whole = a.shift > 4;
    const int p0 = __shfl_sync(0xffffffffu, page_a, 0), p1 = __shfl_sync(0xffffffffu, page_a, 1);
    const int boxes = whole ? (p0 >= 0) : (p0 >= 0) + (p1 >= 0);
    const uint32_t box = whole ? BLK : BLK / 2;
    if (lane < 2) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (lane == 0) {
      if (boxes)
        mbar_expect_tx(bar, 2 * boxes * box);
      else
        mbar_arrive(bar);
    }
    __syncwarp();
    if (lane < 2) {
      const int ps = 1 << a.shift;
      if (page_a >= 0) {
        const int64_t unit = (int64_t)page_a * a.kvh + kh_a;
        if (lane == 0 || !whole) {
          // (rows of the map are 128 bytes: one key, or two of 64 dims)
          const int row = (int)((unit * ps + ((key_a + 16 * lane) & (ps - 1))) * D / 128);
          tma_load_2d(dst + lane * (BLK / 2), &tmk, 0, row, bar);
          tma_load_2d(dst + BLK + lane * (BLK / 2), &tmv, 0, row, bar);
        }
        const uint32_t to = smem_u32(&scale_s[warp][s][lane][0]);
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(a.k_scales + unit) : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + 4), "l"(a.v_scales + unit) : "memory");
      } else {
        scale_s[warp][s][lane][0] = -1.f;
      }
    }
    at += kDecWarps;
    if (at < count) advance(ahead, kDecWarps);
    look_up();
  };
  look_up();
  int issued = 0, consumed = 0;
#pragma unroll
  for (int s = 0; s < kDecStages; ++s) {
    if (at < count) {
      issue(s);
      ++issued;
    }
    cp_async_commit();
  }

  bool alive = true;  // false once a wait gave up: the CTA's barriers stay matched
  bool first_piece = true;
  // queries: head g's dims in the order of the products' steps, as they are
  uint32_t qf[HALVES * 8];
  auto load_q = [&]() {
    const T* qp = static_cast<const T*>(a.q) + (int64_t)here.s.row * a.ldq + (int64_t)(here.kh * a.G + (g < a.G ? g : 0)) * D;
#pragma unroll
    for (int h = 0; h < HALVES * 2; ++h) {
      const T* p = qp + 16 * HALVES * c4 + 8 * h;
      if (d.vec_q) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        qf[4 * h] = v.x, qf[4 * h + 1] = v.y, qf[4 * h + 2] = v.z, qf[4 * h + 3] = v.w;
      } else {
        const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
        for (int k = 0; k < 4; ++k) qf[4 * h + k] = u[2 * k] | (uint32_t)u[2 * k + 1] << 16;
      }
    }
  };
  load_q();
  // a lane's places in a block: its 16-byte chunks of K (keys g, + 8, + 16, + 24 lie 8
  // keys' bytes apart) and its row of V
  uint32_t k_at[HALVES], v_at[NT];
#pragma unroll
  for (int h = 0; h < HALVES; ++h) {
    const int row = D == 128 ? g : g >> 1, chunk = D == 128 ? 2 * c4 + h : (g & 1) * 4 + c4;
    k_at[h] = (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4));
  }
#pragma unroll
  for (int c = 0; c < NT; ++c) {
    const int row = D == 128 ? lane : lane >> 1, chunk = D == 128 ? c : (lane & 1) * 4 + c;
    v_at[c] = (uint32_t)(BLK + row * 128 + ((chunk ^ (row & 7)) << 4));
  }
  int next = warp;  // this warp's next block
  int stage = 0;
  uint32_t phase = 0;
  for (int b = 0; b < count;) {
    // ---- one unit's piece: blocks [b, e), of which b is the unit's block here.j ----
    const DecSeq sq = here.s;
    const int kh = here.kh, j0 = here.j, blocks = sq.blocks;
    const int len = min(count - b, blocks - j0), e = b + len;

    // the queries scaled by a power of two so that the largest lies in [1, 2): bf16's
    // range goes into fp16's
    float fac;
    {
      const bool live = g < a.G;
      fac = a.scale;
      if constexpr (Elem<T>::kMmaFormat == 1) {
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < HALVES * 8; ++k) m = fmaxf(m, fmaxf(fabsf(Elem<T>::lo(qf[k])), fabsf(Elem<T>::hi(qf[k]))));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        // (an exponent whose inverse is a normal number too; infinities stay what they are)
        const uint32_t ex = min(max(__float_as_uint(m) >> 23, 1u), 253u);
        fac *= __uint_as_float(ex << 23);
        const float inv = __uint_as_float((254u - ex) << 23);
#pragma unroll
        for (int k = 0; k < HALVES * 8; ++k) qf[k] = pack_f16(Elem<T>::lo(qf[k]) * inv, Elem<T>::hi(qf[k]) * inv);
      }
#pragma unroll
      for (int k = 0; k < HALVES * 8; ++k) qf[k] = live ? qf[k] : 0u;
    }
    // of the columns' heads, 2 c4 and 2 c4 + 1
    const float fac0 = __shfl_sync(0xffffffffu, fac, 8 * c4), fac1 = __shfl_sync(0xffffffffu, fac, 8 * c4 + 4);

    float o[NT][4];
#pragma unroll
    for (int c = 0; c < NT; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float top = 0.f;  // the largest value scale of this piece's pages so far

    for (; next < e; next += kDecWarps) {
      const int s = stage;
      cp_async_wait<kDecStages - 1>();
      if (alive) {
        int got = 0;
        if (lane == 0)
          got = mbar_wait(smem_u32(&bars_s[warp][s]), phase, a.err, SITE_KV8_PIPE) ? 1 : 0;
        alive = __shfl_sync(0xffffffffu, got, 0) != 0;
      }
      __syncwarp();
      ++consumed;
      if (++stage == kDecStages) stage = 0, phase ^= 1u;
      if (alive && sq.len > 0) {
        const int key0 = (sq.lo / kDecKeys + j0 + next - b) * kDecKeys;
        const uint32_t kb = ring + s * STAGE;
        float ks[2], vs[2], lv[2], iv[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          ks[t] = scale_s[warp][s][t][0];
          vs[t] = scale_s[warp][s][t][1];
          lv[t] = log2_fast(vs[t]);
          iv[t] = rcp_fast(vs[t]);
        }
        const bool edge = key0 < sq.lo || key0 + kDecKeys > sq.len || fminf(ks[0], ks[1]) < 0.f;
        // ---- S^T = K Q^T ----
        float sc[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
            // keys t * 16 + g, and + 8: 8 D bytes on, at the same place of the swizzle
            // where a row holds one key; where it holds two, rows 4 on have bit 2 turned
            const uint32_t p = kb + t * (16 * D);
            const uint4 x = lds_u4(p + k_at[h]), y = lds_u4(p + (D == 128 ? k_at[h] + 8 * D : (k_at[h] + 8 * D) ^ 64));
            const uint32_t lo[4] = {x.x, x.y, x.z, x.w}, hi[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int w = 0; w < 4; ++w)
              mma_f16(sc[t], from_e4m3x2(lo[w]), from_e4m3x2(hi[w]), from_e4m3x2(lo[w] >> 16), from_e4m3x2(hi[w] >> 16),
                      qf[8 * h + 2 * w], qf[8 * h + 2 * w + 1]);
          }
        }
        // ---- softmax over keys t * 16 + 8 u + g, of heads 2 c4 (even) and 2 c4 + 1 ----
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float f0 = fac0 * ks[t], f1 = fac1 * ks[t];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            sc[t][2 * u] = fmaf(sc[t][2 * u], f0, lv[t]);
            sc[t][2 * u + 1] = fmaf(sc[t][2 * u + 1], f1, lv[t]);
          }
        }
        if (edge) {
          // keys that are not seen: no score, and codes of V that count as zero
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const bool page = ks[t] >= 0.f;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int key = key0 + t * 16 + u * 8 + g;
              if (key < sq.lo || key >= sq.len || !page) sc[t][2 * u] = sc[t][2 * u + 1] = -INFINITY;
            }
            if (!page) iv[t] = 0.f;
          }
          if (key0 + lane < sq.lo || key0 + lane >= sq.len || (lane < 16 ? ks[0] : ks[1]) < 0.f) {
#pragma unroll
            for (int c = 0; c < NT; ++c)
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(kb + v_at[c]), "r"(0u) : "memory");
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (the stage is filled by TMA again)
          __syncwarp();
        }
        float mx0 = fmaxf(fmaxf(sc[0][0], sc[0][2]), fmaxf(sc[1][0], sc[1][2]));
        float mx1 = fmaxf(fmaxf(sc[0][1], sc[0][3]), fmaxf(sc[1][1], sc[1][3]));
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, x));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, x));
        }
        // O is scaled anew where a maximum has grown by more than 2^8 (weights stay below it)
        const bool need0 = mx0 > m0 + kGrowth, need1 = mx1 > m1 + kGrowth;
        if (__any_sync(0xffffffffu, need0 || need1)) {
          const float r0 = need0 ? exp2_fast(m0 - mx0) : 1.f, r1 = need1 ? exp2_fast(m1 - mx1) : 1.f;  // (0 from -inf)
#pragma unroll
          for (int c = 0; c < NT; ++c) o[c][0] *= r0, o[c][1] *= r1, o[c][2] *= r0, o[c][3] *= r1;
          l0 *= r0;
          l1 *= r1;
          m0 = need0 ? mx0 : m0;
          m1 = need1 ? mx1 : m1;
        }
        const float ref0 = m0 == -INFINITY ? 0.f : m0 - kBias, ref1 = m1 == -INFINITY ? 0.f : m1 - kBias;
        uint32_t pb[2][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float p0 = exp2_fast(sc[t][0] - ref0), p1 = exp2_fast(sc[t][1] - ref1);
          const float p2 = exp2_fast(sc[t][2] - ref0), p3 = exp2_fast(sc[t][3] - ref1);
          l0 = fmaf(p0 + p2, iv[t], l0);
          l1 = fmaf(p1 + p3, iv[t], l1);
          pb[t][0] = transposed(pack_f16(p0, p1));
          pb[t][1] = transposed(pack_f16(p2, p3));
        }
        // pages of value scales far below others': against their own maximum, in a product of their own
        top = fmaxf(top, fmaxf(ks[0] < 0.f ? 0.f : vs[0], ks[1] < 0.f ? 0.f : vs[1]));
        if (__builtin_expect(fminf(vs[0], vs[1]) < top * kApart, 0)) {
#pragma unroll 1
          for (int t = 0; t < 2; ++t) {
            const bool apart = t ? ks[1] >= 0.f && vs[1] < top * kApart : ks[0] >= 0.f && vs[0] < top * kApart;
            if (!apart) continue;
            const float s0 = t ? sc[1][0] : sc[0][0], s1 = t ? sc[1][1] : sc[0][1], s2 = t ? sc[1][2] : sc[0][2], s3 = t ? sc[1][3] : sc[0][3];
            float a0 = fmaxf(s0, s2), a1 = fmaxf(s1, s3);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
              a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, x));
              a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, x));
            }
            const float w0 = exp2_fast(a0 - ref0), w1 = exp2_fast(a1 - ref1);  // (0 from -inf)
            a0 = a0 == -INFINITY ? 0.f : a0;
            a1 = a1 == -INFINITY ? 0.f : a1;
            const uint32_t b0 = transposed(pack_f16(exp2_fast(s0 - a0), exp2_fast(s1 - a1)));
            const uint32_t b1 = transposed(pack_f16(exp2_fast(s2 - a0), exp2_fast(s3 - a1)));
            // (little code: products a tile at a time, through this lane's place in the records)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll 1
              for (int c = 0; c < JOINERS; ++c) {
                const int row = D == 128 ? lane : lane >> 1, chunk = half * JOINERS + c + (D == 128 ? 0 : (lane & 1) * 4);
                uint32_t v[4];
                ldsm_x4_t(kb + (uint32_t)(BLK + row * 128 + ((chunk ^ (row & 7)) << 4)), v);
                const uint32_t lo = __byte_perm(t ? v[2] : v[0], 0, 0x3120), hi = __byte_perm(t ? v[3] : v[1], 0, 0x3120);
                float u[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16(u, from_e4m3x2(lo), from_e4m3x2(lo >> 16), from_e4m3x2(hi), from_e4m3x2(hi >> 16), b0, b1);
#pragma unroll
                for (int k = 0; k < 4; ++k) rec[warp][c][k][lane] = u[k];
              }
#pragma unroll
              for (int c = 0; c < JOINERS; ++c)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[half * JOINERS + c][k] = fmaf(rec[warp][c][k][lane], k & 1 ? w1 : w0, o[half * JOINERS + c][k]);
            }
            if (t)
              pb[1][0] = pb[1][1] = 0;
            else
              pb[0][0] = pb[0][1] = 0;
          }
        }
        // ---- O^T += V^T P^T ----
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          uint32_t v[4];
          ldsm_x4_t(kb + v_at[c], v);
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = __byte_perm(v[q], 0, 0x3120);  // (two keys of the even dim, two of the odd)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            mma_f16(o[c], from_e4m3x2(v[2 * t]), from_e4m3x2(v[2 * t] >> 16), from_e4m3x2(v[2 * t + 1]),
                    from_e4m3x2(v[2 * t + 1] >> 16), pb[t][0], pb[t][1]);
        }
      }
      __syncwarp();
      if (alive && at < count) {
        issue(s);
        ++issued;
      }
      cp_async_commit();
    }

    b = e;
    if (b < count) {  // the next unit's queries come while this one's pieces are joined
      advance(here, len);
      load_q();
    }
    // ---- the warps' pieces joined; in round r warp w joins tile r JOINERS + w ----
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, x);
      l1 += __shfl_xor_sync(0xffffffffu, l1, x);
    }
    if (g == 0) {
      ml_s[warp][2 * c4][0] = m0, ml_s[warp][2 * c4][1] = l0;
      ml_s[warp][2 * c4 + 1][0] = m1, ml_s[warp][2 * c4 + 1][1] = l1;
    }
    const bool whole_unit = len == blocks;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (first_piece ? 0 : 1);
    float f0[kDecWarps], f1[kDecWarps], M0 = -INFINITY, M1 = -INFINITY, L0 = 0.f, L1 = 0.f;
#pragma unroll
    for (int round = 0; round < 2; ++round) {
#pragma unroll
      for (int c = 0; c < JOINERS; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k) rec[warp][c][k][lane] = o[round * JOINERS + c][k];
      __syncthreads();
      if (warp < JOINERS) {
        if (round == 0) {
#pragma unroll
          for (int w = 0; w < kDecWarps; ++w) {
            f0[w] = ml_s[w][2 * c4][0], f1[w] = ml_s[w][2 * c4 + 1][0];
            M0 = fmaxf(M0, f0[w]);
            M1 = fmaxf(M1, f1[w]);
          }
#pragma unroll
          for (int w = 0; w < kDecWarps; ++w) {
            f0[w] = f0[w] == -INFINITY ? 0.f : exp2_fast(f0[w] - M0);
            f1[w] = f1[w] == -INFINITY ? 0.f : exp2_fast(f1[w] - M1);
            L0 = fmaf(ml_s[w][2 * c4][1], f0[w], L0);
            L1 = fmaf(ml_s[w][2 * c4 + 1][1], f1[w], L1);
          }
        }
        float r[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w)
#pragma unroll
          for (int k = 0; k < 4; ++k) r[k] = fmaf(rec[w][warp][k][lane], (k & 1) ? f1[w] : f0[w], r[k]);
        // dims 16 c + 2 g (r[0], r[1]) and + 1 (r[2], r[3]) of heads 2 c4, 2 c4 + 1
        const int c = round * JOINERS + warp;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int head = 2 * c4 + x, dim = 16 * c + 2 * g;
          if (head >= a.G) continue;
          if (whole_unit) {
            const float inv = sq.len == 0 ? 0.f : 1.f / (x ? L1 : L0);
            T* op = static_cast<T*>(a.out) + (int64_t)sq.row * a.ldo + (int64_t)(kh * a.G + head) * D + dim;
            if (d.vec_o) {
              *reinterpret_cast<uint32_t*>(op) = Elem<T>::pack(r[x] * inv, r[2 + x] * inv);
            } else {
              op[0] = Elem<T>::from(r[x] * inv);
              op[1] = Elem<T>::from(r[2 + x] * inv);
            }
          } else {
            *reinterpret_cast<float2*>(d.parts + (slot * kDecHeads + head) * D + dim) = make_float2(r[x], r[2 + x]);
            if (c == 0 && g == 0) d.parts_ml[slot * kDecHeads + head] = make_float2(x ? M1 : M0, x ? L1 : L0);
          }
        }
      }
      __syncthreads();  // (the records are written again)
    }
    first_piece = false;
  }
  // no copy is under way when the CTA leaves
  cp_async_wait<0>();
  if (lane == 0) {
    for (int i = consumed; i < issued; ++i)
      mbar_wait(smem_u32(&bars_s[warp][i % kDecStages]), (uint32_t)((i / kDecStages) & 1), a.err, SITE_KV8_PIPE);
  }
}

// The workspace: the line, where stretches begin, pieces' maxima and sums, pieces; then the chunks'.
struct Space {
  int64_t starts, ml, parts, chunks, bytes;
};
Space space_of(int head_dim, int max_rows) {
  const int64_t slots = 2ll * kDecWaves * kDecPerSm * num_sms();
  Space s;
  s.starts = 256;
  s.ml = s.starts + up256(slots / 2 * sizeof(DecStart));
  s.parts = s.ml + up256(slots * kDecHeads * 8);
  s.chunks = s.parts + up256(slots * kDecHeads * head_dim * 4);
  s.bytes = s.chunks + (max_rows > 1 ? kv8_chunk_space(head_dim) : 0);
  return s;
}

int check_batch(const sar_kv8_batch& b, const sar_kv8* c) {
  if (!c) return set_error(SAR_ERR_INVALID_ARG, "kv8_attention: null cache");
  SAR_TRY(check_kv8(c, "kv8_attention"));
  if (b.rows < 0 || b.n < 0 || b.n_q_heads < 1 || b.max_rows < 1 || b.max_len < 0 || b.window < 0)
    return set_error(SAR_ERR_INVALID_ARG, "kv8_attention: bad sizes");
  if (b.n_q_heads % c->n_kv_heads || b.n_q_heads / c->n_kv_heads > kDecHeads)
    return set_error(SAR_ERR_UNSUPPORTED, "kv8_attention: query heads are a multiple of the KV heads, at most 8 to each");
  if (b.rows > 1 << 27 || b.n > 1 << 30 || c->n_kv_heads > 1024)
    return set_error(SAR_ERR_UNSUPPORTED, "kv8_attention: rows, sequences or heads above their limits");
  return SAR_OK;
}

// blocks: of the line at most, where the longest sequence is as long as the caller says;
// chunks: workspace of the sequences of several rows, null where there are none.
template <typename T, int D>
int launch_kv8(const DecArgs& d, int64_t blocks, void* chunks, const CUtensorMap& tmk, const CUtensorMap& tmv, cudaStream_t s) {
  const int storage = Elem<T>::kMmaFormat == 1 ? SAR_STORAGE_BF16 : SAR_STORAGE_F16;
  const int smem = 1024 + kDecWarps * kDecStages * 2 * kDecKeys * D;
  SAR_TRY(ensure_smem_attr(reinterpret_cast<const void*>(&kv8_decode_kernel<T, D>), smem, "kv8 decode: set smem attribute"));
  const int grid = d.units ? d.a.n * d.a.kvh : blocks >= (int64_t)d.resident * kDecMany ? kDecWaves * d.resident : d.resident;
  cudaError_t e = launch_pdl(kv8_decode_kernel<T, D>, dim3(grid), dim3(kDecWarps * 32), (size_t)smem, s, tmk, tmv, d);
  if (e != cudaSuccess) return cuda_error(e, "kv8 decode launch");
  count_launches(1);
  // (the chunks' kernel comes before the joins, so that it can start beside this one)
  // one kernel joins what either leaves in pieces
  Kv8Pieces p = {};
  if (!d.units) p.line = d.line, p.starts = d.starts, p.parts = d.parts, p.parts_ml = d.parts_ml;
  if (chunks) SAR_TRY(launch_kv8_chunks(d.a, D, storage, chunks, &p, s));
  if (!d.units || chunks) SAR_TRY(launch_kv8_join(d.a, D, storage, p, grid, s));
  return SAR_OK;
}

}  // namespace
}  // namespace sar

using sar::aligned_to;
using sar::set_error;

extern "C" {

int sar_kv8_attention_workspace(const sar_kv8_batch* batch, const sar_kv8* cache, int64_t* bytes) try {
  if (!batch || !bytes) return set_error(SAR_ERR_INVALID_ARG, "kv8_attention_workspace: null pointer");
  SAR_TRY(sar::check_batch(*batch, cache));
  *bytes = sar::space_of(cache->head_dim, batch->max_rows).bytes;
  return SAR_OK;
} catch (...) {
  return sar::entry_failed("kv8_attention_workspace");
}

int sar_kv8_attention(const sar_kv8_batch* batch, const sar_kv8* cache, void* stream) try {
  if (!batch) return set_error(SAR_ERR_INVALID_ARG, "kv8_attention: null batch");
  const sar_kv8_batch& b = *batch;
  SAR_TRY(sar::check_batch(b, cache));
  if (b.storage != SAR_STORAGE_F16 && b.storage != SAR_STORAGE_BF16)
    return set_error(SAR_ERR_INVALID_ARG, "kv8_attention: bad storage");
  if (!(b.scale >= 0.f && b.scale < INFINITY)) return set_error(SAR_ERR_INVALID_ARG, "kv8_attention: bad scale");
  if (b.rows == 0 || b.n == 0) return SAR_OK;
  if (!b.q || !b.out || !b.row_offsets || !b.lens || !b.block_tables || !b.workspace)
    return set_error(SAR_ERR_INVALID_ARG, "kv8_attention: null pointer");
  const int64_t width = (int64_t)b.n_q_heads * cache->head_dim;
  if (b.ldq < width || b.ldo < width || b.bt_stride < 1 || b.bt_cols < 0 || b.bt_cols > b.bt_stride)
    return set_error(SAR_ERR_INVALID_ARG, "kv8_attention: rows shorter than their heads, or no block table");
  // (256: the blocks looked up ahead of a sequence's end)
  if ((int64_t)b.bt_stride * cache->page_size > INT32_MAX - 256)
    return set_error(SAR_ERR_UNSUPPORTED, "kv8_attention: block tables above 2^31 tokens");
  if (!aligned_to(b.q, 2) || !aligned_to(b.out, 2) || !aligned_to(b.row_offsets, 4) || !aligned_to(b.lens, 4) ||
      !aligned_to(b.block_tables, 4) || !aligned_to(b.workspace, 16))
    return set_error(SAR_ERR_INVALID_ARG, "kv8_attention: array not aligned to its element");
  const sar::Space sp = sar::space_of(cache->head_dim, b.max_rows);
  if (b.workspace_bytes < sp.bytes) return set_error(SAR_ERR_INVALID_ARG, "kv8_attention: workspace too small");
  sar::DecArgs d = {};
  sar::Kv8Attn& a = d.a;
  a.q = b.q;
  a.out = b.out;
  a.ldq = b.ldq;
  a.ldo = b.ldo;
  a.off = b.row_offsets;
  a.lens = b.lens;
  a.bt = b.block_tables;
  a.bt_stride = b.bt_stride;
  a.bt_cols = b.bt_cols > 0 ? b.bt_cols : b.bt_stride;
  a.k_scales = cache->k_scales;
  a.v_scales = cache->v_scales;
  a.k_codes = static_cast<const uint8_t*>(cache->k_codes);
  a.v_codes = static_cast<const uint8_t*>(cache->v_codes);
  a.rows = b.rows;
  a.n = b.n;
  a.qh = b.n_q_heads;
  a.kvh = cache->n_kv_heads;
  a.G = a.qh / a.kvh;
  a.shift = cache->page_size == 16 ? 4 : cache->page_size == 32 ? 5 : 6;
  a.num_pages = cache->num_pages;
  a.max_rows = b.max_rows;
  a.window = b.window;
  a.scale = (b.scale == 0.f ? (float)(1.0 / sqrt((double)cache->head_dim)) : b.scale) * 1.4426950408889634f;
  SAR_TRY(sar::op_flags(&a.err));
  uint8_t* ws = static_cast<uint8_t*>(b.workspace);
  d.line = reinterpret_cast<sar::DecLine*>(ws);
  d.starts = reinterpret_cast<sar::DecStart*>(ws + sp.starts);
  d.parts_ml = reinterpret_cast<float2*>(ws + sp.ml);
  d.parts = reinterpret_cast<float*>(ws + sp.parts);
  // (max_len and the tables' width only guide how work is shared out)
  const int64_t longest = b.max_len > 0 ? b.max_len : a.bt_cols * cache->page_size;
  const int64_t most = (b.window > 0 ? std::min<int64_t>(longest, b.window) : longest) / sar::kDecKeys + 2;
  const int64_t blocks = most * b.n * cache->n_kv_heads;
  d.resident = sar::kDecPerSm * sar::num_sms();
  void* chunks = b.max_rows == 1 || b.rows == 1 ? nullptr : ws + sp.chunks;
  const int64_t units = (int64_t)b.n * cache->n_kv_heads;
  d.units = most <= sar::kDecFew + 2 || (!chunks && most <= sar::kDecUnit + 2 && units >= sar::kDecUnits);
  d.units = d.units && units <= 1 << 20;
  d.vec_q = aligned_to(b.q, 16) && b.ldq % 8 == 0;
  d.vec_o = aligned_to(b.out, 4) && b.ldo % 2 == 0;
  // the codes as rows of 128 bytes (one key, or two of 64 dims), boxes of up to 32 keys of a page
  CUtensorMap tmk, tmv;
  const uint64_t map_rows = (uint64_t)a.num_pages * a.kvh * cache->page_size * cache->head_dim / 128;
  const uint32_t box = (uint32_t)(std::min(cache->page_size, sar::kDecKeys) * cache->head_dim / 128);
  SAR_TRY(sar::make_tmap_bytes(&tmk, cache->k_codes, map_rows, 128, box));
  SAR_TRY(sar::make_tmap_bytes(&tmv, cache->v_codes, map_rows, 128, box));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf = b.storage == SAR_STORAGE_BF16;
  int rc;
  if (cache->head_dim == 128)
    rc = bf ? sar::launch_kv8<__nv_bfloat16, 128>(d, blocks, chunks, tmk, tmv, s) : sar::launch_kv8<__half, 128>(d, blocks, chunks, tmk, tmv, s);
  else
    rc = bf ? sar::launch_kv8<__nv_bfloat16, 64>(d, blocks, chunks, tmk, tmv, s) : sar::launch_kv8<__half, 64>(d, blocks, chunks, tmk, tmv, s);
  return rc;
} catch (...) {
  return sar::entry_failed("kv8_attention");
}

}  // extern "C"
