// Attention of sequences with several rows over the 8-bit paged cache, on the
// 5th-generation tensor cores.
//
// A unit is 256 (row, query head) pairs of one sequence and KV head, packed row by
// row, so that a chunk of a few tokens wastes no tensor rows on absent ones and every
// key is converted once for the whole group; pairs [0, 128) are tile A, the rest B.
//   warps 0..7   softmax, four per tile, a row to a thread: scores S from tensor memory,
//                running maximum and sum, P (fp16) back over S; O rescaled where a row's
//                maximum has grown by more than 2^8; at the end O / sum.
//   warps 13, 14 fetch pages' codes by TMA: K's as they are multiplied, V's 64 keys a step.
//   warps 8..11  convert V's from e4m3 to fp16 (exactly) into two stages of 128 keys.
//   warp 12      one thread issues S_x(j) = Q_x K_j^T and O_x += P_x(j) V_j, the tiles in
//                turn, so that one tile's products run under the other's softmax.
// K is multiplied in e4m3 as it lies in the cache (a conversion took the place of the
// tensor cores as what bounds this kernel).  A query is then a sum of e4m3 numbers:
// scaled by a power of two so that its row's largest lies in [128, 256), two parts of
// four significant bits hold bf16's eight, three fp16's eleven, off by 2^-10 at most;
// e4m3 products run at twice the rate, so two parts cost what one fp16 product does.
// Page scales act as in the single-token kernel: with raw scores S and
// t = S k_scale scale + log2(v_scale), 2^(t - m) weighs V's codes and its sum takes it
// times 1 / v_scale, 16 keys (which lie in one page) at a time: one multiplication
// more per 16 keys and row.
//
// NaN codes of V count as zero in the product, where they would reach rows that do not
// see their key; the blocks that have any are marked, and at a piece's end its rows look through
// those of their keys that they see (a NaN under 64 rows 200000 deep: 131 us; 2650 when
// they looked through all of the piece's, 114 without a NaN).
//
// Value scales far apart would lose the weights of the smaller: pages far from most are passed
// over by the loop and follow at the piece's end (8192 rows 495 us; 541 when they were taken in the loop).
//
// Units' blocks of 128 keys form one line.  Every CTA (one per SM) takes an equal stretch of
// it, or every unit gets as many CTAs, or a CTA a whole unit, whichever should end first;
// pieces of a unit are joined by the kernel behind (attn_kv8_join.cu).  With four or more
// units to an SM a CTA always takes a whole one, the longest of a sequence first.
//
// Bound by a tile's chain (its Q K^T, its softmax, its P V, and the handing over, about
// 2 us for a block's two tiles), which the two tiles hide from one another in part, and by
// a piece's queries and results, as long as some blocks.  8192 rows of 32 heads, bf16:
// 495 us, 1.11 PFLOP/s; 512 rows 16384 deep, f16, beside five single tokens: 162 us, 0.84
// PFLOP/s; 25 chunks of up to 6 rows in a window of 1024 keys, beside seven: 34 us.
// Taken at an earlier state: steps of 64 keys with two buffers of scores, so that a tile's
// next product does not wait for its softmax (666 for 554 us and 195 for 172: products 64
// columns wide run at half the rate); both tiles on the same 128 pairs, where there are no
// more, with the blocks in turn (180 for 171 us; 42.5 for 43.7 with 25 short chunks).
// The loop over blocks is sensitive to what else is in the function: with a piece's
// results and the search for NaN out of line the first took 510 us, with all in line 554,
// with the queries out of line too 669; with a warp of their own for the scales 623.
#include <algorithm>

#include "kv8.cuh"
#include "tc05.cuh"

namespace sar {

namespace {

constexpr int kKeys = 128;               // keys of a block
constexpr int kSoftWarps = 8, kConvWarps = 4;
constexpr int kChunkThreads = (kSoftWarps + kConvWarps + 4) * 32;  // (whole warpgroups: the last has one warp at work)
constexpr int kTileRegion = 128 * 128;   // [128 rows][128 bytes]: 64 dims of 128 rows
constexpr int kScaleRing = 4;             // blocks whose scales are kept: three K stages ahead, and the softmax's
constexpr int kScaleFloats = 28;         // of a block: eight runs' factors, log2 and inverse of the value scales, a flag
constexpr int kPieceRing = 4;            // pieces that are known at once: scales are fetched three blocks ahead, V's codes turned two
constexpr int kMarks = 512;              // of a piece's blocks, for one or some of which each stands
constexpr int kRawSteps = 3;              // steps of 64 keys of V whose codes are under way
constexpr int kMostK = 3;                 // K stages
constexpr int kLeastBlocks = 4;          // of a stretch
constexpr int kPieceBlocks = 12;         // a CTA's second piece takes as long as so many blocks more (four chunks of up to
                                         // 512 rows 90 us; 106 where 8 or 5 are reckoned; others alike)
constexpr uint32_t kApartBits = 8u << 23; // of two numbers a factor of 1 / kApart from one another
constexpr uint32_t kColsS = 128;         // S_x at x * 128; P over its last 64 columns
constexpr uint32_t kColsO = 256;         // O_x at 256 + x * 128

struct ChunkBars {
  uint64_t k_full[kMostK], k_free[kMostK], v_full[2], v_free[2];
  uint64_t raw_full[kRawSteps], raw_free[kRawSteps];
  uint64_t s_full[2], p_full[2];
  uint64_t q_ready, mma_done;
  uint32_t tmem;
  uint32_t read[kScaleRing];  // runs of a block whose V was read
  uint32_t nan[kPieceRing];   // a piece's number + 1, where V has NaN codes
  uint32_t apart[kPieceRing]; // ... where value scales lie far from most
  uint32_t odd[kPieceRing];   // ... where either
  float low[kPieceRing];      // the least scale of those that the loop over blocks weighs
};

struct ChunkArgs8 {
  Kv8Attn a;
  ChunkPlan* plan;
  float* parts;      // [2 * SMs][D / 4][256][4]
  float2* parts_ml;  // [2 * SMs][256]
  int sms, vec_q, vec_o;
};

template <typename T, int D>
struct ChunkSmem {
  static constexpr int kParts = Elem<T>::kMmaFormat == 1 ? 2 : 3;  // e4m3 numbers to a query's element
  static constexpr int kPart = 128 * D;                            // of 128 rows
  static constexpr int kStagesK = kParts == 2 ? 3 : 2;
  static constexpr int kStageV = (D / 64) * kTileRegion;           // fp16
  static constexpr int kRawStep = 64 * D;
  static constexpr int kK = 2 * kParts * kPart, kV = kK + kStagesK * kPart, kRaw = kV + 2 * kStageV;
  static constexpr int kBars = kRaw + kRawSteps * kRawStep;
  static constexpr int kScales = kBars + 288;
  static constexpr int kTable = kScales + kScaleRing * kScaleFloats * 4;  // before [tiles + 1], seq, u
  static constexpr int kNan = kTable + (3 * kMostTiles + 1) * 4;  // [pieces][marks] bytes
  static constexpr int kBytes = 1024 + kNan + kPieceRing * kMarks;
};
static_assert(sizeof(ChunkBars) <= 288, "barrier area");
static_assert(ChunkSmem<__half, 128>::kBytes <= 226 * 1024, "shared memory per CTA");

// Instruction descriptor: fp32 sums, M = 128; both operands of format 0 (fp16 of
// kind::f16, e4m3 of kind::f8f6f4), A K-major, B K-major or MN-major.
__device__ __forceinline__ uint32_t idesc_of(int n, uint32_t b_mn) {
  return (1u << 4) | (b_mn << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// D (+)= A B^T over K = 32 of e4m3.
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Descriptor of a K-major operand whose rows are D bytes, with a swizzle as wide.
template <int D>
__device__ __forceinline__ uint64_t rows_desc(uint32_t saddr) {
  if constexpr (D == 128) return sw128_desc(saddr);
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)(512 >> 4) << 32;  // eight rows
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)4 << 61;  // 64-byte swizzle
  return d;
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* err) {
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(smem_u32(bar), parity, err, SITE_KV8_PIPE) ? 1 : 0;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();
  return ok != 0;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 of_pair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void sts_u4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// (rows * G stays below 2^30)
__device__ __forceinline__ int tiles_of(int rows, int G) { return rows < 2 ? 0 : (rows * G + 255) >> 8; }

// Tile u of a sequence: its pairs, and the blocks of 128 keys that they see.
struct Tile {
  int pair0;           // its first pair
  int pairs;           // up to 256
  int j0, j1, j1a;     // blocks [j0, j1), of which tile A's pairs end at j1a
  int lo;              // the oldest key that any row sees
};
__device__ __forceinline__ Tile tile_of(const Kv8Attn& a, int rows, int len, int u) {
  Tile t;
  t.pair0 = u * 256;
  t.pairs = min(256, rows * a.G - t.pair0);
  const unsigned G = a.G;
  const int first = len - rows + (int)((unsigned)t.pair0 / G);
  const int last = len - rows + (int)((unsigned)(t.pair0 + t.pairs - 1) / G);
  const int last_a = len - rows + (int)((unsigned)(t.pair0 + min(t.pairs, 128) - 1) / G);
  // (rows in front of the sequence see nothing; their positions less a window may pass 32 bits)
  t.lo = a.window > 0 ? max(0, max(first, -1) - a.window + 1) : 0;
  t.j0 = t.lo / kKeys;
  t.j1 = max(last, 0) / kKeys + 1;
  t.j1a = max(last_a, 0) / kKeys + 1;
  return t;
}

// 16-byte chunk c of a row of a warp's queries, or of its 16-bit results: a part's chunks
// after another's, swizzled as the product reads the queries.
template <typename T, int D>
__device__ __forceinline__ uint32_t chunk_at(uint32_t base, int row, int c) {
  const int k = c % (D / 16);
  return base + (uint32_t)(c / (D / 16) * ChunkSmem<T, D>::kPart + row * D + ((D == 128 ? k ^ (row & 7) : k ^ (row >> 1 & 3)) << 4));
}
// A warp's 32 rows of queries, pairs pair0 on of which `live` are the unit's, as sums of
// e4m3 numbers.  The rows come into the place of their own first two parts, all under way
// together, and are turned there, a row's eight dims to a lane (with a row to a thread
// and two loads at a time a unit's queries took 10 us: 2048 rows of a prompt 286 us for 217
// when its units were cut evenly).
// Returns what the row of this lane's scores is to be multiplied by.
template <typename T, int D>
__device__ __forceinline__ float chunk_queries(const ChunkArgs8& args, uint32_t base, int row0, int kh, int pair0, int live) {
  using M = ChunkSmem<T, D>;
  constexpr int CHUNKS = D / 8, STEP_ROWS = 32 / CHUNKS;
  const Kv8Attn& a = args.a;
  const int lane = threadIdx.x & 31, ch = lane % CHUNKS, of_step = lane / CHUNKS;
#pragma unroll 1
  for (int i = 0; i < CHUNKS; ++i) {
    const int row = i * STEP_ROWS + of_step;
    const uint32_t to = chunk_at<T, D>(base, row, ch);
    if (row >= live) {
      sts_u4(to, 0, 0, 0, 0);
      continue;
    }
    const unsigned of = (unsigned)(pair0 + row), tok = of / (unsigned)a.G;
    const T* qp = static_cast<const T*>(a.q) + (int64_t)(row0 + (int)tok) * a.ldq + (int64_t)(kh * a.G + (int)(of - tok * a.G)) * D + 8 * ch;
    if (args.vec_q) {
      cp_async16(to, qp, 16);
    } else {
      const unsigned short* h = reinterpret_cast<const unsigned short*>(qp);
      sts_u4(to, h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16, h[4] | (uint32_t)h[5] << 16, h[6] | (uint32_t)h[7] << 16);
    }
  }
  cp_async_commit();
  cp_async_wait<0>();
  __syncwarp();
  float fac = a.scale;
#pragma unroll 1
  for (int i = 0; i < CHUNKS; ++i) {
    const uint4 v = lds_u4(chunk_at<T, D>(base, i * STEP_ROWS + of_step, ch));
    float f[8] = {Elem<T>::lo(v.x), Elem<T>::hi(v.x), Elem<T>::lo(v.y), Elem<T>::hi(v.y),
                  Elem<T>::lo(v.z), Elem<T>::hi(v.z), Elem<T>::lo(v.w), Elem<T>::hi(v.w)};
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
#pragma unroll
    for (int o = CHUNKS / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // (powers whose inverse is a normal number too)
    const uint32_t ex = min(max(__float_as_uint(m) >> 23, 10u), 253u);
    const float of_lane = __shfl_sync(0xffffffffu, __uint_as_float((ex - 7) << 23), lane % STEP_ROWS * CHUNKS);
    if (lane / STEP_ROWS == i) fac = a.scale * of_lane;
    const float inv = __uint_as_float((261u - ex) << 23);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= inv;
    const uint32_t at = chunk_at<T, D>(base, i * STEP_ROWS + of_step, ch >> 1) + (ch & 1) * 8;
    __syncwarp();  // (the rows have been read)
#pragma unroll
    for (int k = 0; k < M::kParts; ++k) {
      uint32_t u[2];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t code = k == 0 ? to_e4m3x2(f[2 * e], f[2 * e + 1]) : finite_e4m3x2(f[2 * e], f[2 * e + 1]);
        const float2 g = e4m3x2_floats(code);
        f[2 * e] -= g.x, f[2 * e + 1] -= g.y;
        u[e >> 1] = e & 1 ? u[e >> 1] | code << 16 : code;
      }
      asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at + (uint32_t)(k * M::kPart)), "r"(u[0]), "r"(u[1]) : "memory");
    }
  }
  return fac;
}
// Block j's mark among those of a piece of nb blocks; what marks it: stamps of a place's pieces
// differ for so long that an old one costs time alone.
__device__ __forceinline__ int mark_of(int j, int nb) { return nb <= kMarks ? j : (int)((int64_t)j * kMarks / nb); }
__device__ __forceinline__ uint8_t stamp_of(uint32_t piece) { return (uint8_t)(piece / kPieceRing % 255 + 1); }
// NaN into O in the dims in which a value is NaN under a key of [lo, pos], of the piece's marked
// blocks.  The lanes look through four keys of a block each and tell one another of those that have any.
template <int D>
__device__ __noinline__ void nan_into(const Kv8Attn& a, uint32_t ocol, const uint8_t* marks, uint32_t stamp, int seq, int len, int kh,
                                      int ja, int nb, int lo, int pos) {
  const int lane = threadIdx.x & 31, n = min(nb, kMarks);
  uint32_t nan[D / 32] = {};
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += 32) {
#pragma unroll 1
    for (uint32_t set = __ballot_sync(0xffffffffu, i0 + lane < n && marks[i0 + lane] == stamp); set; set &= set - 1) {
      const int64_t i = i0 + __ffs(set) - 1;  // it stands for blocks [i nb / n, (i + 1) nb / n), rounded up
      const int k1 = (ja + (int)(((i + 1) * nb + n - 1) / n)) * kKeys;
#pragma unroll 1
      for (int k0 = (ja + (int)((i * nb + n - 1) / n)) * kKeys; k0 < k1; k0 += 32) {
        const int key = k0 + lane;
        const int g = key < len ? a.bt[(int64_t)seq * a.bt_stride + (key >> a.shift)] : -1;
        uint32_t mine[D / 32] = {}, any = 0;
        if (g >= 0 && g < a.num_pages) {
          const uint8_t* c = a.v_codes + ((((int64_t)g * a.kvh + kh) << a.shift) + (key & ((1 << a.shift) - 1))) * D;
#pragma unroll
          for (int k = 0; k < D / 4; ++k) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(c + 4 * k);
            const uint32_t m = (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
            mine[k >> 3] |= ((m & 1) | (m >> 7 & 2) | (m >> 14 & 4) | (m >> 21 & 8)) << ((k & 7) * 4);
            any |= m;
          }
        }
        for (uint32_t have = __ballot_sync(0xffffffffu, any != 0); have; have &= have - 1) {
          const int from = __ffs(have) - 1;
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            const uint32_t bits = __shfl_sync(0xffffffffu, mine[k], from);
            if (k0 + from >= lo && k0 + from <= pos) nan[k] |= bits;
          }
        }
      }
    }
  }
#pragma unroll
  for (int c = 0; c < D; c += 16) {
    const uint32_t bits = nan[c >> 5] >> (c & 16);
    uint32_t u[16];
    tmem_ld16(ocol + c, u);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (bits >> e & 1) u[e] = 0x7fc00000u;
    tmem_st16(ocol + c, u);
  }
  tmem_wait_st();
}
// The page of a run of 16 keys, -1 where the call reads none of the page's keys or it is out of range.
__device__ __forceinline__ int run_page(const Kv8Attn& a, int seq, int len, int key, int oldest) {
  const int ps = 1 << a.shift, first = key & ~(ps - 1);
  const int page = first < len && first + ps > oldest ? a.bt[(int64_t)seq * a.bt_stride + (key >> a.shift)] : -1;
  return page < a.num_pages ? page : -1;
}
// The least value scale of a piece that the loop over its blocks weighs, 2^-4 of the median of 32
// pages' (its power of two; page: this lane's): one page of a large scale does not send all others
// the slow way.  (Out of line: 512 rows 16384 deep 162 us, 174 with it in the loads' warp.)
__device__ __noinline__ float usual_scales(const Kv8Attn& a, int page, int kh) {
  const int ex = page >= 0 ? (int)(__float_as_uint(a.v_scales[(int64_t)page * a.kvh + kh]) >> 23) : -1;
  const int half = (__popc(__ballot_sync(0xffffffffu, ex >= 0)) + 1) / 2;
  int e = 0;  // the largest exponent that at least half of the pages reach
#pragma unroll 1
  for (int bit = 128; bit > 0; bit >>= 1)
    if (half > 0 && __popc(__ballot_sync(0xffffffffu, ex >= (e | bit))) >= half) e |= bit;
  return __uint_as_float((uint32_t)min(max(e - 4, 1), 246) << 23);
}
// Runs of 16 keys whose pages' value scales are far from most pages' (less than low, or more than
// low / kApart): the loop over a piece's blocks passes over them, and here they follow, with weights
// in fp32.  O has the products of all blocks; returns the row's maximum and sum with these keys'.
// q: where the warp's queries lie, whose scores are to be multiplied by fac.  Slow (a run 23 us, a block of eight in the loop 2), for scales that a model's values hardly ever have.
template <typename T, int D>
__device__ __noinline__ float2 runs_apart(const Kv8Attn& a, uint32_t q, float fac, uint32_t ocol, float low, int seq, int len, int kh, int ja,
                                          int jb, int oldest, int lo, int pos, float m, float l) {
  using M = ChunkSmem<T, D>;
  const int lane = threadIdx.x & 31, ps = 1 << a.shift;
#pragma unroll 1
  for (int j0 = ja; j0 < jb; j0 += 4) {  // a run of four blocks' to a lane
    const int j = j0 + lane / 8, key = j * kKeys + lane % 8 * 16;
    const int page = j < jb ? run_page(a, seq, len, key, oldest) : -1;
    float ks = 0.f, vs = low;
    if (page >= 0) ks = a.k_scales[(int64_t)page * a.kvh + kh], vs = a.v_scales[(int64_t)page * a.kvh + kh];
#pragma unroll 1
    for (uint32_t runs = __ballot_sync(0xffffffffu, __float_as_uint(vs) - __float_as_uint(low) > kApartBits); runs; runs &= runs - 1) {
      const int from = __ffs(runs) - 1, k0 = __shfl_sync(0xffffffffu, key, from);
      const int64_t unit = (int64_t)__shfl_sync(0xffffffffu, page, from) * a.kvh + kh;
      const int64_t codes = ((unit << a.shift) + (k0 & (ps - 1))) * D;
      const float f = fmaxf(__shfl_sync(0xffffffffu, ks, from) * fac, 1.2e-38f), v_scale = __shfl_sync(0xffffffffu, vs, from);
      const float off = log2_fast(v_scale), iv = rcp_fast(v_scale);
      float w[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) w[e] = 0.f;
#pragma unroll 1
      for (int c = 0; c < D / 16; ++c) {
        float x[16] = {};
#pragma unroll
        for (int k = 0; k < M::kParts; ++k) {
          const uint4 v = lds_u4(chunk_at<T, D>(q, lane, c) + (uint32_t)(k * M::kPart));
          const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float2 u = e4m3x2_floats(words[i >> 2] >> (8 * (i & 2)));
            x[i] += u.x, x[i + 1] += u.y;
          }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint4 v = *reinterpret_cast<const uint4*>(a.k_codes + codes + e * D + c * 16);
          const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float2 u = e4m3x2_floats(words[i >> 2] >> (8 * (i & 2)));
            w[e] = fmaf(x[i], u.x, fmaf(x[i + 1], u.y, w[e]));
          }
        }
      }
      float top_w = m;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        w[e] = k0 + e >= lo && k0 + e <= pos ? fmaf(w[e], f, off) : -INFINITY;
        top_w = fmaxf(top_w, w[e]);
      }
      const float grown = top_w == -INFINITY ? 1.f : exp2_fast(m - top_w);  // (0 from -inf)
      m = top_w;
      const float ref = m == -INFINITY ? 0.f : m - kBias;
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        w[e] = exp2_fast(w[e] - ref);
        sum += w[e];
      }
      l = fmaf(sum, iv, l * grown);
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t u[16];
        float o[16];
        tmem_ld16(ocol + c, u);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __uint_as_float(u[i]) * grown;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint4 v = *reinterpret_cast<const uint4*>(a.v_codes + codes + e * D + c);
          const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float2 x = e4m3x2_floats(words[i >> 2] >> (8 * (i & 2)));
            // (NaN codes as zero, as in the product)
            o[i] = fmaf(w[e], x.x == x.x ? x.x : 0.f, o[i]);
            o[i + 1] = fmaf(w[e], x.y == x.y ? x.y : 0.f, o[i + 1]);
          }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(o[i]);
        tmem_st16(ocol + c, u);
      }
      tmem_wait_st();
    }
  }
  return make_float2(m, l);
}
// A row of O times inv, in 16 bits, row by row through the place of the warp's own
// queries' first two parts (other warps may be at the next piece already).
template <typename T, int D>
__device__ __noinline__ void chunk_rows_out(const ChunkArgs8& args, uint32_t ocol, uint32_t base, float inv, int64_t to,
                                            int live) {
  constexpr int CHUNKS = D / 8, STEP_ROWS = 32 / CHUNKS;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    float o[32];
    tmem_ld32(ocol + c, *reinterpret_cast<uint32_t(*)[32]>(o));
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; e += 8)
      sts_u4(chunk_at<T, D>(base, lane, (c + e) >> 3), Elem<T>::pack(o[e] * inv, o[e + 1] * inv), Elem<T>::pack(o[e + 2] * inv, o[e + 3] * inv),
             Elem<T>::pack(o[e + 4] * inv, o[e + 5] * inv), Elem<T>::pack(o[e + 6] * inv, o[e + 7] * inv));
  }
  __syncwarp();
#pragma unroll 4
  for (int i = 0; i < CHUNKS; ++i) {
    const int row = i * STEP_ROWS + lane / CHUNKS, ch = lane % CHUNKS;
    const int64_t of = __shfl_sync(0xffffffffu, to, row);
    const uint4 v = lds_u4(chunk_at<T, D>(base, row, ch));
    if (row >= live) continue;
    T* op = static_cast<T*>(args.a.out) + of + 8 * ch;
    if (args.vec_o) {
      *reinterpret_cast<uint4*>(op) = v;
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) reinterpret_cast<unsigned short*>(op)[e] = (unsigned short)(w[e >> 1] >> (16 * (e & 1)));
    }
  }
  __syncwarp();
}
// A row of O as it is, four dims of all of a unit's rows next to one another.
template <int D>
__device__ __noinline__ void chunk_piece_out(const ChunkArgs8& args, uint32_t ocol, int64_t slot, int row) {
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    float o[32];
    tmem_ld32(ocol + c, *reinterpret_cast<uint32_t(*)[32]>(o));
    tmem_wait_ld();
    float4* pp = reinterpret_cast<float4*>(args.parts) + (slot * (D / 4) + c / 4) * 256 + row;
#pragma unroll
    for (int e = 0; e < 8; ++e) pp[e * 256] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kChunkThreads, 1)
    kv8_chunk_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                     const __grid_constant__ ChunkArgs8 args) {
  using M = ChunkSmem<T, D>;
  constexpr int PASS = kConvWarps * 32 * 16 / D;  // keys of a pass of the converting warps, 16 bytes to a thread
  constexpr int STEP_PASSES = 64 / PASS;
  const Kv8Attn& a = args.a;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto q_reg = [&](int x) { return sbase + (uint32_t)(x * M::kParts * M::kPart); };
  auto k_reg = [&](int s) { return sbase + (uint32_t)(M::kK + s * M::kPart); };
  auto v_reg = [&](int s) { return sbase + (uint32_t)(M::kV + s * M::kStageV); };
  ChunkBars* bars = reinterpret_cast<ChunkBars*>(smem + M::kBars);
  float* scales = reinterpret_cast<float*>(smem + M::kScales);
  int32_t* before = reinterpret_cast<int32_t*>(smem + M::kTable);
  int32_t* t_seq = before + kMostTiles + 1;
  int32_t* t_u = t_seq + kMostTiles;
  __shared__ int64_t sums[kChunkThreads / 32];
  __shared__ int first_s[2], most_s, least_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  for (int i = threadIdx.x; i < kPieceRing * kMarks; i += kChunkThreads) smem[M::kNan + i] = 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMostK; ++s) {
      mbar_init(smem_u32(&bars->k_full[s]), 1);
      mbar_init(smem_u32(&bars->k_free[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&bars->v_full[s]), kConvWarps);
      mbar_init(smem_u32(&bars->v_free[s]), 1);
      mbar_init(smem_u32(&bars->s_full[s]), 1);
      mbar_init(smem_u32(&bars->p_full[s]), kSoftWarps / 2);
    }
    for (int s = 0; s < kRawSteps; ++s) {
      mbar_init(smem_u32(&bars->raw_full[s]), 1);
      mbar_init(smem_u32(&bars->raw_free[s]), kConvWarps);
    }
    mbar_init(smem_u32(&bars->q_ready), kSoftWarps);
    mbar_init(smem_u32(&bars->mma_done), 1);
    for (int s = 0; s < kPieceRing; ++s) bars->nan[s] = bars->apart[s] = bars->odd[s] = 0;
    most_s = 0;
    least_s = 1 << 30;
    fence_mbar_init();
  }
  // Launched right behind the single tokens' kernel, which has waited for what came
  // before it when it lets this one start, and whose results this one does not read:
  // only the last CTA waits for it, so that the kernels behind see both complete.
  pdl_launch_dependents();
  const bool waits = blockIdx.x == gridDim.x - 1;

  // ---- the plan: tiles of every sequence, then this CTA's stretch or unit ----
  auto block_sum = [&](int64_t v, int64_t& total) -> int64_t {  // exclusive
    int64_t incl = v;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    total = 0;
#pragma unroll 1
    for (int w = 0; w < kChunkThreads / 32; ++w) {
      if (w < warp) incl += sums[w];
      total += sums[w];
    }
    return incl - v;
  };
  const int per = (int)(((unsigned)a.n + kChunkThreads - 1) / kChunkThreads);
  const int i0 = min(a.n, (int)threadIdx.x * per), i1 = min(a.n, i0 + per);
  int64_t nt = 0, at0 = 0, all64 = 0;
  bool stretches = false;
  // twice over this thread's sequences: to count their tiles, then to find its own or list them
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {
    int64_t t = at0;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      int r0, rows, len;
      const int k = kv8_sequence(a, i, r0, rows, len) ? tiles_of(rows, a.G) : 0;
      if (round && stretches) {
        for (int u = 0; u < k; ++u) t_seq[t + u] = i, t_u[t + u] = u;
      } else if (round && blockIdx.x / (unsigned)a.kvh >= t && blockIdx.x / (unsigned)a.kvh < t + k) {
        first_s[0] = i;
        first_s[1] = k - 1 - (int)(blockIdx.x / (unsigned)a.kvh - t);  // (the longest first)
      }
      t += k;
    }
    if (round == 0) {
      at0 = block_sum(t, nt);
      // (a line's blocks, as many as the block tables allow, stay within 32 bits)
      stretches = nt <= kMostTiles && nt * a.kvh < 4 * args.sms &&
                  nt * a.kvh * (((a.bt_cols << a.shift) / kKeys) + 1) < (1 << 30);
    }
  }
  __syncthreads();
  int b0 = 0, b1 = 1;
  if (stretches) {
    int blocks = 0;
    int row0 = 0, rows = 0, len = 0;
    Tile tl = {};
    if (threadIdx.x < nt) {
      kv8_sequence(a, t_seq[threadIdx.x], row0, rows, len);
      tl = tile_of(a, rows, len, t_u[threadIdx.x]);
      blocks = tl.j1 - tl.j0;
      atomicMax(&most_s, blocks);
      atomicMin(&least_s, blocks);
    }
    const int64_t at = block_sum(blocks, all64);
    const int all = (int)(all64 * a.kvh), units = (int)nt * a.kvh, most = most_s;
    int C = max(1, min(args.sms, all / kLeastBlocks));
    // Times in blocks: an equal stretch, with the pieces of as short units as there are ...
    const int even = all / C, P = kPieceBlocks;
    int best = even + P * (even / max(1, least_s) + 1), each = 0;
    // ... the same number of CTAs to each unit, where these are alike (within a quarter), so
    // that a CTA has one piece although some SMs stay idle (512 rows 2048 deep 58 us, 73 cut
    // evenly; 256 rows 16384 deep 104 and 115; three unlike ones of 33 to 100 rows 3000 to
    // 1000 deep 54 and 49) ...
    if (units > 0 && units <= args.sms && (int64_t)most * units <= all + all / 4) {
      const int k = min(args.sms / units, max(1, most / kLeastBlocks));
      if (most / k <= even + P) each = k, best = min(best, most / k + P);
    }
    // ... and a unit to a CTA, the last ones, which are a sequence's longest, first (2048
    // rows of a prompt 75 us, 286 cut evenly; 16384 deep 480 and 463)
    if (units > 0) {
      const int rounds = (units + args.sms - 1) / args.sms;
      if (min(rounds * most, even + (most + 1) / 2) + P * rounds < best && (units > args.sms || most + P < best)) each = 1;
    }
    if (each > 0) C = each * units;
    if (threadIdx.x < nt) {
      before[threadIdx.x] = (int)at;
      if (blockIdx.x == 0) {
        args.plan->tile[threadIdx.x] = {(int)at, row0, len - rows, tl.pair0, tl.pairs};
      }
    }
    if (threadIdx.x == 0) {
      before[nt] = (int)all64;
      if (blockIdx.x == 0) {
        args.plan->tile[nt].before = (int)all64;
        args.plan->all = all;
        args.plan->each = each;
        args.plan->ctas = C;
        args.plan->tiles = (int)nt;
      }
    }
    __syncthreads();
    if (all == 0 || blockIdx.x >= (unsigned)C) {
      if (waits) pdl_wait();
      return;
    }
    if (each > 0) {
      const int from = (int)(blockIdx.x / (unsigned)each), part = (int)blockIdx.x - from * each;
      const int unit = each == 1 ? units - 1 - from : from;
      const int t = (int)((unsigned)unit / (unsigned)a.kvh), kh = unit - t * a.kvh;
      const int nb = before[t + 1] - before[t], u0 = before[t] * a.kvh + kh * nb, parts = min(each, nb);
      if (part >= parts) {
        if (waits) pdl_wait();
        return;
      }
      b0 = u0 + line_at(nb, part, parts);
      b1 = u0 + line_at(nb, part + 1, parts);
    } else {
      b0 = line_at(all, blockIdx.x, C);
      b1 = line_at(all, blockIdx.x + 1, C);
    }
  } else {
    if (blockIdx.x == 0 && threadIdx.x == 0) args.plan->all = 0;
    if (blockIdx.x >= nt * a.kvh) {
      if (waits) pdl_wait();
      return;
    }
  }

  // A piece: blocks [ja, jb) of one unit.
  struct Piece {
    int seq, kh, row0, rows, len, ja, jb, na;  // na: blocks of tile A
    Tile t;
    int next;
    bool whole;
  };
  auto piece_at = [&](int b) -> Piece {
    Piece p;
    int u, o = 0, nb = 0;
    if (stretches) {
      int lo = 0, hi = (int)nt;
#pragma unroll 1
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before[mid] * a.kvh <= b)
          lo = mid;
        else
          hi = mid;
      }
      p.seq = t_seq[lo];
      u = t_u[lo];
      nb = before[lo + 1] - before[lo];
      o = b - before[lo] * a.kvh;
      p.kh = (int)((unsigned)o / (unsigned)nb);
      o -= p.kh * nb;
    } else {
      p.seq = first_s[0];
      u = first_s[1];
      p.kh = (int)(blockIdx.x % (unsigned)a.kvh);
    }
    kv8_sequence(a, p.seq, p.row0, p.rows, p.len);
    p.t = tile_of(a, p.rows, p.len, u);
    p.ja = p.t.j0 + o;
    p.jb = stretches ? p.t.j0 + min(nb, o + (b1 - b)) : p.t.j1;
    p.whole = p.ja == p.t.j0 && p.jb == p.t.j1;
    p.next = stretches ? b + (p.jb - p.ja) : b1;
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

  // Registers: 512 threads start with 128 each; 56 for the products' and loads' warpgroup and
  // 72 for the converting one leave 192 for the softmax (256 * 192 + 128 * 72 + 128 * 56 = 512 * 128).
  if (warp >= kSoftWarps + kConvWarps) {
    // ---------------- products ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == kSoftWarps + kConvWarps && elect_one()) {
      const uint32_t id_s = idesc_of(kKeys, 0), id_pv = idesc_of(D, 1);
      const uint64_t dqa = rows_desc<D>(q_reg(0)), dk = rows_desc<D>(k_reg(0));
      const uint64_t dv0 = sw128_desc_mn(v_reg(0), kTileRegion, 1024);
      bool ok = true;
      uint32_t base = 0, done_a = 0, done_b = 0, pieces = 0;  // blocks so far: of the stages, of each tile
      for (int b = b0; b < b1; ++pieces) {
        const Piece p = piece_at(b);
        const int nb = p.jb - p.ja;
        const bool has_b = p.t.pairs > 128;
        if (ok) ok = mbar_wait(smem_u32(&bars->q_ready), pieces & 1, a.err, SITE_KV8_PIPE);
        tc_fence_after();
        // S_x(j); the last tile to read the block frees its K stage
        auto issue_s = [&](int x, int j) -> bool {
          const uint32_t jt = base + j, s = jt % M::kStagesK;
          const bool first = x == 0 || j >= p.na, last = x == 1 || !has_b;
          if (first && !mbar_wait(smem_u32(&bars->k_full[s]), (jt / M::kStagesK) & 1, a.err, SITE_KV8_PIPE)) return false;
          tc_fence_after();
          const uint32_t d = tmem + kColsS * (uint32_t)x;
          const uint64_t db = dk + s * (M::kPart / 16), dq = dqa + (uint32_t)x * (M::kParts * M::kPart / 16);
#pragma unroll
          for (int kk = 0; kk < M::kParts * (D / 32); ++kk)
            mma_f8(d, dq + (uint64_t)(kk / (D / 32) * (M::kPart / 16) + kk % (D / 32) * 2), db + (uint64_t)(kk % (D / 32) * 2), id_s,
                   kk != 0);
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
          const uint32_t pcol = tmem + kColsS * (uint32_t)x + 64, dO = tmem + kColsO + kColsS * (uint32_t)x;
          const uint64_t dv = dv0 + s * (M::kStageV / 16);
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            mma_f16_ts(dO, pcol + kk * 8, dv + (uint64_t)(kk * (16 * 128 / 16)), id_pv, (j > 0 || kk > 0) ? 1u : 0u);
          if (last) mma_commit(smem_u32(&bars->v_free[s]));
          return true;
        };
        // S_A(0), S_B(0), then P_A V(j - 1), S_A(j), P_B V(j - 1), S_B(j)
#pragma unroll 1
        for (int k = 0; k <= 2 * nb + 1 && ok; ++k) {
          const int j = k >> 1, x = k & 1, last = x ? (has_b ? nb : 0) : p.na;
          if (j > 0 && j <= last) ok = issue_pv(x, j - 1);
          if (ok && j < last) ok = issue_s(x, j);
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
    if (warp == kSoftWarps + kConvWarps + 1 || warp == kSoftWarps + kConvWarps + 2) {
      // ---------------- codes to shared memory: K's, V's ----------------
      // Lanes 0..7 know the pages (and the K warp's the scales) of a block's eight runs of 16
      // keys, looked up ahead; boxes are whole pages.
      const bool is_k = warp == kSoftWarps + kConvWarps + 1;
      const CUtensorMap* map = is_k ? &tmk : &tmv;
      const int ps = 1 << a.shift, run = lane & 7;
      const uint32_t firsts = ps == 16 ? 0xffu : ps == 32 ? 0x55u : 0x11u;  // the runs that boxes begin with
      bool ok = true;
      uint32_t jt = 0, pieces = 0;
      if (lane == 0) tma_prefetch_desc(map);
      for (int b = b0; b < b1 && ok; ++pieces) {
        const Piece p = piece_at(b);
        const int nb = p.jb - p.ja;
        b = p.next;
        // whether the call reads of the run's page, and the page
        auto wanted = [&](int j) -> bool {
          const int first = ((p.ja + j) * kKeys + run * 16) & ~(ps - 1);
          return j < nb && first < p.len && first + ps > p.t.lo;
        };
        auto look_up = [&](int j) -> int {
          return wanted(j) ? a.bt[(int64_t)p.seq * a.bt_stride + (((p.ja + j) * kKeys + run * 16) >> a.shift)] : -1;
        };
        // scales of the block behind the present one, pages of two: no load is waited for
        int next = look_up(0), next2 = look_up(1);
        const int sample = is_k ? run_page(a, p.seq, p.len, (p.ja + (int)((int64_t)nb * lane / 32)) * kKeys + lane % 8 * 16, p.t.lo) : -1;
        float ks_next, vs_next;
        auto scales_of = [&](int g) {
          ks_next = vs_next = 1.f;
          if (is_k && g >= 0 && g < a.num_pages) {
            ks_next = a.k_scales[(int64_t)g * a.kvh + p.kh];
            vs_next = a.v_scales[(int64_t)g * a.kvh + p.kh];
          }
        };
        scales_of(next);
        float low = 0.f;  // pages of value scales within [low, low / kApart] are weighed in the loop
        if (is_k) low = usual_scales(a, sample, p.kh);
        for (int j = 0; j < nb && ok; ++j, ++jt) {
          int page = next;
          const float ks = ks_next, vs = vs_next;
          const bool lost = wanted(j) && (page < 0 || page >= a.num_pages);
          if (lost) {
            if (is_k && lane < 8) report(a.err, SAR_ERR_BOUNDS, SITE_KV8_PAGE, page);
            page = -1;
          }
          next = next2;
          next2 = look_up(j + 2);
          scales_of(next);
          const uint32_t pages = __ballot_sync(0xffffffffu, page >= 0) & 0xffu, boxes = pages & firsts;
          // (rows of the maps are as long as a key's)
          const int row = (int)(((int64_t)page * a.kvh + p.kh) << a.shift);
          int y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, row, i);
          if (is_k) {
            const uint32_t s = jt % M::kStagesK, bar = smem_u32(&bars->k_full[s]);
            // (few instructions: all roles' loops contend for the instruction cache)
            const bool apart = page >= 0 && __float_as_uint(vs) - __float_as_uint(low) > kApartBits;
            const bool over = __any_sync(0xffffffffu, lost || apart);
            ok = warp_wait(&bars->k_free[s], ((jt / M::kStagesK) & 1) ^ 1, a.err);
            if (!ok) break;
            if (lane < 8) {
              float* sc = scales + (jt % kScaleRing) * kScaleFloats + lane;
              if (lane == 0) sc[24] = over ? 1.f : 0.f;
              if (apart) {
                bars->apart[pieces % kPieceRing] = bars->odd[pieces % kPieceRing] = pieces + 1;
                bars->low[pieces % kPieceRing] = low;
              }
              sc[0] = lost || apart ? -1.f : ks;  // negative: keys that are passed over
              sc[8] = log2_fast(vs);
              sc[16] = rcp_fast(vs);
            }
            __syncwarp();
            if (elect_one()) {
              if (boxes)
                mbar_expect_tx(bar, (uint32_t)__popc(boxes) * (uint32_t)(ps * D));
              else
                mbar_arrive(bar);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (boxes >> i & 1) tma_load_2d(k_reg(0) + s * M::kPart + i * (16 * D), map, 0, y[i], bar);
            }
            __syncwarp();
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t st = 2 * jt + h, slot = st % kRawSteps, bar = smem_u32(&bars->raw_full[slot]);
              if (ok) ok = warp_wait(&bars->raw_free[slot], ((st / kRawSteps) & 1) ^ 1, a.err);
              if (!ok) break;
              if (elect_one()) {
                if (h == 0) bars->read[jt % kScaleRing] = pages;
                const uint32_t half = boxes >> (4 * h) & 15;
                if (half)
                  mbar_expect_tx(bar, (uint32_t)__popc(half) * (uint32_t)(ps * D));
                else
                  mbar_arrive(bar);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (half >> i & 1)
                    tma_load_2d(sbase + (uint32_t)M::kRaw + slot * M::kRawStep + i * (16 * D), map, 0, y[4 * h + i], bar);
              }
              __syncwarp();
            }
          }
        }
      }
      // no copy is under way when the CTA leaves
      if (lane == 0) {
        const uint32_t stages = is_k ? M::kStagesK : kRawSteps, n = is_k ? jt : 2 * jt;
        for (uint32_t i = n > stages ? n - stages : 0; i < n; ++i)
          mbar_wait(smem_u32(is_k ? &bars->k_full[i % stages] : &bars->raw_full[i % stages]), (i / stages) & 1, a.err, SITE_KV8_PIPE);
      }
    }
    __syncwarp();
  } else if (warp >= kSoftWarps) {
    // ---------------- codes to fp16 ----------------
    // Steps of 64 keys of V, 16 bytes of a key to a thread, consecutive bytes to
    // consecutive threads.  head_dim 128: lanes of the second half of a key write their
    // two chunks the other way round, so that eight lanes touch every bank once.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const int t = threadIdx.x - kSoftWarps * 32;
    const int c4 = t & 3, half = D == 128 ? (t >> 2) & 1 : 0, rin = D == 128 ? t >> 3 : t >> 2;
    bool ok = true;
    uint32_t jt = 0, pieces = 0;
    for (int b = b0; b < b1 && ok; ++pieces) {
      const Piece p = piece_at(b);
      b = p.next;
#pragma unroll 1
      for (int k = 2 * p.ja; k < 2 * p.jb; ++k) {  // steps of the sequence
        const uint32_t s = jt & 1, st = 2 * jt + (k & 1), slot = st % kRawSteps;
        if (!(k & 1)) ok = warp_wait(&bars->v_free[s], ((jt >> 1) & 1) ^ 1, a.err);
        if (ok) ok = warp_wait(&bars->raw_full[slot], (st / kRawSteps) & 1, a.err);
        if (!ok) break;
        uint4 w[STEP_PASSES];
#pragma unroll
        for (int i = 0; i < STEP_PASSES; ++i)
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                       : "r"(sbase + (uint32_t)(M::kRaw + slot * M::kRawStep + i * (kConvWarps * 512) + t * 16)));
        // codes of keys behind the end, and of pages that were not read, count as zero
        const uint32_t read = bars->read[jt % kScaleRing] >> (4 * (k & 1)) & 15;
        if (k * 64 + 64 > p.len || read != 15) {
#pragma unroll
          for (int i = 0; i < STEP_PASSES; ++i) {
            const int key = i * PASS + rin;
            if (k * 64 + key >= p.len || !(read >> (key >> 4) & 1)) w[i] = make_uint4(0, 0, 0, 0);
          }
        }
        const uint32_t dst = v_reg(s) + (uint32_t)(half * kTileRegion);
        __half2 nan = __floats2half2_rn(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < STEP_PASSES; ++i) {
          const int row = (k & 1) * 64 + i * PASS + rin;
          const uint32_t h[8] = {from_e4m3x2(w[i].x), from_e4m3x2(w[i].x >> 16), from_e4m3x2(w[i].y), from_e4m3x2(w[i].y >> 16),
                                 from_e4m3x2(w[i].z), from_e4m3x2(w[i].z >> 16), from_e4m3x2(w[i].w), from_e4m3x2(w[i].w >> 16)};
#pragma unroll
          for (int e = 0; e < 8; ++e) nan = __hfma2(*reinterpret_cast<const __half2*>(&h[e]), __floats2half2_rn(0.f, 0.f), nan);
          const uint32_t at = dst + (uint32_t)(row * 128), c0 = (uint32_t)(((2 * c4) ^ (row & 7)) << 4), c1 = c0 ^ 16;
          sts_u4(at + (half ? c1 : c0), half ? h[4] : h[0], half ? h[5] : h[1], half ? h[6] : h[2], half ? h[7] : h[3]);
          sts_u4(at + (half ? c0 : c1), half ? h[0] : h[4], half ? h[1] : h[5], half ? h[2] : h[6], half ? h[3] : h[7]);
        }
        if (!(__low2float(nan) == 0.f && __high2float(nan) == 0.f)) {
          // NaN codes: zero, and known to have been there
          bars->nan[pieces % kPieceRing] = bars->odd[pieces % kPieceRing] = pieces + 1;
          smem[M::kNan + pieces % kPieceRing * kMarks + mark_of((k >> 1) - p.ja, p.jb - p.ja)] = stamp_of(pieces);
#pragma unroll 1
          for (int i = 0; i < STEP_PASSES * 8; ++i) {
            const int row = (k & 1) * 64 + (i >> 3) * PASS + rin;
            const uint32_t at = dst + (uint32_t)(row * 128 + (((2 * c4 + (i >> 2 & 1)) ^ (row & 7)) << 4) + (i & 3) * 4);
            uint32_t x;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(at));
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(pack_f16(f.x == f.x ? f.x : 0.f, f.y == f.y ? f.y : 0.f)) : "memory");
          }
        }
        if (k & 1) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // visible to the tensor core
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&bars->raw_free[slot]));
          if (k & 1) mbar_arrive(smem_u32(&bars->v_full[s]));
        }
        jt += k & 1;
      }
    }
    __syncwarp();
  } else {
    // ---------------- softmax: a row to a thread ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int x = warp >> 2, qq = warp & 3;
    const int r = qq * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(qq * 32) << 16);
    const uint32_t scol = lane_base + kColsS * (uint32_t)x, ocol = lane_base + kColsO + kColsS * (uint32_t)x;
    bool alive = true;  // false once a wait gave up
    uint32_t base = 0, mine_done = 0, pieces = 0;
    for (int b = b0; b < b1; ++pieces) {
      const Piece p = piece_at(b);
      const int nb = x == 0 ? p.na : p.t.pairs > 128 ? p.jb - p.ja : 0;
      const bool valid = x * 128 + r < p.t.pairs;
      const unsigned pair = valid ? p.t.pair0 + x * 128 + r : 0u;
      const int token = (int)(pair / (unsigned)a.G), head = p.kh * a.G + (int)(pair % (unsigned)a.G);
      const int pos = valid ? p.len - p.rows + token : -1;  // keys (pos - window, pos] are seen
      const int lo = a.window > 0 ? max(pos, -1) - a.window + 1 : 0;
      const float fac = chunk_queries<T, D>(args, q_reg(x) + (uint32_t)(qq * 32 * D), p.row0, p.kh, p.t.pair0 + x * 128 + qq * 32,
                                            p.t.pairs - x * 128 - qq * 32);
      {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();  // (the piece before's O has been read)
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->q_ready));
      }

      float m_used = -INFINITY, l = 0.f;
      for (int j = 0; j < nb && alive; ++j) {
        // (every lane polls: a broadcast costs the chain of a block's steps its latency)
        alive = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->s_full[x]), (mine_done + j) & 1, a.err, SITE_KV8_PIPE));
        if (!alive) break;
        tc_fence_after();
        // (loops that are not unrolled: six roles' code contends for the instruction cache)
        const int key0 = (p.ja + j) * kKeys;
        const uint32_t sc = sbase + (uint32_t)(M::kScales + ((base + j) % kScaleRing) * (kScaleFloats * 4));
        const bool lost = lds_f4(sc + 96).x != 0.f;
        if (__any_sync(0xffffffffu, key0 + kKeys - 1 > pos || key0 < lo || lost)) {
          // keys that this row does not see, and pages out of range: -inf, in tensor memory
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const int k0 = key0 + 32 * c;  // bit e: key k0 + e is seen
            uint32_t seen = pos < k0 ? 0u : pos - k0 >= 31 ? 0xffffffffu : (2u << (pos - k0)) - 1;
            seen &= lo <= k0 ? 0xffffffffu : lo - k0 > 31 ? 0u : 0xffffffffu << (lo - k0);
            if (lost) {
              const float4 k4 = lds_f4(sc + (c >> 1) * 16);
              if ((c & 1 ? k4.z : k4.x) < 0.f) seen &= 0xffff0000u;
              if ((c & 1 ? k4.w : k4.y) < 0.f) seen &= 0xffffu;
            }
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t u[16];
              tmem_ld16(scol + c * 32 + h * 16, u);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (!(seen >> (16 * h + e) & 1)) u[e] = 0xff800000u;
              tmem_st16(scol + c * 32 + h * 16, u);
            }
          }
          tmem_wait_st();
        }
        // (a factor is above zero, where -inf times it would be NaN)
        auto factor = [&](float k) { return fmaxf(fabsf(k) * fac, 1.2e-38f); };
        float sv[64], first[64];  // keys 64 .. 127, and those before
        tmem_ld32(scol, reinterpret_cast<uint32_t*>(first));
        tmem_ld32(scol + 32, reinterpret_cast<uint32_t*>(first) + 32);
        tmem_ld32(scol + 64, reinterpret_cast<uint32_t*>(sv));
        tmem_ld32(scol + 96, reinterpret_cast<uint32_t*>(sv) + 32);
        float4 k4 = lds_f4(sc + 16), lv4 = lds_f4(sc + 48);
        float pm = -INFINITY;
        auto largest = [&](const float* x, const float4& k, const float4& lv) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            // (three to an instruction, in two chains)
            float x0 = x[g * 16], x1 = x[g * 16 + 1];
#pragma unroll
            for (int e = 2; e < 14; e += 4) {
              x0 = fmaxf(fmaxf(x0, x[g * 16 + e]), x[g * 16 + e + 1]);
              x1 = fmaxf(fmaxf(x1, x[g * 16 + e + 2]), x[g * 16 + e + 3]);
            }
            x0 = fmaxf(fmaxf(x0, x[g * 16 + 14]), x[g * 16 + 15]);
            pm = fmaxf(pm, fmaf(fmaxf(x0, x1), factor(g == 0 ? k.x : g == 1 ? k.y : g == 2 ? k.z : k.w),
                                g == 0 ? lv.x : g == 1 ? lv.y : g == 2 ? lv.z : lv.w));
          }
        };
        {
          const float4 k0 = lds_f4(sc), lv0 = lds_f4(sc + 32);
          tmem_wait_ld();
          largest(first, k0, lv0);
        }
        largest(sv, k4, lv4);
        const float m_new = fmaxf(m_used, pm);
        const bool need = m_new > m_used + kGrowth;
        // P_x(j - 1) V has landed before S_x(j), which was issued behind it
        if (__any_sync(0xffffffffu, need)) {
          const float rs = need ? exp2_fast(m_used - m_new) : 1.f;  // 0 while m_used is -inf
          if (__any_sync(0xffffffffu, need && m_used != -INFINITY)) {
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t u[16];
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
        const float ref = m_used == -INFINITY ? 0.f : m_used - kBias;
        // P lies over the scores' upper half
        auto weigh = [&](const float* x, int c, const float4& k, const float4& lv) {
          const float4 iv = lds_f4(sc + 64 + c * 16);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t u[16];
#pragma unroll
            for (int gg = 0; gg < 2; ++gg) {
              const int g = 2 * h + gg;
              const float f = factor(g == 0 ? k.x : g == 1 ? k.y : g == 2 ? k.z : k.w);
              const float off = (g == 0 ? lv.x : g == 1 ? lv.y : g == 2 ? lv.z : lv.w) - ref;
              const uint64_t f2 = pair_of(f, f), off2 = pair_of(off, off);
              uint64_t ls[2] = {0, 0};
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 t = of_pair(fma_pair(pair_of(x[g * 16 + 2 * e], x[g * 16 + 2 * e + 1]), f2, off2));
                const float p0 = exp2_fast(t.x), p1 = exp2_fast(t.y);
                ls[e & 1] = add_pair(ls[e & 1], pair_of(p0, p1));
                u[gg * 8 + e] = pack_f16(p0, p1);
              }
              const float2 sum = of_pair(add_pair(ls[0], ls[1]));
              l = fmaf(sum.x + sum.y, g == 0 ? iv.x : g == 1 ? iv.y : g == 2 ? iv.z : iv.w, l);
            }
            tmem_st16(scol + 64 + c * 32 + h * 16, u);
          }
        };
        weigh(sv, 1, k4, lv4);
        k4 = lds_f4(sc);
        lv4 = lds_f4(sc + 32);
        weigh(first, 0, k4, lv4);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[x]));
      }
      // ---- O / sum, or the piece as it is ----
      if (alive) alive = warp_wait(&bars->mma_done, pieces & 1, a.err);
      if (alive && x * 128 < p.t.pairs) {
        tc_fence_after();
        // (the places are this piece's until the warps that write them are four ahead, and those wait for this one's rows)
        const uint32_t place = pieces % kPieceRing;
        if (nb > 0 && *reinterpret_cast<volatile uint32_t*>(&bars->odd[place]) == pieces + 1) {
          if (*reinterpret_cast<volatile uint32_t*>(&bars->apart[place]) == pieces + 1) {
            const float2 ml = runs_apart<T, D>(a, q_reg(x) + (uint32_t)(qq * 32 * D), fac, ocol, bars->low[place], p.seq, p.len, p.kh, p.ja, p.jb,
                                               p.t.lo, lo, pos, m_used, l);
            m_used = ml.x;
            l = ml.y;
          }
          if (*reinterpret_cast<volatile uint32_t*>(&bars->nan[place]) == pieces + 1)
            nan_into<D>(a, ocol, smem + M::kNan + place * kMarks, stamp_of(pieces), p.seq, p.len, p.kh, p.ja, p.jb - p.ja, lo, pos);
        }
        __syncwarp();
        const int64_t slot = 2 * (int64_t)blockIdx.x + (pieces == 0 ? 0 : 1);
        // (a row that sees keys and has no sum is NaN)
        const float inv = pos < 0 ? 0.f : 1.f / l;
        if (!p.whole) args.parts_ml[slot * 256 + x * 128 + r] = make_float2(m_used, l);
        const int64_t to = (int64_t)(p.row0 + token) * a.ldo + (int64_t)head * D;
        if (p.whole)
          chunk_rows_out<T, D>(args, ocol, q_reg(x) + (uint32_t)(qq * 32 * D), inv, to, p.t.pairs - x * 128 - qq * 32);
        else if (nb > 0)
          chunk_piece_out<D>(args, ocol, slot, x * 128 + r);
      }
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
  if (waits) pdl_wait();
}

template <typename T, int D>
int launch_chunk8(const ChunkArgs8& c, const CUtensorMap& tmk, const CUtensorMap& tmv, cudaStream_t s) {
  const int smem = ChunkSmem<T, D>::kBytes;
  SAR_TRY(ensure_smem_attr(reinterpret_cast<const void*>(&kv8_chunk_kernel<T, D>), smem, "kv8 chunk: set smem attribute"));
  // as many CTAs as units can come to, one per SM at least
  const int64_t pairs = (int64_t)c.a.rows * c.a.G;
  const int64_t tiles = pairs / 256 + std::min(c.a.n, c.a.rows / 2);
  const int64_t grid = std::max(tiles * c.a.kvh, (int64_t)c.sms);
  if (grid > INT32_MAX) return set_error(SAR_ERR_UNSUPPORTED, "kv8_attention: more than 2^31 units");
  cudaError_t e = launch_pdl(kv8_chunk_kernel<T, D>, dim3((unsigned)grid), dim3(kChunkThreads), (size_t)smem, s, tmk, tmv, c);
  if (e != cudaSuccess) return cuda_error(e, "kv8 chunk launch");
  count_launches(1);
  return SAR_OK;
}
}  // namespace

int64_t kv8_chunk_space(int head_dim) {
  const int64_t slots = 2ll * num_sms() * 256;
  return up256(sizeof(ChunkPlan)) + up256(slots * 8) + slots * head_dim * 4;
}

static ChunkArgs8 chunk_args(const Kv8Attn& a, void* space) {
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
  return c;
}

int launch_kv8_chunks(const Kv8Attn& a, int head_dim, int storage, void* space, Kv8Pieces* p, cudaStream_t s) {
  const ChunkArgs8 c = chunk_args(a, space);
  p->plan = c.plan;
  p->chunk_parts = c.parts;
  p->chunk_parts_ml = c.parts_ml;
  // the codes as rows of head_dim bytes, a page to a box: K swizzled as the product reads it
  CUtensorMap k, v;
  const uint64_t map_rows = (uint64_t)a.num_pages * a.kvh << a.shift;
  SAR_TRY(make_tmap_rows8(&k, a.k_codes, map_rows, head_dim, 1u << a.shift, true));
  SAR_TRY(make_tmap_rows8(&v, a.v_codes, map_rows, head_dim, 1u << a.shift, false));
  const bool bf = storage == SAR_STORAGE_BF16;
  if (head_dim == 128) return bf ? launch_chunk8<__nv_bfloat16, 128>(c, k, v, s) : launch_chunk8<__half, 128>(c, k, v, s);
  return bf ? launch_chunk8<__nv_bfloat16, 64>(c, k, v, s) : launch_chunk8<__half, 64>(c, k, v, s);
}

}  // namespace sar
