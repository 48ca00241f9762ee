// The 8-bit KV cache on the device: where codes lie, and e4m3 in and out.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace sar {

// Exponents of a page's scale.  Between them attention's weights, which carry a
// page's value scale in their exponent, stay inside fp32's range; magnitudes of at most
// 2^-10 of a page's scale become zero (2^-50 under the least), those over 448 * 2^60 saturate.
constexpr int kKv8Least = -40, kKv8Most = 60;

// Attention weighs V's codes by 2^(t - m), t = S k_scale scale + log2(v_scale) and m near the
// largest t so far (its growth by 2^kGrowth is tolerated before m follows), in fp16.  fp16's
// subnormal numbers are off by 2^-25, so the weights lie 2^kBias higher: up to 2^15, where fp16 ends
// at 2^16, and off by 2^-32 of 2^m.  A page of a small value scale beside larger ones
// has small weights for large probabilities: pages whose scales lie within a factor of
// 1 / kApart are weighed together (off by 2^-24 of the row's largest probability), others apart.
constexpr float kGrowth = 8.f, kBias = 7.f, kApart = 1.f / 256.f;

// The smallest power of two s within those exponents with a <= 448 s, for a finite
// a >= 0: 448 = 1.75 * 2^8.
__device__ __forceinline__ float kv8_scale(float a) {
  const uint32_t u = __float_as_uint(a);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = min(max(e, kKv8Least), kKv8Most);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Two values to e4m3, nearest even, at most 448 in magnitude; NaN stays NaN.
__device__ __forceinline__ uint32_t finite_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// The same; infinities become NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  return finite_e4m3x2(fabsf(lo) == INFINITY ? NAN : lo, fabsf(hi) == INFINITY ? NAN : hi);
}

// 2^x by the SFU (relative error 2^-22; 2^-inf = 0): a weight that is rounded to
// fp16 next.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A scale's logarithm and inverse by the SFU (relative error 2^-22): both are factors of a
// weight that is rounded to fp16.
__device__ __forceinline__ float log2_fast(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 lds_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// Two e4m3 codes (the low 16 bits) as fp16, exactly.
__device__ __forceinline__ uint32_t from_e4m3x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_floats(uint32_t codes) {
  const uint32_t h = from_e4m3x2(codes);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A call's batch (pointers as in sar_kv8_batch) for the attention kernels.
struct Kv8Attn {
  const void* q;
  void* out;
  int64_t ldq, ldo;
  const int32_t* off;
  const int32_t* lens;
  const int32_t* bt;
  int64_t bt_stride, bt_cols;  // a table's place, and the pages that it holds
  const float* k_scales;
  const float* v_scales;
  const uint8_t* k_codes;
  const uint8_t* v_codes;
  int rows, n, qh, kvh, G, shift, num_pages, max_rows, window;
  float scale;  // of the scores, times log2(e): softmax in base 2
  int* err;
};

// Sequence i's rows and length; false where the call leaves it out.
__device__ __forceinline__ bool kv8_sequence(const Kv8Attn& a, int i, int& row0, int& rows, int& len) {
  row0 = a.off[i];
  const int row1 = a.off[i + 1];
  len = a.lens[i];
  rows = row1 - row0;
  return row0 >= 0 && row1 >= row0 && row1 <= a.rows && rows <= a.max_rows && len >= 0 &&
         len <= (a.bt_cols << a.shift);
}

// ---- how single tokens' work is cut (attn_kv8.cu), for the kernel that joins it ----
constexpr int kDecHeads = 8;    // query heads of a KV head: the products' columns
constexpr int kDecLeast = 4;    // blocks of a CTA's stretch at least, where there are so few
constexpr int kDecWaves = 2;    // CTAs to a place on an SM, where there are
constexpr int kDecMany = 256;   // so many blocks to a place

// Where a CTA's stretch begins inside a unit: that unit (seq < 0: it does not).
struct DecStart {
  int64_t u0;      // the unit's first block on the line
  int32_t blocks;  // of the unit
  int32_t seq, kh, row;
};
// How the line is cut.  SMs are not equally near to the memory that their keys lie in:
// of CTAs with equal stretches the last ended 25% after the median.  So the
// resident CTAs take equal shares of the line's first 7/8, and as many more
// share the rest, each started as a place on an SM gets free (128 sequences of up to 8192
// keys 174 us, 181 in equal stretches).
struct DecLine {
  int64_t all, head;  // blocks; those of the first CTAs
  int32_t first, ctas;
  __device__ __forceinline__ static int64_t quotient(int64_t x, int64_t y) {
    // (64-bit divisions are long; these are made before anything is loaded)
    return x >> 32 == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
  }
  __device__ __forceinline__ static DecLine of(int64_t all, int resident, int grid) {
    DecLine l;
    l.all = all;
    const bool many = all >= (int64_t)resident * kDecMany && grid >= kDecWaves * resident;
    l.first = many ? resident : (int)max((int64_t)1, min((int64_t)min(resident, grid), all / kDecLeast));
    l.ctas = many ? kDecWaves * resident : l.first;
    l.head = many ? all - all / 8 : all;
    return l;
  }
  // CTA c's first block, and the CTA that has block b
  __device__ __forceinline__ int64_t at(int c) const {
    return c <= first ? quotient(head * c, first) : head + quotient((all - head) * (c - first), ctas - first);
  }
  __device__ __forceinline__ int cta(int64_t b) const {
    return (int)(b < head ? quotient((b + 1) * first - 1, head) : first + quotient((b - head + 1) * (ctas - first) - 1, all - head));
  }
};

// ---- how the work of sequences of several rows is cut (attn_kv8_chunk.cu) ----
constexpr int kMostTiles = 256;  // of a call whose CTAs take stretches

// The plan, in the workspace, for the joining kernel: tiles of 256 (row, head) pairs.
struct ChunkPlan {
  int32_t all;   // blocks on the line; 0: nothing to join
  int32_t each;  // CTAs to a unit; 0: equal stretches of the line, of ctas CTAs
  int32_t ctas, tiles;
  struct {
    int32_t before;  // blocks of the tiles before, of a KV head
    int32_t row0, past, pair0, pairs;  // the sequence's first row, its tokens before that; the tile's pairs
  } tile[kMostTiles + 1];
};
// CTA c of C has blocks [line(c), line(c + 1)) of the line, or of the unit of each = C.
__device__ __forceinline__ int line_at(int all, int c, int C) { return (int)((int64_t)all * c / C); }

// What the joining kernel takes (attn_kv8_join.cu): single tokens' pieces, where line is
// not null, and the chunks', where plan is not.
struct Kv8Pieces {
  const DecLine* line;
  const DecStart* starts;   // [CTAs]
  const float* parts;       // [2 * CTAs][8][D]: a CTA's first and last piece
  const float2* parts_ml;   // [2 * CTAs][8] maximum and sum
  const ChunkPlan* plan;
  const float* chunk_parts;      // [2 * SMs][D / 4][256][4]
  const float2* chunk_parts_ml;  // [2 * SMs][256]
  int dec_blocks, vec_o;
};

inline int64_t up256(int64_t x) { return (x + 255) & ~int64_t(255); }

// Sequences of several rows (attn_kv8_chunk.cu): the workspace that they take, and their
// kernel, launched right behind the single tokens'; it adds its pieces to p.
int64_t kv8_chunk_space(int head_dim);
int launch_kv8_chunks(const Kv8Attn& a, int head_dim, int storage, void* space, Kv8Pieces* p, cudaStream_t s);
// Joins both kernels' pieces; dec_ctas: of the single tokens' kernel.
int launch_kv8_join(const Kv8Attn& a, int head_dim, int storage, const Kv8Pieces& p, int dec_ctas, cudaStream_t s);

}  // namespace sar
