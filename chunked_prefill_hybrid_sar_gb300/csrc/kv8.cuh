// The 8-bit KV cache on the device: where codes lie, and e4m3 in and out.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace sar {

// Exponents of a page's scale.  Between them attention's weights, which carry a
// page's value scale in their exponent, stay inside fp32's range; magnitudes under
// 2^-49 become zero, those over 448 * 2^60 saturate.
constexpr int kKv8Least = -40, kKv8Most = 60;

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
  int64_t bt_stride;
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
         len <= (a.bt_stride << a.shift);
}

// Sequences of several rows (attn_kv8_chunk.cu): the workspace that they take, their
// kernel, launched right behind the single tokens', and the one that joins its pieces.
int64_t kv8_chunk_space(int head_dim);
int launch_kv8_chunks(const Kv8Attn& a, int head_dim, int storage, void* space, cudaStream_t s);
int launch_kv8_chunk_join(const Kv8Attn& a, int head_dim, int storage, void* space, cudaStream_t s);

}  // namespace sar
