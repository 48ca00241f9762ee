// Microscaled 4-bit rows: quantisation and its inverse.
//
// A row is cut into blocks of B columns; block b of row r keeps one scale byte
// s and B e2m1 codes q (0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign), and stands for
// q * s * tensor_scale.  Two formats: NV (B = 16, s an e4m3 number) and MX
// (B = 32, s = 2^(byte - 127)).
//
// Codes lie two to a byte, [rows][cols / 2].  Scales lie in tiles of 128 rows x
// 4 blocks, 512 bytes each, in the order in which the 4-bit product's tensor
// cores take them (see include/sar_ops.h), so that the product copies a tile
// from global memory to tensor memory without touching it.
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace sar {

namespace {

constexpr int kThreads = 256;
constexpr int kSeg = 16;         // columns per quantising thread: an NV block, half an MX block
constexpr int kQuantPerSm = 16;   // quantising CTAs per SM (about five at a time), each walking its share
constexpr int kDequantEach = 4;  // units of 16 output bytes per dequantising thread

// n / d for n < 2^31 as a multiplication and a shift (Granlund and Montgomery
// 1994: mul = ceil(2^(31 + l) / d) with 2^l >= d): the division of an item's
// number into row and column would otherwise cost a thread as much as six of its
// sixteen elements.
struct Divisor {
  uint32_t d, mul, shift;
};
Divisor divisor(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  return {d, (uint32_t)(((1ull << (31 + l)) + d - 1) / d), 31 + l};
}
__device__ __forceinline__ uint32_t over(uint32_t n, const Divisor& v) {
  return (uint32_t)(((uint64_t)n * v.mul) >> v.shift);
}

template <typename X>
__device__ __forceinline__ float to_f32(X v) {
  if constexpr (sizeof(X) == 4)
    return v;
  else
    return Elem<X>::to(v);
}

// a / b correctly rounded, r = 1 / b correctly rounded (Markstein 1990; no
// overflow on the way).  The remainder's sign as written keeps a negative zero
// negative.
__device__ __forceinline__ float quotient(float a, float b, float r) {
  const float q = a * r;
  return fmaf(-fmaf(q, b, -a), r, q);
}

// The larger of m and |u| in each half, NaN if u's is one.
template <typename X>
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t u) {
  using P = typename std::conditional<std::is_same<X, __nv_bfloat16>::value, __nv_bfloat162, __half2>::type;
  const P r = __hmax2_nan(*reinterpret_cast<P*>(&m), __habs2(*reinterpret_cast<P*>(&u)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// 16 consecutive values as they lie in memory.
template <typename X>
struct Raw {
  static constexpr int kWords = kSeg * sizeof(X) / 4;
  uint32_t u[kWords];
  // vec: the address is 16-byte aligned
  __device__ __forceinline__ void load(const X* p, bool vec) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i)
        *reinterpret_cast<uint4*>(u + 4 * i) = __ldg(reinterpret_cast<const uint4*>(p) + i);
    } else if constexpr (sizeof(X) == 4) {
#pragma unroll
      for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(p[i]);
    } else {
      const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = (uint32_t)h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
    }
  }
  // The values as fp32, and the largest of their magnitudes (infinity or NaN if
  // one is): patterns without the sign rise with the magnitude, a NaN's is above
  // infinity's; 16-bit ones are compared two at a time.
  __device__ __forceinline__ float unpack(float (&v)[16]) const {
    uint32_t m = 0;
    if constexpr (sizeof(X) == 4) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        m = max(m, u[i] & 0x7fffffffu);
        v[i] = __uint_as_float(u[i]);
      }
      return __uint_as_float(m);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m = max_abs2<X>(m, u[i]);
        v[2 * i] = Elem<X>::lo(u[i]);
        v[2 * i + 1] = Elem<X>::hi(u[i]);
      }
      return Elem<X>::lo(max(m & 0xffffu, m >> 16));
    }
  }
};

// Eight values as e2m1 codes, the first in the lowest bits; to nearest even, at
// most 6 in magnitude.
__device__ __forceinline__ uint32_t pack8(const float* v) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w;
}

// Byte offset of the scale tile of (row, tile column) plus the row's place in it.
__device__ __forceinline__ size_t scale_offset(uint32_t row, uint32_t tile, uint32_t tiles) {
  return ((size_t)(row >> 7) * tiles + tile) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// Each thread quantises 16 columns.  With t = x * inv_g and a = max |t| over
// the block:
//   NV  s = e4m3(min(a / 6, 448)),           q = e2m1(t / s)  (0 where s = 0)
//   MX  s = 2^max(floor(log2 a) - 2, -127),  q = e2m1(t / s)
// both roundings to nearest even, e2m1 saturating at 6 (a scale that was
// rounded down leaves t / s up to 6.4, MX's floor up to 8).  A block with a NaN
// or an infinity gets a NaN scale and zero codes.
//
// t / s has to fall on the right side of e2m1's seven borders.  For MX the
// factor is a power of two.  For NV the quotient is formed with r = 1 / s and
// corrected once by its exact remainder, which rounds t / s correctly.  Such a
// rounded quotient never rounds onto a border b it does not equal: b * s has 7
// significant bits at most, so a different t is at least one of its own units
// away from it, which is more than half a unit of b after the division.  Two
// fused multiply-adds per element instead of a division (~10 instructions).
//
// Bound by HBM (fp32, MX) or, for 16-bit rows in NV, by the 13 instructions per
// element as well; each thread walks several segments with the next one's loads
// on their way (28672 x 4096 bf16 NV: 53.8 us, against 60.7 with a segment to a
// thread, when 58% of the warps were resident and issued 0.66 a clock).
//
// The 4 scale bytes that neighbour in a tile's row are gathered from the lanes
// and stored as one word.  Columns are padded to whole tiles: the padding
// blocks' scales are written as zero, as the product reads them.
template <typename X, bool NV>
__global__ void __launch_bounds__(kThreads)
    fp4_quantize_kernel(const X* __restrict__ x, int64_t ldx, uint32_t rows, uint32_t cols, uint32_t tiles, Divisor segs,
                        float inv_g, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int vec) {
  constexpr uint32_t kSegsPerTile = NV ? 4 : 8;
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t n = rows * segs.d, step = gridDim.x * kThreads;
  // where segment i lies (n is whole groups of kSegsPerTile lanes)
  auto place = [&](uint32_t i, uint32_t& row, uint32_t& seg) {
    row = over(i, segs);
    seg = i - row * segs.d;
    return i < n && seg * kSeg < cols;
  };
  uint32_t i = blockIdx.x * kThreads + threadIdx.x, row, seg;
  Raw<X> raw;
  bool has = place(i, row, seg);
  if (has) raw.load(x + (int64_t)row * ldx + seg * kSeg, vec != 0);
  for (uint32_t i0 = blockIdx.x * kThreads; i0 < n; i0 += step) {  // (all lanes as often)
    const Raw<X> now = raw;
    const bool has_now = has, live = i < n;
    const uint32_t row_now = row, seg_now = seg;
    i += step;
    has = place(i, row, seg);
    if (has) raw.load(x + (int64_t)row * ldx + seg * kSeg, vec != 0);
    float v[16];
    uint32_t ab = 0;  // the block's max |t| as a pattern
    if (has_now) {
      // max |x| * inv_g is max |x * inv_g|: the rounding keeps the order
      ab = __float_as_uint(now.unpack(v) * inv_g);
      if (inv_g != 1.f) {
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] *= inv_g;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = 0.f;
    }
    if constexpr (!NV) ab = max(ab, __shfl_xor_sync(0xffffffffu, ab, 1));
    const bool bad = ab >= 0x7f800000u;
    bool zero = bad;  // no codes
    uint32_t byte;
    if constexpr (NV) {
      const __nv_fp8_storage_t s8 =
          __nv_cvt_float_to_fp8(quotient(__uint_as_float(ab), 6.f, 1.f / 6.f), __NV_SATFINITE, __NV_E4M3);
      byte = bad ? 0x7Fu : (uint32_t)s8;
      const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(s8, __NV_E4M3)));
      zero = bad || s == 0.f;
      const float r = __frcp_rn(s);
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = quotient(v[k], s, r);
    } else {
      const uint32_t e = ab >> 23;  // biased exponent (0: zero or subnormal)
      byte = bad ? 0xFFu : e >= 2 ? e - 2 : 0u;
      const float r = __uint_as_float((254u - (bad ? 127u : byte)) << 23);
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] *= r;
    }
    if (!has_now) byte = 0;
    if (has_now) {
      const uint32_t w[2] = {pack8(v), pack8(v + 8)};
      *reinterpret_cast<uint2*>(codes + (size_t)row_now * (cols / 2) + seg_now * (kSeg / 2)) = zero ? make_uint2(0, 0) : make_uint2(w[0], w[1]);
    }
    const uint32_t lane = threadIdx.x & 31;
    uint32_t word;
    if constexpr (NV) {
      word = byte << (8 * (lane & 3));
      word |= __shfl_xor_sync(0xffffffffu, word, 1);
      word |= __shfl_xor_sync(0xffffffffu, word, 2);
    } else {
      word = (lane & 1) ? 0u : byte << (8 * ((lane >> 1) & 3));
      word |= __shfl_xor_sync(0xffffffffu, word, 2);
      word |= __shfl_xor_sync(0xffffffffu, word, 4);
    }
    if (live && (lane & (kSegsPerTile - 1)) == 0)
      *reinterpret_cast<uint32_t*>(scales + scale_offset(row_now, seg_now / kSegsPerTile, tiles)) = word;
  }
}

// y = code * s * g: the product of a code and its scale is exact in fp32 (3 and
// 4 significant bits); * g rounds once, the conversion to Y once more.  MX's three
// largest scales (2^125 and up) times a code can pass fp32 where the whole product
// does not: they are taken 2^8 lower and g 2^8 higher, both exact.  (From g = 2^100
// on such a block overflows whatever g is, but its zeros have to stay zeros.)
//
// A unit is 16 bytes of output (8 or 4 columns), neighbouring lanes take
// neighbouring units and a thread takes four of them kThreads units apart, so
// that a warp's store covers 512 whole bytes (a thread's 16 columns as two
// stores: 69.0 us for 20480 x 7168 bf16, every sector written in two halves; so
// 60.0 us, 6.3 TB/s).  Bound by HBM.
template <typename Y, bool NV>
__global__ void __launch_bounds__(kThreads)
    fp4_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, uint32_t rows,
                          uint32_t cols, uint32_t tiles, Divisor units, float g, Y* __restrict__ y, int64_t ldy, int vec) {
  constexpr uint32_t kCols = 16 / sizeof(Y);
  constexpr int kEach = kDequantEach;
  pdl_wait();
  pdl_launch_dependents();
  const uint64_t n = (uint64_t)rows * units.d;
  uint32_t c[kEach], b[kEach], row[kEach], col[kEach];
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const uint64_t i = ((uint64_t)blockIdx.x * kEach + u) * kThreads + threadIdx.x;
    if (i >= n) break;
    row[u] = over((uint32_t)i, units);
    const uint32_t unit = (uint32_t)i - row[u] * units.d;
    col[u] = unit * kCols;
    const uint32_t block = col[u] / (NV ? 16 : 32);
    const uint8_t* at = codes + (size_t)row[u] * (cols / 2) + unit * (kCols / 2);
    c[u] = sizeof(Y) == 4 ? (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(at))
                          : __ldg(reinterpret_cast<const uint32_t*>(at));
    b[u] = __ldg(scales + scale_offset(row[u], block >> 2, tiles) + (block & 3));
  }
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const uint64_t i = ((uint64_t)blockIdx.x * kEach + u) * kThreads + threadIdx.x;
    if (i >= n) break;
    float s, gs = g;
    if constexpr (NV) {
      s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b[u], __NV_E4M3)));
    } else {  // 2^(b - 127); 2^-127 is a subnormal
      const bool high = b[u] >= 252;
      s = __uint_as_float(b[u] == 255 ? 0x7fc00000u : b[u] == 0 ? 0x00400000u : (high ? b[u] - 8 : b[u]) << 23);
      if (high) gs = fminf(g, 0x1p100f) * 256.f;
    }
    float v[kCols];
#pragma unroll
    for (int k = 0; k < (int)kCols / 2; ++k) {
      const __half2 h(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)((c[u] >> (8 * k)) & 0xffu), __NV_E2M1));
      v[2 * k] = __low2float(h) * s * gs;
      v[2 * k + 1] = __high2float(h) * s * gs;
    }
    Y* dst = y + (int64_t)row[u] * ldy + col[u];
    if (!vec) {
#pragma unroll
      for (int k = 0; k < (int)kCols; ++k) {
        if constexpr (sizeof(Y) == 4)
          dst[k] = v[k];
        else
          dst[k] = Elem<Y>::from(v[k]);
      }
    } else if constexpr (sizeof(Y) == 4) {
      *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      *reinterpret_cast<uint4*>(dst) = make_uint4(Elem<Y>::pack(v[0], v[1]), Elem<Y>::pack(v[2], v[3]),
                                                  Elem<Y>::pack(v[4], v[5]), Elem<Y>::pack(v[6], v[7]));
    }
  }
}

bool good_format(int format) { return format == SAR_FP4_NV || format == SAR_FP4_MX; }
bool good_type(int type) { return type == SAR_TYPE_F16 || type == SAR_TYPE_BF16 || type == SAR_TYPE_F32; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The checks that both directions share; *blocks and *div receive the launch's
// size and work items per row.
int check_rows(const char* what, bool quantising, const void* x, int64_t ld, int rows, int cols, int type, int format,
               float scale, const void* codes, const void* scales, uint32_t* blocks, Divisor* div) {
  auto refuse = [what](int code, const char* why) { return set_error(code, std::string(what) + why); };
  if (rows < 0 || cols <= 0) return refuse(SAR_ERR_INVALID_ARG, ": bad shape");
  if (!good_format(format)) return refuse(SAR_ERR_INVALID_ARG, ": bad format");
  if (!good_type(type)) return refuse(SAR_ERR_INVALID_ARG, ": bad element type");
  if (cols % 32) return refuse(SAR_ERR_UNSUPPORTED, ": columns must be a multiple of 32");
  if (ld < cols) return refuse(SAR_ERR_INVALID_ARG, ": row stride below the row's length");
  if (!(scale > 0.f) || !std::isfinite(scale) || !std::isfinite(1.f / scale))
    return refuse(SAR_ERR_INVALID_ARG, ": the tensor scale must be positive and finite, as its inverse");
  *blocks = 0;
  if (rows == 0) return SAR_OK;
  if (!x || !codes || !scales) return refuse(SAR_ERR_INVALID_ARG, ": null pointer");
  if (reinterpret_cast<uintptr_t>(x) & (type == SAR_TYPE_F32 ? 3 : 1))
    return refuse(SAR_ERR_INVALID_ARG, ": rows not aligned to their element");
  if (!aligned16(codes) || !aligned16(scales))
    return refuse(SAR_ERR_INVALID_ARG, ": codes and scales must be 16-byte aligned");
  // work items: 16 columns of a row padded to whole scale tiles (quantising), 16
  // bytes of output (dequantising)
  const uint64_t per_row = quantising ? (uint64_t)fp4_tiles(cols, format) * (format == SAR_FP4_NV ? 4 : 8)
                                      : (uint64_t)cols * (type == SAR_TYPE_F32 ? 4 : 2) / 16;
  const uint64_t items = rows * per_row;
  if (items >= 1ull << 31) return refuse(SAR_ERR_UNSUPPORTED, ": more than 2^31 work items");
  const int per_block = kThreads * (quantising ? 1 : kDequantEach);
  *blocks = (uint32_t)((items + per_block - 1) / per_block);
  if (quantising) *blocks = std::min<uint32_t>(*blocks, (uint32_t)num_sms() * kQuantPerSm);
  *div = divisor((uint32_t)per_row);
  return SAR_OK;
}

template <typename X>
int quantize(const void* x, int64_t ldx, int rows, int cols, int format, float inv_g, void* codes, void* scales,
             uint32_t blocks, Divisor div, cudaStream_t s) {
  const int vec = aligned16(x) && (ldx * (int64_t)sizeof(X)) % 16 == 0;
  const uint32_t tiles = (uint32_t)fp4_tiles(cols, format);
  auto fn = format == SAR_FP4_NV ? fp4_quantize_kernel<X, true> : fp4_quantize_kernel<X, false>;
  const cudaError_t e = launch_pdl(fn, dim3(blocks), dim3(kThreads), 0, s, static_cast<const X*>(x), ldx, (uint32_t)rows,
                                   (uint32_t)cols, tiles, div, inv_g, static_cast<uint8_t*>(codes),
                                   static_cast<uint8_t*>(scales), vec);
  if (e != cudaSuccess) return cuda_error(e, "fp4 quantise launch");
  count_launches(1);
  return SAR_OK;
}

template <typename Y>
int dequantize(const void* codes, const void* scales, int rows, int cols, int format, float g, void* y, int64_t ldy,
               uint32_t blocks, Divisor div, cudaStream_t s) {
  const int vec = aligned16(y) && (ldy * (int64_t)sizeof(Y)) % 16 == 0;
  const uint32_t tiles = (uint32_t)fp4_tiles(cols, format);
  auto fn = format == SAR_FP4_NV ? fp4_dequantize_kernel<Y, true> : fp4_dequantize_kernel<Y, false>;
  const cudaError_t e =
      launch_pdl(fn, dim3(blocks), dim3(kThreads), 0, s, static_cast<const uint8_t*>(codes),
                 static_cast<const uint8_t*>(scales), (uint32_t)rows, (uint32_t)cols, tiles, div, g, static_cast<Y*>(y), ldy, vec);
  if (e != cudaSuccess) return cuda_error(e, "fp4 dequantise launch");
  count_launches(1);
  return SAR_OK;
}

}  // namespace

}  // namespace sar

using sar::set_error;

extern "C" {

int sar_op_fp4_scale_bytes(int32_t rows, int32_t cols, int32_t format, int64_t* out) try {
  if (!out || rows < 0 || cols <= 0 || !sar::good_format(format))
    return set_error(SAR_ERR_INVALID_ARG, "fp4_scale_bytes: bad argument");
  if (cols % 32) return set_error(SAR_ERR_UNSUPPORTED, "fp4_scale_bytes: columns must be a multiple of 32");
  *out = ((int64_t)rows + 127) / 128 * sar::fp4_tiles(cols, format) * 512;
  return SAR_OK;
} catch (...) {
  return sar::entry_failed("fp4_scale_bytes");
}

int sar_op_fp4_quantize(const void* x, int64_t ldx, int32_t rows, int32_t cols, int32_t type, int32_t format,
                        float tensor_scale, void* codes, void* scales, void* stream) try {
  uint32_t blocks = 0;
  sar::Divisor div;
  SAR_TRY(sar::check_rows("fp4_quantize", true, x, ldx, rows, cols, type, format, tensor_scale, codes, scales, &blocks,
                          &div));
  if (blocks == 0) return SAR_OK;
  const float inv = 1.f / tensor_scale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (type == SAR_TYPE_F32) return sar::quantize<float>(x, ldx, rows, cols, format, inv, codes, scales, blocks, div, s);
  if (type == SAR_TYPE_BF16)
    return sar::quantize<__nv_bfloat16>(x, ldx, rows, cols, format, inv, codes, scales, blocks, div, s);
  return sar::quantize<__half>(x, ldx, rows, cols, format, inv, codes, scales, blocks, div, s);
} catch (...) {
  return sar::entry_failed("fp4_quantize");
}

int sar_op_fp4_dequantize(const void* codes, const void* scales, int32_t rows, int32_t cols, int32_t format,
                          float tensor_scale, void* y, int64_t ldy, int32_t type, void* stream) try {
  uint32_t blocks = 0;
  sar::Divisor div;
  SAR_TRY(sar::check_rows("fp4_dequantize", false, y, ldy, rows, cols, type, format, tensor_scale, codes, scales, &blocks,
                          &div));
  if (blocks == 0) return SAR_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (type == SAR_TYPE_F32)
    return sar::dequantize<float>(codes, scales, rows, cols, format, tensor_scale, y, ldy, blocks, div, s);
  if (type == SAR_TYPE_BF16)
    return sar::dequantize<__nv_bfloat16>(codes, scales, rows, cols, format, tensor_scale, y, ldy, blocks, div, s);
  return sar::dequantize<__half>(codes, scales, rows, cols, format, tensor_scale, y, ldy, blocks, div, s);
} catch (...) {
  return sar::entry_failed("fp4_dequantize");
}

}  // extern "C"
