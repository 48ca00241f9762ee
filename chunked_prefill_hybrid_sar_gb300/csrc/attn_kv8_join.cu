// Joins the pieces of units that several CTAs of the 8-bit cache's attention share, in
// their order: one kernel for single tokens' and chunks' (a kernel of its own for either
// cost a mixed call 3 us more).
//
// Bound by latencies: the plan, a piece's maxima and sums, its rows.  Pieces' loads
// do not wait for their maxima, and several are under way together.  Between 3.5 us (where
// nothing is to be joined) and 10 (152 CTAs' pieces, 35 MB).  Single tokens: a warp to a
// head, 4 to 5 us; with a CTA to a head and its warps' sums joined again, 9 to 11.
#include "kv8.cuh"

namespace sar {

namespace {

constexpr int kJoinWarps = 8;
constexpr int kJoinRows = 16;  // (row, head) pairs of a chunk's unit that a CTA joins

// The single tokens' unit that CTA first + 1 begins inside of, if no CTA before does: a
// warp to a head, the loads of eight pieces under way together.
template <typename T, int D>
__device__ __forceinline__ void join_tokens(const Kv8Attn& a, const Kv8Pieces& p, int first) {
  constexpr int E = D / 32, AT_ONCE = 8;  // dims of a lane
  const int head = threadIdx.x >> 5, lane = threadIdx.x & 31, second = first + 1;
  const DecLine line = *p.line;
  const DecStart u = p.starts[second];
  if (head >= a.G || line.all == 0 || second >= line.ctas || u.seq < 0) return;
  const int64_t begins = line.at(first);  // the CTA before's first block
  if (begins > u.u0) return;
  const int last = line.cta(u.u0 + u.blocks - 1);
  // the first CTA's piece is its last one, unless the unit begins with it
  auto slot = [&](int c) { return (int64_t)(2 * c + (c == first && begins != u.u0 ? 1 : 0)) * kDecHeads + head; };
  float M = -INFINITY, L = 0.f, A[E];
#pragma unroll
  for (int e = 0; e < E; ++e) A[e] = 0.f;
  for (int c0 = first; c0 <= last; c0 += AT_ONCE) {
    float2 ml[AT_ONCE];
    float v[AT_ONCE][E];
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      const int64_t s = slot(min(c0 + k, last));
      ml[k] = c0 + k <= last ? p.parts_ml[s] : make_float2(-INFINITY, 0.f);
      const float* row = p.parts + s * D + lane * E;
      if constexpr (E == 4) {
        const float4 x = *reinterpret_cast<const float4*>(row);
        v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(row);
        v[k][0] = x.x, v[k][1] = x.y;
      }
    }
    float mn = M;
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) mn = fmaxf(mn, ml[k].x);
    const float f = M == -INFINITY ? 0.f : exp2_fast(M - mn);
    L *= f;
#pragma unroll
    for (int e = 0; e < E; ++e) A[e] *= f;
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      const bool some = ml[k].x != -INFINITY;
      const float w = some ? exp2_fast(ml[k].x - mn) : 0.f;
      L = fmaf(ml[k].y, w, L);
#pragma unroll
      for (int e = 0; e < E; ++e) A[e] = fmaf(some ? v[k][e] : 0.f, w, A[e]);
    }
    M = mn;
  }
  const float inv = 1.f / L;
  T* op = static_cast<T*>(a.out) + (int64_t)u.row * a.ldo + (int64_t)(u.kh * a.G + head) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    if (p.vec_o) {
      *reinterpret_cast<uint32_t*>(op + e) = Elem<T>::pack(A[e] * inv, A[e + 1] * inv);
    } else {
      op[e] = Elem<T>::from(A[e] * inv), op[e + 1] = Elem<T>::from(A[e + 1] * inv);
    }
  }
}

// 16 pairs of a unit of a chunk; a thread has four dims of a pair, or two times four.
template <typename T, int D>
__device__ __forceinline__ void join_chunk(const Kv8Attn& a, const Kv8Pieces& p, int64_t all, int each, int C, int item) {
  constexpr int E = kJoinRows * D / 4 / (kJoinWarps * 32), AT_ONCE = 4 / E;
  static_assert(E == 1 || E == 2, "elements of a thread");
  const int sub = item % (256 / kJoinRows), unit = item / (256 / kJoinRows);
  const int t = (int)((unsigned)unit / (unsigned)a.kvh), kh = unit - t * a.kvh;
  const auto tile = p.plan->tile[t];
  const int nb = p.plan->tile[t + 1].before - tile.before;
  const int64_t u0 = (int64_t)tile.before * a.kvh + (int64_t)kh * nb, u1 = u0 + nb;
  // the CTAs of its first and last block
  const int c0 = each ? unit * each : (int)DecLine::quotient((u0 + 1) * C - 1, all);
  const int c1 = each ? c0 + min(each, nb) - 1 : (int)DecLine::quotient(u1 * C - 1, all);
  const int r = sub * kJoinRows + threadIdx.x % kJoinRows;
  if (c0 == c1 || r >= tile.pairs) return;
  const bool starts = each || line_at((int)all, c0, C) == u0;
  const float4* parts = reinterpret_cast<const float4*>(p.chunk_parts) + (int64_t)(threadIdx.x / kJoinRows) * 256 + r;
  float Mx = -INFINITY, L = 0.f;
  float4 A[E];
#pragma unroll
  for (int e = 0; e < E; ++e) A[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = c0; c <= c1; c += AT_ONCE) {
    float2 ml[AT_ONCE];
    float4 v[AT_ONCE][E];
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      const int ck = min(c + k, c1);
      const int64_t slot = 2 * ck + (ck == c0 && !starts ? 1 : 0);
      ml[k] = c + k <= c1 ? p.chunk_parts_ml[slot * 256 + r] : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < E; ++e) v[k][e] = parts[(slot * (D / 4) + e * (kJoinWarps * 32 / kJoinRows)) * 256];
    }
    float mn = Mx;
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) mn = fmaxf(mn, ml[k].x);
    const float f = Mx == -INFINITY ? 0.f : exp2_fast(Mx - mn);
    L *= f;
#pragma unroll
    for (int e = 0; e < E; ++e) A[e].x *= f, A[e].y *= f, A[e].z *= f, A[e].w *= f;
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      if (ml[k].x == -INFINITY) {
        L += ml[k].y;  // (zero, or NaN; its rows may never have been written)
        continue;
      }
      const float g = exp2_fast(ml[k].x - mn);
      L = fmaf(ml[k].y, g, L);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        A[e].x = fmaf(v[k][e].x, g, A[e].x);
        A[e].y = fmaf(v[k][e].y, g, A[e].y);
        A[e].z = fmaf(v[k][e].z, g, A[e].z);
        A[e].w = fmaf(v[k][e].w, g, A[e].w);
      }
    }
    Mx = mn;
  }
  const unsigned pair = (unsigned)(tile.pair0 + r);
  const int token = (int)(pair / (unsigned)a.G), head = kh * a.G + (int)(pair % (unsigned)a.G);
  const float inv = tile.past + token < 0 ? 0.f : 1.f / L;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int dim = 4 * (threadIdx.x / kJoinRows + e * (kJoinWarps * 32 / kJoinRows));
    T* op = static_cast<T*>(a.out) + (int64_t)(tile.row0 + token) * a.ldo + (int64_t)head * D + dim;
    if (p.vec_o) {
      *reinterpret_cast<uint2*>(op) =
          make_uint2(Elem<T>::pack(A[e].x * inv, A[e].y * inv), Elem<T>::pack(A[e].z * inv, A[e].w * inv));
    } else {
      op[0] = Elem<T>::from(A[e].x * inv), op[1] = Elem<T>::from(A[e].y * inv);
      op[2] = Elem<T>::from(A[e].z * inv), op[3] = Elem<T>::from(A[e].w * inv);
    }
  }
}

// The first dec_blocks CTAs: a single token's unit each; the others share the chunks' units.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) kv8_join_kernel(const __grid_constant__ Kv8Attn a,
                                                                   const __grid_constant__ Kv8Pieces p) {
  pdl_wait();
  pdl_launch_dependents();
  if ((int)blockIdx.x < p.dec_blocks) {
    join_tokens<T, D>(a, p, blockIdx.x);
    return;
  }
  const int all = p.plan->all, each = p.plan->each, C = p.plan->ctas;
  if (all == 0) return;
  const int items = p.plan->tiles * a.kvh * (256 / kJoinRows);
  for (int w = blockIdx.x - p.dec_blocks; w < items; w += gridDim.x - p.dec_blocks) join_chunk<T, D>(a, p, all, each, C, w);
}

template <typename T, int D>
int launch_join(const Kv8Attn& a, const Kv8Pieces& p, cudaStream_t s) {
  const unsigned grid = (unsigned)(p.dec_blocks + (p.plan ? 8 * num_sms() : 0));
  const cudaError_t e = launch_pdl(kv8_join_kernel<T, D>, dim3(grid), dim3(kJoinWarps * 32), 0, s, a, p);
  if (e != cudaSuccess) return cuda_error(e, "kv8 join launch");
  count_launches(1);
  return SAR_OK;
}

}  // namespace

int launch_kv8_join(const Kv8Attn& a, int head_dim, int storage, const Kv8Pieces& pieces, int dec_ctas, cudaStream_t s) {
  Kv8Pieces p = pieces;
  p.dec_blocks = p.line ? dec_ctas - 1 : 0;
  p.vec_o = aligned_to(a.out, 8) && a.ldo % 4 == 0;
  const bool bf = storage == SAR_STORAGE_BF16;
  if (head_dim == 128) return bf ? launch_join<__nv_bfloat16, 128>(a, p, s) : launch_join<__half, 128>(a, p, s);
  return bf ? launch_join<__nv_bfloat16, 64>(a, p, s) : launch_join<__half, 64>(a, p, s);
}

}  // namespace sar
