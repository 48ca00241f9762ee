// Head norms, the rotary embedding and the append to the 8-bit cache, behind a
// step's QKV projection.
//
// A group of head_dim / 8 lanes has a row's head: eight elements a lane, four from
// each half of the head, so that a rotation pair sits in one lane.  mean(h^2) is a
// sum over the group.  Angles: position * theta / 2 pi as a fixed-point fraction of
// a turn, 64 bits that wrap, which reduces any position exactly; then two short series.
// They are formed once per row and reused for all of a CTA's heads.
//
// Query heads are independent.  For the cache the unit is a run: the rows of a call
// in one page, which share a scale for each head.  A CTA takes the runs that begin
// in its window of rows (they may end up to 63 rows behind it), keeps their rows'
// keys or values in registers, joins the rows' largest magnitudes by a shared-memory
// maximum per run (whose order does not matter), and writes codes: the input is read once.
//
// Rows of queries are bound by memory (12288 x 56 heads of 128, bf16: 61 us, where a copy of
// them takes 53).  The cache's part (8 + 8 heads: 39 us; 45 where every row of a run searched the
// maxima of the others) is bound by a CTA's chain of slots, rows, maxima, barrier and codes: issue
// slots are 46% used and memory 18%, with 29 of 64 warps on an SM, which wait for loads,
// shared memory, one another and the barrier in like parts.
// Both in one launch 98 us on inputs that are not in L2, against 63 for the bytes.  At an
// earlier state (98): their CTAs in turn instead of the cache's first, 98 too; a window's
// tasks side by side, 105, as the longest then come last as well.
#include <math.h>

#include <algorithm>

#include "kv8.cuh"

namespace sar {

namespace {

constexpr int kQkThreads = 512;

struct QkArgs {
  sar_qk_rows r;
  sar_kv8 c;
  int shift;           // log2 page_size
  int q_heads_per, kv_heads_per;     // heads of a CTA
  int q_tasks, k_tasks, kv_tasks;    // CTAs of a window of rows: queries, k_out, cache (keys, then values)
  int vec_q, vec_k, vec_v, vec_qo, vec_ko;  // rows whose pieces of four are aligned
  int* err;
  uint64_t turn[64];   // theta_i / (2 pi) in units of 2^-64 turns
};

template <typename T>
__device__ __forceinline__ float to_f(T x) {
  if constexpr (sizeof(T) == 4)
    return x;
  else
    return Elem<T>::to(x);
}

// Four adjacent elements.
template <typename T>
__device__ __forceinline__ void load4(const T* p, bool vec, float* x) {
  if (vec) {
    if constexpr (sizeof(T) == 4) {
      const float4 v = *reinterpret_cast<const float4*>(p);
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      x[0] = Elem<T>::lo(v.x), x[1] = Elem<T>::hi(v.x), x[2] = Elem<T>::lo(v.y), x[3] = Elem<T>::hi(v.y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = to_f<T>(p[e]);
  }
}

template <typename T>
__device__ __forceinline__ void store4(T* p, bool vec, const float* x) {
  if (vec) {
    *reinterpret_cast<uint2*>(p) = make_uint2(Elem<T>::pack(x[0], x[1]), Elem<T>::pack(x[2], x[3]));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = Elem<T>::from(x[e]);
  }
}

// Asks for a line to come to L2.
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int LANES>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// (cos, sin) of a lane's four frequencies at a position, off by little more than the
// rounding to fp32 (a key that lies near a border of two codes falls on the side that the
// formula's does): the angle less its nearest multiple of a quarter turn, x = hi + lo, and
// Taylor's series on |x| <= pi / 4, whose first terms are added last, with what they lose.
__device__ __forceinline__ void angles(const QkArgs& a, int pos, int i0, float* cs, float* sn) {
  constexpr float kTo = (float)(3.14159265358979323846 / 2147483648.0);  // from units of 2^-31 half turns
  constexpr float kToLow = (float)(3.14159265358979323846 / 2147483648.0 - (double)kTo);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint64_t t = (uint64_t)(int64_t)pos * a.turn[i0 + e];
    const uint32_t h = (uint32_t)(t >> 32);  // half turns in units of 2^-31, around the circle
    const uint32_t quarter = (h + (1u << 29)) >> 30;
    const int32_t r = (int32_t)(h - (quarter << 30));
    const float rf = (float)r, hi = rf * kTo;
    const float lo = fmaf(rf, kTo, -hi) + fmaf(rf, kToLow, (float)(r - (int32_t)rf) * kTo);
    const float x2 = hi * hi;
    const float s = hi + fmaf(hi * x2, fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, -1.f / 39916800.f, 1.f / 362880.f), -1.f / 5040.f),
                                                     1.f / 120.f), -1.f / 6.f), lo);
    const float low2 = fmaf(hi, hi, -x2), w = fmaf(-0.5f, x2, 1.f);
    const float c = w + (fmaf(-0.5f, x2, 1.f - w) - fmaf(hi, lo, 0.5f * low2) +
                         x2 * x2 * fmaf(x2, fmaf(x2, fmaf(x2, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f));
    const float u = quarter & 1 ? s : c, v = quarter & 1 ? c : s;
    cs[e] = (quarter + 1) & 2 ? -u : u;
    sn[e] = quarter & 2 ? -v : v;
  }
}

template <int D>
__device__ __forceinline__ void norm_rope(float* x, const float* gain, bool normed, float eps, bool turned, const float* cs,
                                          const float* sn) {
  if (normed) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
    const float inv = rsqrtf(group_sum<D / 8>(ss) * (1.0f / D) + eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * gain[e];
  }
  if (turned) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float u = x[e], w = x[e + 4];
      // (products rounded before they are added, as fp32 programs of this formula have them: of
      // keys on a border of two codes, both then take the same)
      x[e] = __fsub_rn(__fmul_rn(u, cs[e]), __fmul_rn(w, sn[e]));
      x[e + 4] = __fadd_rn(__fmul_rn(w, cs[e]), __fmul_rn(u, sn[e]));
    }
  }
}

// TI: the rows' type; TO: the 16-bit type written.
template <typename TI, typename TO, int D>
__global__ void __launch_bounds__(kQkThreads, 2) qk_rows_kernel(const __grid_constant__ QkArgs a) {
  constexpr int LANES = D / 8, GROUPS = kQkThreads / LANES;  // rows of a pass, and of a window
  constexpr int PASSES = (GROUPS + 63 + GROUPS - 1) / GROUPS;
  constexpr int SPAN = PASSES * GROUPS;  // rows that a window's runs can reach
  const sar_qk_rows& r = a.r;
  const int grp = threadIdx.x / LANES, l = threadIdx.x % LANES;
  const int w0 = blockIdx.x * GROUPS, task = blockIdx.y;
  pdl_wait();
  pdl_launch_dependents();

  if (task >= a.kv_tasks) {
    // ---- heads that are written as rows: queries, or keys ----
    const bool is_q = task < a.kv_tasks + a.q_tasks;
    const int row = w0 + grp;
    const int h0 = is_q ? (task - a.kv_tasks) * a.q_heads_per : (task - a.kv_tasks - a.q_tasks) * a.q_heads_per;
    const int h1 = min(h0 + a.q_heads_per, is_q ? r.n_q_heads : r.n_kv_heads);
    const bool live = row < r.rows;
    const float* gp = is_q ? r.q_gain : r.k_gain;
    float gain[8], cs[4], sn[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) gain[e] = gp ? gp[4 * l + e] : 1.f, gain[4 + e] = gp ? gp[D / 2 + 4 * l + e] : 1.f;
    if (r.positions) angles(a, live ? r.positions[row] : 0, 4 * l, cs, sn);
    const int64_t ld = is_q ? r.ldq : r.ldk, ldo = is_q ? r.ldq_out : r.ldk_out;
    const TI* src = static_cast<const TI*>(is_q ? r.q : r.k) + (live ? row : 0) * ld + 4 * l;
    TO* dst = static_cast<TO*>(is_q ? r.q_out : r.k_out) + row * ldo + 4 * l;
    const bool vi = is_q ? a.vec_q : a.vec_k, vo = is_q ? a.vec_qo : a.vec_ko;
    constexpr int AT_ONCE = 4;  // heads whose loads are under way together
    constexpr int LINES = D * (int)sizeof(TI) / 128;  // of a head
    for (int h = h0; h < h1; h += AT_ONCE) {
      // the next heads come to L2 while these are worked on
      for (int k = l; k < AT_ONCE * LINES; k += LANES)
        if (live && h + AT_ONCE + k / LINES < h1)
          prefetch_l2(reinterpret_cast<const char*>(src - 4 * l + (h + AT_ONCE) * D) + k * 128);
      float x[AT_ONCE][8];
#pragma unroll
      for (int u = 0; u < AT_ONCE; ++u) {
        const TI* p = src + min(h + u, h1 - 1) * D;
        load4<TI>(p, vi, x[u]);
        load4<TI>(p + D / 2, vi, x[u] + 4);
      }
#pragma unroll
      for (int u = 0; u < AT_ONCE; ++u) {
        norm_rope<D>(x[u], gain, gp != nullptr, r.eps, r.positions != nullptr, cs, sn);
        if (live && h + u < h1) {
          store4<TO>(dst + (h + u) * D, vo, x[u]);
          store4<TO>(dst + (h + u) * D + D / 2, vo, x[u] + 4);
        }
      }
    }
    return;
  }

  // ---- keys or values of some KV heads, of the runs that begin in this window ----
  __shared__ int slot_s[SPAN];
  __shared__ uint32_t flag_s[(SPAN + 31) / 32];  // rows that do not go on from the row before
  __shared__ uint32_t amax_s[3][GROUPS];  // a run's largest magnitude (its bits, which order as it does), three heads in turn
  extern __shared__ __align__(16) float angle_s[];  // [SPAN][LANES][8], where a CTA has several heads
  const bool is_k = task < a.kv_tasks / 2;
  const int kh0 = (is_k ? task : task - a.kv_tasks / 2) * a.kv_heads_per, kh1 = min(kh0 + a.kv_heads_per, r.n_kv_heads);
  const int ps = a.c.page_size;
  const int64_t n_slots = (int64_t)a.c.num_pages * ps;
  for (int i = threadIdx.x; i < 3 * GROUPS; i += kQkThreads) amax_s[0][i] = 0;
  int begins = 0;
  if (threadIdx.x < (SPAN + 31) / 32 * 32) {
    const int i = threadIdx.x, row = w0 + i;
    int s = -1;
    bool flag = true;
    if (i < SPAN && row < r.rows) {
      s = r.slots[row];
      const int before = row > 0 ? r.slots[row - 1] : -1;
      if (s < 0 || s >= n_slots) {
        if (s != -1 && task == 0 && i < GROUPS) report(a.err, SAR_ERR_BOUNDS, SITE_KV8_SLOT, row);
        s = -1;
      } else {
        flag = row == 0 || (s & (ps - 1)) == 0 || before != s - 1;
      }
    }
    const uint32_t m = __ballot_sync(0xffffffffu, flag);
    if (i < SPAN) slot_s[i] = s;
    if ((i & 31) == 0) flag_s[i >> 5] = m;
    begins = s >= 0 && flag && i < GROUPS;
  }
  if (!__syncthreads_or(begins)) return;  // (three windows of four, in chunks over pages of 64)
  // row i's run: the last flagged row up to i; -1 where i is in no run of this window
  auto run_of = [&](int i) -> int {
    if (slot_s[i] < 0) return -1;
    int w = i >> 5;
    uint32_t m = flag_s[w] & (0xffffffffu >> (31 - (i & 31)));
    while (m == 0 && w > 0) m = flag_s[--w];
    if (m == 0) return -1;
    const int s = (w << 5) + 31 - __clz(m);
    return s < GROUPS ? s : -1;
  };
  const int64_t ld = is_k ? r.ldk : r.ldv;
  const TI* src = static_cast<const TI*>(is_k ? r.k : r.v) + w0 * ld + 4 * l;
  const bool vec = is_k ? a.vec_k : a.vec_v;
  float* scales = is_k ? a.c.k_scales : a.c.v_scales;
  uint8_t* codes = static_cast<uint8_t*>(is_k ? a.c.k_codes : a.c.v_codes);
  int run[PASSES];
  bool one[PASSES];  // all rows of this warp are of one run
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    run[p] = run_of(p * GROUPS + grp);
    one[p] = __all_sync(0xffffffffu, run[p] == __shfl_sync(0xffffffffu, run[p], 0));
    // all of this CTA's heads of the row come to L2
    constexpr int LINES = D * (int)sizeof(TI) / 128;
    for (int k = l; run[p] >= 0 && k < (kh1 - kh0) * LINES; k += LANES)
      prefetch_l2(reinterpret_cast<const char*>(src - 4 * l + (p * GROUPS + grp) * ld + kh0 * D) + k * 128);
  }
  int turn = 0;
#pragma unroll 1
  for (int kh = kh0; kh < kh1; ++kh) {
    uint32_t* now = amax_s[turn];
    float x[PASSES][8], old[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int i = p * GROUPS + grp;
      old[p] = 0.f;
      if (run[p] >= 0) {
        load4<TI>(src + i * ld + kh * D, vec, x[p]);
        load4<TI>(src + i * ld + kh * D + D / 2, vec, x[p] + 4);
        const int first = slot_s[run[p]];
        // (the page goes on: what it has so far)
        if (first & (ps - 1)) old[p] = scales[(int64_t)(first >> a.shift) * a.c.n_kv_heads + kh];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[p][e] = 0.f;
      }
    }
    if (is_k && (r.k_gain || r.positions)) {
      float gain[8];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        gain[e] = r.k_gain ? r.k_gain[4 * l + e] : 1.f, gain[4 + e] = r.k_gain ? r.k_gain[D / 2 + 4 * l + e] : 1.f;
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        // (passes without a row of this window's runs, as all but the first of single tokens)
        if (!__any_sync(0xffffffffu, run[p] >= 0)) continue;
        float cs[4], sn[4];
        if (r.positions) {
          // formed once, kept for the CTA's other heads
          float4* kept = reinterpret_cast<float4*>(angle_s) + ((p * GROUPS + grp) * LANES + l) * 2;
          if (kh == kh0) {
            angles(a, run[p] >= 0 ? r.positions[w0 + p * GROUPS + grp] : 0, 4 * l, cs, sn);
            if (kh1 - kh0 > 1) kept[0] = make_float4(cs[0], cs[1], cs[2], cs[3]), kept[1] = make_float4(sn[0], sn[1], sn[2], sn[3]);
          } else {
            const float4 c = kept[0], t = kept[1];
            cs[0] = c.x, cs[1] = c.y, cs[2] = c.z, cs[3] = c.w;
            sn[0] = t.x, sn[1] = t.y, sn[2] = t.z, sn[3] = t.w;
          }
        }
        norm_rope<D>(x[p], gain, r.k_gain != nullptr, r.eps, r.positions != nullptr, cs, sn);
      }
    }
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      if (!__any_sync(0xffffffffu, run[p] >= 0)) continue;
      auto largest = [&]() -> uint32_t {
        float m = fabsf(x[p][0]);
#pragma unroll
        for (int e = 1; e < 7; e += 2) m = fmaxf(fmaxf(m, fabsf(x[p][e])), fabsf(x[p][e + 1]));  // (passes over NaN)
        m = fmaxf(fmaxf(m, fabsf(x[p][7])), 0.f);
        return one[p] ? __reduce_max_sync(0xffffffffu, __float_as_uint(m)) : __float_as_uint(group_max<LANES>(m));
      };
      uint32_t m = largest();
      if (__any_sync(0xffffffffu, m == 0x7f800000u)) {  // infinities become NaN, and count for nothing
#pragma unroll
        for (int e = 0; e < 8; ++e) x[p][e] = fabsf(x[p][e]) < INFINITY ? x[p][e] : NAN;
        m = largest();
      }
      if (one[p] ? (threadIdx.x & 31) == 0 : l == 0 && run[p] >= 0) atomicMax(&now[run[p]], m);
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      if (!__any_sync(0xffffffffu, run[p] >= 0)) continue;
      const int i = p * GROUPS + grp;
      const bool live = run[p] >= 0;
      if (!live) continue;
      const float scale = fmaxf(kv8_scale(__uint_as_float(now[run[p]])), old[p]);
      const int slot = slot_s[i];
      const int64_t unit = (int64_t)(slot >> a.shift) * a.c.n_kv_heads + kh;
      uint8_t* page = codes + unit * ps * D;
      const int o = (slot & (ps - 1)) * D + 4 * l;
      // a power of two's inverse, exactly, without the division; a page that another program
      // filled may go on under a scale that is none, and then h / s itself is rounded (by the
      // inverse it was off a little, and ties fell to the wrong code)
      const uint32_t bits = __float_as_uint(scale);
      float inv = __uint_as_float(0x7f000000u - bits);
      if (bits & 0x7fffffu) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[p][e] = __fdiv_rn(x[p][e], scale);
        inv = 1.f;  // (such a scale is the old one: nothing is rounded anew)
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float* u = x[p] + 4 * half;
        *reinterpret_cast<uint32_t*>(page + o + half * (D / 2)) =
            finite_e4m3x2(u[0] * inv, u[1] * inv) | finite_e4m3x2(u[2] * inv, u[3] * inv) << 16;
      }
      if (run[p] != i) continue;
      // the run's first row: the scale, and what the page held under a smaller one
      if (l == 0) scales[unit] = scale;
      if (old[p] > 0.f && scale > old[p]) {
        const float ratio = old[p] * inv;
#pragma unroll 1
        for (int j = 4 * l; j < (slot & (ps - 1)) * D; j += 4 * LANES) {
          const uint32_t c = *reinterpret_cast<const uint32_t*>(page + j);
          const float2 u = e4m3x2_floats(c), w = e4m3x2_floats(c >> 16);
          *reinterpret_cast<uint32_t*>(page + j) = finite_e4m3x2(u.x * ratio, u.y * ratio) | finite_e4m3x2(w.x * ratio, w.y * ratio) << 16;
        }
      }
    }
    // (a barrier lies between this and the head that writes there, as between the last reads and this)
    if (threadIdx.x < GROUPS) amax_s[turn == 0 ? 2 : turn - 1][threadIdx.x] = 0;
    turn = turn == 2 ? 0 : turn + 1;
  }
}

template <typename TI, typename TO>
int launch_qk(const QkArgs& a, cudaStream_t s) {
  const int D = a.r.head_dim;
  const int window = kQkThreads / (D / 8);
  const dim3 grid((unsigned)(((int64_t)a.r.rows + window - 1) / window), (unsigned)(a.kv_tasks + a.q_tasks + a.k_tasks));
  const int passes = (window + 63 + window - 1) / window;
  const size_t smem = a.kv_heads_per > 1 && a.r.positions ? (size_t)passes * kQkThreads * 32 : 0;
  if (smem > 0)
    SAR_TRY(ensure_smem_attr(D == 128 ? reinterpret_cast<const void*>(&qk_rows_kernel<TI, TO, 128>)
                                      : reinterpret_cast<const void*>(&qk_rows_kernel<TI, TO, 64>),
                             (int)smem, "qk rows: set smem attribute"));
  const cudaError_t e = D == 128 ? launch_pdl(qk_rows_kernel<TI, TO, 128>, grid, dim3(kQkThreads), smem, s, a)
                                 : launch_pdl(qk_rows_kernel<TI, TO, 64>, grid, dim3(kQkThreads), smem, s, a);
  if (e != cudaSuccess) return cuda_error(e, "qk rows launch");
  count_launches(1);
  return SAR_OK;
}

}  // namespace

int check_kv8(const sar_kv8* c, const char* what) {
  const std::string w(what);
  if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return set_error(SAR_ERR_INVALID_ARG, w + ": null cache");
  if (c->num_pages < 1 || c->n_kv_heads < 1) return set_error(SAR_ERR_INVALID_ARG, w + ": bad cache sizes");
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64)
    return set_error(SAR_ERR_UNSUPPORTED, w + ": pages of 16, 32 or 64 tokens");
  if (c->head_dim != 64 && c->head_dim != 128) return set_error(SAR_ERR_UNSUPPORTED, w + ": head_dim 64 or 128");
  // (a TMA row coordinate is a 32-bit number)
  if ((int64_t)c->num_pages * c->page_size > INT32_MAX ||
      (int64_t)c->num_pages * c->page_size * c->n_kv_heads > INT32_MAX)
    return set_error(SAR_ERR_UNSUPPORTED, w + ": cache rows above 2^31");
  if (!aligned_to(c->k_codes, 16) || !aligned_to(c->v_codes, 16) || !aligned_to(c->k_scales, 4) || !aligned_to(c->v_scales, 4))
    return set_error(SAR_ERR_INVALID_ARG, w + ": cache not aligned");
  return SAR_OK;
}

}  // namespace sar

using sar::aligned_to;
using sar::set_error;

extern "C" int sar_qk_norm_rope(const sar_qk_rows* rows, const sar_kv8* cache, void* stream) try {
  if (!rows) return set_error(SAR_ERR_INVALID_ARG, "qk_norm_rope: null rows");
  const sar_qk_rows& r = *rows;
  if (r.rows < 0 || r.n_q_heads < 0 || r.n_kv_heads < 0)
    return set_error(SAR_ERR_INVALID_ARG, "qk_norm_rope: bad sizes");
  if (r.type != SAR_TYPE_F16 && r.type != SAR_TYPE_BF16 && r.type != SAR_TYPE_F32)
    return set_error(SAR_ERR_INVALID_ARG, "qk_norm_rope: bad element type");
  if ((r.out_type != SAR_TYPE_F16 && r.out_type != SAR_TYPE_BF16) || (r.type != SAR_TYPE_F32 && r.out_type != r.type))
    return set_error(SAR_ERR_INVALID_ARG, "qk_norm_rope: the output type is 16-bit, and the rows' type where that is");
  if (r.head_dim != 64 && r.head_dim != 128) return set_error(SAR_ERR_UNSUPPORTED, "qk_norm_rope: head_dim 64 or 128");
  if (r.n_q_heads > 1024 || r.n_kv_heads > 1024) return set_error(SAR_ERR_UNSUPPORTED, "qk_norm_rope: more than 1024 heads");
  if (r.rows > 1 << 30) return set_error(SAR_ERR_UNSUPPORTED, "qk_norm_rope: more than 2^30 rows");
  if ((r.q_gain || r.k_gain) && !(r.eps >= 0.f)) return set_error(SAR_ERR_INVALID_ARG, "qk_norm_rope: negative eps");
  if (r.positions && !(r.rope_base > 0.f && r.rope_base < INFINITY))
    return set_error(SAR_ERR_INVALID_ARG, "qk_norm_rope: rope_base must be positive and finite");
  if (cache) {
    SAR_TRY(sar::check_kv8(cache, "qk_norm_rope"));
    if (cache->n_kv_heads != r.n_kv_heads || cache->head_dim != r.head_dim)
      return set_error(SAR_ERR_INVALID_ARG, "qk_norm_rope: the cache has other heads");
  }
  if (r.rows == 0) return SAR_OK;
  const bool q_rows = r.q && r.n_q_heads > 0;
  if ((r.q != nullptr) != (r.q_out != nullptr)) return set_error(SAR_ERR_INVALID_ARG, "qk_norm_rope: q and q_out go together");
  if (r.k_out && !r.k) return set_error(SAR_ERR_INVALID_ARG, "qk_norm_rope: k_out without k");
  if (cache && (!r.k || !r.v || !r.slots)) return set_error(SAR_ERR_INVALID_ARG, "qk_norm_rope: a cache needs k, v and slots");
  if (cache && r.k_out == r.k)
    return set_error(SAR_ERR_INVALID_ARG, "qk_norm_rope: with a cache k_out is not k");
  const int64_t dq = (int64_t)r.n_q_heads * r.head_dim, dk = (int64_t)r.n_kv_heads * r.head_dim;
  if ((q_rows && (r.ldq < dq || r.ldq_out < dq)) || (r.k && r.ldk < dk) || (r.k_out && r.ldk_out < dk) ||
      (cache && r.ldv < dk))
    return set_error(SAR_ERR_INVALID_ARG, "qk_norm_rope: rows shorter than their heads");
  const uintptr_t size = r.type == SAR_TYPE_F32 ? 4 : 2;
  if (!aligned_to(r.q, size) || !aligned_to(r.k, size) || !aligned_to(r.v, size) || !aligned_to(r.q_out, 2) ||
      !aligned_to(r.k_out, 2) || !aligned_to(r.q_gain, 4) || !aligned_to(r.k_gain, 4) || !aligned_to(r.positions, 4) ||
      !aligned_to(r.slots, 4))
    return set_error(SAR_ERR_INVALID_ARG, "qk_norm_rope: array not aligned to its element");
  if ((q_rows && r.q_out == r.q && (r.type == SAR_TYPE_F32 || r.ldq != r.ldq_out)) ||
      (r.k_out && r.k_out == r.k && (r.type == SAR_TYPE_F32 || r.ldk != r.ldk_out)))
    return set_error(SAR_ERR_INVALID_ARG, "qk_norm_rope: rows written over have the same 16-bit type and stride");

  sar::QkArgs a = {};
  a.r = r;
  if (cache) a.c = *cache;
  if (!q_rows) a.r.n_q_heads = 0;
  a.shift = !cache ? 0 : cache->page_size == 16 ? 4 : cache->page_size == 32 ? 5 : 6;
  auto vec = [](const void* p, int64_t ld, uintptr_t piece, uintptr_t el) {
    return aligned_to(p, piece) && ld * (int64_t)el % (int64_t)piece == 0;
  };
  a.vec_q = vec(r.q, r.ldq, 4 * size, size);
  a.vec_k = vec(r.k, r.ldk, 4 * size, size);
  a.vec_v = vec(r.v, r.ldv, 4 * size, size);
  a.vec_qo = vec(r.q_out, r.ldq_out, 8, 2);
  a.vec_ko = vec(r.k_out, r.ldk_out, 8, 2);
  // heads to a CTA: as few as let all CTAs be resident at once (two to an SM), and no
  // more than amortise a row's angles and slots
  const int64_t windows = ((int64_t)r.rows * (r.head_dim / 8) + sar::kQkThreads - 1) / sar::kQkThreads;
  auto up = [](int n, int per) { return (n + per - 1) / per; };
  a.q_heads_per = a.kv_heads_per = 1;
  while (true) {
    a.q_tasks = up(a.r.n_q_heads, a.q_heads_per);
    a.k_tasks = r.k_out ? up(r.n_kv_heads, a.q_heads_per) : 0;
    a.kv_tasks = cache ? 2 * up(r.n_kv_heads, a.kv_heads_per) : 0;
    if (windows * (a.q_tasks + a.k_tasks + a.kv_tasks) <= 2 * sar::num_sms()) break;
    if (a.q_heads_per < 16 && (a.kv_heads_per >= 4 || a.q_tasks + a.k_tasks >= a.kv_tasks))
      a.q_heads_per *= 2;
    else if (a.kv_heads_per < 4)
      a.kv_heads_per *= 2;
    else
      break;
  }
  if (a.q_tasks + a.k_tasks + a.kv_tasks == 0) return SAR_OK;
  if (r.positions) {
    // (kept for the thread's next call: they depend on these two numbers alone)
    static thread_local float base = 0.f;
    static thread_local int dim = 0;
    static thread_local uint64_t turn[64];
    if (base != r.rope_base || dim != r.head_dim) {
      for (int i = 0; i < r.head_dim / 2; ++i) {
        const double t = pow((double)r.rope_base, -2.0 * i / r.head_dim) / 6.283185307179586476925286766559;
        turn[i] = (uint64_t)ldexp(t - floor(t), 64);
      }
      base = r.rope_base;
      dim = r.head_dim;
    }
    for (int i = 0; i < r.head_dim / 2; ++i) a.turn[i] = turn[i];
  }
  SAR_TRY(sar::op_flags(&a.err));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (r.type == SAR_TYPE_F32)
    return r.out_type == SAR_TYPE_BF16 ? sar::launch_qk<float, __nv_bfloat16>(a, s) : sar::launch_qk<float, __half>(a, s);
  return r.type == SAR_TYPE_BF16 ? sar::launch_qk<__nv_bfloat16, __nv_bfloat16>(a, s) : sar::launch_qk<__half, __half>(a, s);
} catch (...) {
  return sar::entry_failed("qk_norm_rope");
}
