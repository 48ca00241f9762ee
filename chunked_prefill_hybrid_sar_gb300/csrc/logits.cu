// What a request asks of its logits between the LM head and the pick: penalties
// for tokens it has seen, biases, a grammar's mask; and the table of seen tokens
// that the penalties read.
//
// Token state: uint16 [slots][ld], one row per live request.  Bit 15: the token
// is in the request's prompt; low 15 bits: how often the request has generated
// it (stays at 32767).  16 bits per token because the table is read whole at
// every pick: at 4 bytes it would be as much traffic as the logits themselves.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "tc05.cuh"

namespace sar {

namespace {

// ---- token state -------------------------------------------------------------

constexpr int kStateThreads = 512;
constexpr int kStateSpan = 8192;  // tokens per CTA of a resetting call: 32 KB of counters

struct StateArgs {
  uint16_t* state;
  int64_t ld;
  int n_slots, vocab;
  const int32_t* slots;
  int n;
  const int32_t* offsets;
  const int32_t* tokens;
  int n_tokens;
  const int32_t* prompt_lens;
  int vec;  // rows are 16-byte aligned
  int* err;
};

// A resetting call: CTA (span, row) counts the row's tokens that fall into its
// span of the vocabulary in shared memory and writes the span whole, so the row
// is neither cleared nor read first.  Every span's CTA reads the row's list
// (from L2 after the first), eight tokens of a thread at a time.  Bound by the
// latency of that chain of loads, not by bytes (64 histories of up to 8192 tokens
// over 64000: 7.1 us; 8.6 with one token at a time).  Shared-memory atomics on
// whole numbers: the result does not depend on their order.
__global__ void __launch_bounds__(kStateThreads) state_reset_kernel(const StateArgs a) {
  __shared__ __align__(16) uint32_t cnt[kStateSpan];
  pdl_wait();
  pdl_launch_dependents();
  const int r = blockIdx.y, lo = blockIdx.x * kStateSpan, hi = min(a.vocab, lo + kStateSpan);
  const bool first_cta = blockIdx.x == 0;
  // (all on their way at once)
  const int slot = a.slots[r], b = a.offsets[r], e = a.offsets[r + 1], prompt = a.prompt_lens ? a.prompt_lens[r] : 0;
  int again = 0;
  for (int i = threadIdx.x; i < r; i += kStateThreads) again |= a.slots[i] == slot;
  for (int i = threadIdx.x; i < kStateSpan / 4; i += kStateThreads) reinterpret_cast<uint4*>(cnt)[i] = make_uint4(0, 0, 0, 0);
  again = __syncthreads_or(again);
  if (slot < 0 || slot >= a.n_slots || again) {
    if (first_cta && threadIdx.x == 0) report(a.err, SAR_ERR_BOUNDS, SITE_STATE_SLOT, r);
    return;
  }
  if (b < 0 || e < b || e > a.n_tokens) {
    if (first_cta && threadIdx.x == 0) report(a.err, SAR_ERR_BOUNDS, SITE_STATE_OFFSET, r);
    return;
  }
  const int n_prompt = min(max(prompt, 0), e - b);
  constexpr int kU = 8;  // tokens of a thread on their way at once
  for (int i0 = b + (int)threadIdx.x; i0 < e; i0 += kU * kStateThreads) {
    int t[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) t[u] = i0 + u * kStateThreads < e ? __ldg(a.tokens + i0 + u * kStateThreads) : lo;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int i = i0 + u * kStateThreads;
      if (i >= e) break;
      if (t[u] >= lo && t[u] < hi) {
        if (i - b < n_prompt)
          atomicOr(&cnt[t[u] - lo], 0x80000000u);
        else
          atomicAdd(&cnt[t[u] - lo], 1u);
      } else if (first_cta && (t[u] < 0 || t[u] >= a.vocab)) {
        report(a.err, SAR_ERR_BOUNDS, SITE_STATE_TOKEN, i);
      }
    }
  }
  __syncthreads();
  auto packed = [&](int i) { return (uint32_t)min(cnt[i] & 0x7fffffffu, 0x7fffu) | (cnt[i] >> 31 << 15); };
  uint16_t* row = a.state + (int64_t)slot * a.ld + lo;
  const int n = hi - lo;
  if (a.vec) {
    for (int i = 8 * threadIdx.x; i + 8 <= n; i += 8 * kStateThreads) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = packed(i + 2 * k) | packed(i + 2 * k + 1) << 16;
      *reinterpret_cast<uint4*>(row + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    for (int i = (n & ~7) + (int)threadIdx.x; i < n; i += kStateThreads) row[i] = (uint16_t)packed(i);
  } else {
    for (int i = threadIdx.x; i < n; i += kStateThreads) row[i] = (uint16_t)packed(i);
  }
}

__device__ __forceinline__ void state_count(uint16_t* at, bool prompt) {
  unsigned short* p = reinterpret_cast<unsigned short*>(at);
  unsigned short old = *p, was;
  do {
    was = old;
    const unsigned short now = prompt                        ? (unsigned short)(was | 0x8000u)
                               : (was & 0x7fffu) == 0x7fffu ? was
                                                            : (unsigned short)(was + 1);
    if (now == was) return;
    old = atomicCAS(p, was, now);
  } while (old != was);
}

// An appending call: one thread per token, its row found by bisection, and one per
// row that reports offsets which are out of range or fall (such a row may hold no
// token that a thread could meet).  Where all offsets rise the bisection ends at
// the token's row; where some fall it ends at one row at most.
__global__ void __launch_bounds__(256) state_append_kernel(const StateArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < a.n) {
    const int b = a.offsets[i], e = a.offsets[i + 1];
    if (b < 0 || e < b || e > a.n_tokens) report(a.err, SAR_ERR_BOUNDS, SITE_STATE_OFFSET, i);
  }
  if (i >= a.n_tokens) return;
  int lo = 0, hi = a.n;  // the last row that begins at or before i
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.offsets[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  const int b = a.offsets[lo], e = a.offsets[lo + 1];
  if (i < b || i >= e) return;          // a token of no row
  if (b < 0 || e > a.n_tokens) return;  // a row that is passed over (reported above)
  const int slot = a.slots[lo], t = a.tokens[i];
  if (slot < 0 || slot >= a.n_slots) {
    report(a.err, SAR_ERR_BOUNDS, SITE_STATE_SLOT, lo);
  } else if (t < 0 || t >= a.vocab) {
    report(a.err, SAR_ERR_BOUNDS, SITE_STATE_TOKEN, i);
  } else {
    state_count(a.state + (int64_t)slot * a.ld + t, a.prompt_lens && i - b < a.prompt_lens[lo]);
  }
}

// ---- logits --------------------------------------------------------------------

constexpr int kCtlThreads = 512;  // that work on tokens; one more warp fetches
constexpr int kCtlTile = 8192;    // tokens per CTA and step
constexpr int kCtlStages = 2;     // steps on their way
constexpr int kCtlLeast = 4096;   // tokens that a CTA is started for
constexpr int kCtlSpan = 32768;   // tokens per pass over a row's biases: two bitmaps of 4 KB
constexpr long kCtlPerSm = 2;     // CTAs that fit an SM's shared memory
// Biases of a row.  A span's work on its list has to stay far below the waits' 2 s
// (2^24 biases that repeat every token of a span: 1.6 s).
constexpr int kCtlMostBiases = 1 << 21;
constexpr int kCtlSlice = 64;     // tokens whose repeated biases a warp adds up at a time

struct CtlArgs {
  const void* x;
  int64_t ldx;
  void* y;
  int64_t ldy;
  int32_t* picks;
  int vocab, chunk;  // tokens per CTA of a row's cluster
  sar_logit_controls c;
  int* err;
};

// What a row's tokens are changed by.
struct RowCtl {
  const uint16_t* state = nullptr;  // null: no penalties
  const uint32_t* mask = nullptr;   // null: every token allowed
  float rep = 1.f, pres = 0.f, freq = 0.f;
  float inv_rep = 1.f;               // correctly rounded
  uint32_t ordinary = 0x40000000u;   // 2^64 over 2^-64 as bit patterns; 0: always divide
};

// The penalties, in the order and with the roundings the header gives (no fused
// multiply-add: f * count is rounded before it is taken off).  x / rep is formed
// with the row's 1 / rep and corrected by its exact remainder, which rounds it
// correctly (Markstein 1990) while nothing on the way over- or underflows;
// otherwise it is divided.  s != 0.
__device__ __forceinline__ float penalised(float x, uint32_t s, const RowCtl& w) {
  const uint32_t made = s & 0x7fffu;
  const float q = __fmul_rn(x, w.inv_rep), less = __fmul_rn(x, w.rep);
  const float div = __fmaf_rn(-__fmaf_rn(q, w.rep, -x), w.inv_rep, q);
  // |x| outside [2^-64, 2^64), or a factor of unusual size
  const bool odd = (__float_as_uint(x) & 0x7fffffffu) - 0x1f800000u >= w.ordinary;
  float y = x > 0.f ? div : less;
  if (__builtin_expect(odd, 0) && x > 0.f) y = __fdiv_rn(x, w.rep);
  y = __fsub_rn(y, __fmul_rn(w.freq, (float)made));
  return made ? __fsub_rn(y, w.pres) : y;
}

// The larger logit, then the lower token; NaN and -inf never come here.
struct Best {
  float v = -INFINITY;
  int i = 0x7fffffff;
  // (of tokens that come in rising order only a larger one counts)
  __device__ __forceinline__ void take_later(float x, int t) {
    if (x > v) {
      v = x;
      i = t;
    }
  }
  // the best of the warp's lanes, in all of them
  __device__ __forceinline__ void warp() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float x = __shfl_xor_sync(0xffffffffu, v, o);
      const int t = __shfl_xor_sync(0xffffffffu, i, o);
      take(x, t);
    }
  }
  __device__ __forceinline__ void take(float x, int t) {
    if (x > v || (x == v && t < i && x > -INFINITY)) {
      v = x;
      i = t;
    }
  }
};

// The part of a tile's array that a bulk copy can bring to shared memory: the
// elements [lo, hi) of [t0, t1) that lie in whole 16-byte pieces.  The few others
// (rows at odd addresses) are read where they are.
struct Window {
  int lo, hi;
};
__device__ __forceinline__ Window window(const void* base, int t0, int t1, int size) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(base) + (uintptr_t)t0 * size;
  const uintptr_t e = reinterpret_cast<uintptr_t>(base) + (uintptr_t)t1 * size;
  Window w = {t0 + (int)((0 - p) & 15) / size, t1 - (int)(e & 15) / size};
  if (w.hi <= w.lo) w.lo = w.hi = t0;
  return w;
}

// Where a stage's arrays begin and end.
struct Placed {
  Window x, s, m;  // logits and token state by token, mask by word
};

// Masks K tokens (bit k of `on`: allowed) and takes the largest into `best`, those
// of `raw` left out of both.  A NaN loses; which token leads is looked up only
// where one of them is above `bar`, what the warp had reached by the tile before
// (a lane's own best would be passed by some lane of the warp at nearly every step).
template <int K, typename Token>
__device__ __forceinline__ void lead(float (&v)[K], uint32_t on, uint32_t raw, float bar, Best& best, const Token& token) {
  const uint32_t off = ~on & ~raw & ((1u << K) - 1);
  if (off) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (off >> k & 1) v[k] = -INFINITY;
  }
  float top = v[0];
#pragma unroll
  for (int k = 1; k < K; ++k) top = fmaxf(top, v[k]);
  if (top > bar) {  // (also where a token left out has the largest)
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (!(raw >> k & 1)) best.take_later(v[k], token(k));
  }
}

template <typename T>
__device__ __forceinline__ float ctl_load(const T* p) {
  if constexpr (sizeof(T) == 4)
    return *p;
  else
    return Elem<T>::to(*p);
}
template <typename T>
__device__ __forceinline__ void ctl_store(T* p, float v) {
  if constexpr (sizeof(T) == 4)
    *p = v;
  else
    *p = Elem<T>::from(v);
}

// Finishes the tokens of [s0, s1) that a long list names repeatedly (`twice`, in
// shared memory): a warp takes a slice of 64 tokens that holds such, reads the list
// once (its first 512 entries in shared memory) and adds up their biases in list
// order; lane k holds the sums of the slice's tokens k and 32 + k.  Returns the best
// of this lane's tokens.  256 x 64000 written, 1300 biases a row: 67 us (157 with a
// search per entry; 513 a row 41 and 39).  Not inlined: inside the kernel it made
// the dense pass spill (the same without a list 21.7 us, and 20.8 so).
template <typename T>
__device__ __noinline__ Best finish_repeated(const T* x, T* y, const int32_t* tokens, const float* values, int b0, int b1,
                                             int s0, int s1, const uint32_t* twice, const int* list_t, const float* list_v,
                                             const RowCtl w) {
  Best best;
  const int lane = threadIdx.x & 31;
  for (int q = threadIdx.x >> 5; q * kCtlSlice < s1 - s0; q += kCtlThreads / 32) {
    const uint32_t rep0 = twice[2 * q], rep1 = twice[2 * q + 1];
    if (!(rep0 | rep1)) continue;
    const int base = s0 + q * kCtlSlice;
    float sum0 = -0.f, sum1 = -0.f;  // (what adding a first bias leaves as it is)
    constexpr int kU = 8;            // loads of a lane under way at once
    static_assert(kCtlThreads % (32 * kU) == 0, "the list's head is whole steps");
    for (int e0 = b0; e0 < b1; e0 += 32 * kU) {
      const bool head = e0 - b0 < kCtlThreads;  // (whole steps are)
      const int* at_t = head ? list_t : tokens;
      const float* at_v = head ? list_v : values;
      const int first = head ? e0 - b0 : e0;
      int t[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int e = 32 * u + lane;
        t[u] = e0 + e < b1 ? at_t[first + e] : -1;
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint32_t at = (uint32_t)t[u] - (uint32_t)base;  // (beyond the slice also where t is out of range)
        const bool in = at < kCtlSlice && ((at < 32 ? rep0 : rep1) >> (at & 31) & 1);
        uint32_t hits = __ballot_sync(0xffffffffu, in);
        if (!hits) continue;
        const float v = in ? at_v[first + 32 * u + lane] : 0.f;
        for (; hits; hits &= hits - 1) {  // in list order
          const int from = __ffs(hits) - 1;
          const uint32_t to = __shfl_sync(0xffffffffu, at, from);
          const float more = __shfl_sync(0xffffffffu, v, from);
          if (to == (uint32_t)lane) sum0 = __fadd_rn(sum0, more);
          if (to == (uint32_t)lane + 32) sum1 = __fadd_rn(sum1, more);
        }
      }
    }
    for (int h = 0; h < 2; ++h) {
      if (!((h ? rep1 : rep0) >> lane & 1)) continue;
      const int t = base + 32 * h + lane;
      const uint32_t seen = w.state ? w.state[t] : 0, on = w.mask ? __ldg(w.mask + (t >> 5)) >> (t & 31) & 1 : 1;
      float v = ctl_load<T>(x + t);
      v = on ? __fadd_rn(seen ? penalised(v, seen, w) : v, h ? sum1 : sum0) : -INFINITY;
      best.take(v, t);
      if (y) ctl_store<T>(y + t, v);
    }
  }
  return best;
}

// One pass over the logits: a cluster of CTAs shares each row, every CTA takes
// one stretch of the vocabulary and the stretches' best tokens meet through
// distributed shared memory, so that a lone row is read by as many SMs as the
// cluster has CTAs, and one launch without a workspace does penalties, biases,
// mask, store and pick.
//
// Logits, token state and mask words come in tiles of 8192 tokens by bulk copies
// of a warp of its own, two tiles at a time: with ordinary loads a thread's
// registers hold too little of what has to be on its way (256 x 64000 fp32, pick
// only: 30 us, and 15.4 so).  With everything on and the logits written that size
// takes 36 us, 4.5 TB/s.  A further tile costs what reading HBM takes (256 rows,
// penalties and pick, inputs that rotate through 400 MB and more: 15.9 us at 32768
// tokens, 22.8 at 65536, so 7.2 TB/s of logits and state between them); a CTA's
// start, first loads and join cost about 6 us, and 256 rows leave 104 SMs with two
// CTAs and 48 with one.  One row of 32000, eight CTAs: 6.1 us, the chain of indexes,
// state, a cluster's join and a write.
//
// Biases come as a list per row.  Their tokens are marked in a bitmap of the
// stretch; the dense pass leaves marked tokens as they are, and the list's
// threads then finish one each: penalties from the original logit, the token's
// biases added up in list order, mask.  A second bitmap marks tokens that are
// listed again.  In a list of up to 512 those alone search it, in shared memory;
// in a longer one, where every such search would make the work grow with the
// length's square, each warp takes slices of 64 tokens that hold a repeated one
// and reads the list once for each.
//
// VEC: rows at 16-byte boundaries; a thread takes 4 neighbouring tokens at a
// time, otherwise single ones.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kCtlThreads + 32, kCtlPerSm) logits_control_kernel(const CtlArgs a) {
  extern __shared__ __align__(16) uint8_t stage_mem[];  // [stages] logits, state, mask words of a tile
  __shared__ uint32_t listed[kCtlSpan / 32], twice[kCtlSpan / 32];
  __shared__ int list_t[kCtlThreads];  // the list's first entries
  __shared__ float list_v[kCtlThreads];
  __shared__ __align__(8) uint64_t full[kCtlStages], empty[kCtlStages];
  __shared__ Placed placed[kCtlStages];
  __shared__ float best_v[kCtlThreads / 32];
  __shared__ int best_i[kCtlThreads / 32];
  __shared__ Best cta_best;
  constexpr uint32_t kState = kCtlTile * sizeof(T), kMask = kState + kCtlTile * 2, kStage = kMask + kCtlTile / 8;
  const int r = blockIdx.y, rank = blockIdx.x, tid = threadIdx.x;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const bool tells = rank == 0 && tid == 0;
  if (tid == 0) {
    for (int i = 0; i < kCtlStages; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), kCtlThreads / 32);
    }
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  const sar_logit_controls& c = a.c;
  const T* x = static_cast<const T*>(a.x) + (int64_t)r * a.ldx;
  T* y = a.y ? static_cast<T*>(a.y) + (int64_t)r * a.ldy : nullptr;
  const int lo = rank * a.chunk, hi = min(a.vocab, lo + a.chunk);
  const int tiles = hi > lo ? (hi - lo + kCtlTile - 1) / kCtlTile : 0;
  RowCtl w;

  // The fetching warp brings tile i to its stage: the logits, which wait for no
  // index, and then the rest.
  const bool fetches = warp == kCtlThreads / 32;
  const uint32_t stage0 = __shfl_sync(0xffffffffu, smem_u32(stage_mem), 0), full0 = __shfl_sync(0xffffffffu, smem_u32(full), 0);
  auto fetch_x = [&](int i) {
    const int t0 = lo + i * kCtlTile, t1 = min(hi, t0 + kCtlTile);
    const uint32_t st = stage0 + (uint32_t)(i % kCtlStages) * kStage, bar = full0 + (uint32_t)(i % kCtlStages) * 8;
    const Window wx = window(x, t0, t1, sizeof(T));
    const uint32_t bytes = (uint32_t)((wx.hi - wx.lo) * sizeof(T));
    if (elect_one()) {
      placed[i % kCtlStages].x = wx;
      if (bytes > 0) {
        asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
        bulk_g2s(st, x + wx.lo, bytes, bar);
      }
    }
    __syncwarp();
  };
  auto fetch_rest = [&](int i) {
    const int t0 = lo + i * kCtlTile, t1 = min(hi, t0 + kCtlTile);
    const uint32_t st = stage0 + (uint32_t)(i % kCtlStages) * kStage, bar = full0 + (uint32_t)(i % kCtlStages) * 8;
    const Window ws = w.state ? window(w.state, t0, t1, 2) : Window{0, 0};
    const Window wm = w.mask ? window(w.mask, t0 >> 5, (t1 + 31) >> 5, 4) : Window{0, 0};
    if (elect_one()) {
      placed[i % kCtlStages].s = ws;
      placed[i % kCtlStages].m = wm;
      mbar_expect_tx(bar, (uint32_t)((ws.hi - ws.lo) * 2 + (wm.hi - wm.lo) * 4));
      if (ws.hi > ws.lo) bulk_g2s(st + kState, w.state + ws.lo, (uint32_t)(ws.hi - ws.lo) * 2, bar);
      if (wm.hi > wm.lo) bulk_g2s(st + kMask, w.mask + wm.lo, (uint32_t)(wm.hi - wm.lo) * 4, bar);
    }
    __syncwarp();
  };
  if (fetches)
    for (int i = 0; i < min(tiles, kCtlStages); ++i) fetch_x(i);

  // the row's indexes and factors, all on their way at once
  int slot = c.state ? c.slots[r] : -1;
  int m = !c.mask ? -1 : c.mask_rows ? c.mask_rows[r] : r;
  int b0 = c.bias_offsets ? c.bias_offsets[r] : 0, b1 = c.bias_offsets ? c.bias_offsets[r + 1] : 0;
  if (c.repetition) w.rep = c.repetition[r];
  if (c.presence) w.pres = c.presence[r];
  if (c.frequency) w.freq = c.frequency[r];
  if (c.state && (slot >= c.n_slots || slot < -1)) {
    if (tells) report(a.err, SAR_ERR_BOUNDS, SITE_CONTROL_SLOT, r);
    slot = -1;
  }
  if (slot >= 0 && (c.repetition || c.presence || c.frequency)) w.state = c.state + (int64_t)slot * c.state_ld;
  if (c.mask && (m >= c.n_masks || m < -1)) {
    if (tells) report(a.err, SAR_ERR_BOUNDS, SITE_CONTROL_MASK, r);
    m = -1;
  }
  w.inv_rep = __frcp_rn(w.rep);
  if (!(w.rep > 1e-10f && w.rep < 1e10f)) w.ordinary = 0;
  if (m >= 0) w.mask = c.mask + (int64_t)m * c.mask_ld;
  if (b0 < 0 || b1 < b0 || b1 > c.n_biases || b1 - b0 > kCtlMostBiases) {
    if (tells) report(a.err, SAR_ERR_BOUNDS, SITE_CONTROL_BIAS, r);
    b0 = b1 = 0;
  }
  if (fetches) {
    for (int i = 0; i < min(tiles, kCtlStages); ++i) fetch_rest(i);
    int i = kCtlStages;  // tiles before it are on their way
    for (; i < tiles; ++i) {
      // (a stage that was not given back stays as it is: no tile overwrites one that is being read)
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&empty[i % kCtlStages]), (uint32_t)(i / kCtlStages - 1) & 1u, a.err,
                                             SITE_CONTROL_PIPE)))
        break;
      fetch_x(i);
      fetch_rest(i);
    }
    // whatever the working warps did, no copy is under way when the CTA leaves
    for (int j = max(0, i - kCtlStages); j < min(i, tiles); ++j)
      mbar_wait(smem_u32(&full[j % kCtlStages]), (uint32_t)(j / kCtlStages) & 1u, a.err, SITE_CONTROL_PIPE);
  }
  // the working threads alone
  auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kCtlThreads) : "memory"); };

  Best best;
  bool alive = true;      // false once a wait gave up: what this thread has read is not the row's
  float bar = -INFINITY;  // the warp's best logit of the tiles before
  for (int s0 = lo; s0 < hi && tid < kCtlThreads; s0 += kCtlSpan) {
    const int s1 = min(hi, s0 + kCtlSpan);
    // this thread's first listed token of the span, with what finishing it reads
    // loaded ahead of the dense pass (which leaves it as it is)
    int et = -1;
    float ev = 0.f, ex = 0.f;
    uint32_t es = 0, em = 1;
    if (b1 > b0) {
      sync();  // the last span's bitmaps are done with
      for (int i = tid; i < kCtlSpan / 32; i += kCtlThreads) listed[i] = twice[i] = 0;
      sync();
      for (int e = b0 + tid; e < b1; e += kCtlThreads) {
        const int t = __ldg(c.bias_tokens + e);
        if (e < b0 + kCtlThreads) {
          ev = __ldg(c.bias_values + e);
          list_t[tid] = t;
          list_v[tid] = ev;
        }
        if (t >= s0 && t < s1) {
          const uint32_t bit = 1u << (t & 31);
          if (atomicOr(&listed[(t - s0) >> 5], bit) & bit) atomicOr(&twice[(t - s0) >> 5], bit);
          if (e < b0 + kCtlThreads) {
            et = t;
            ex = ctl_load<T>(x + t);
            if (w.state) es = w.state[t];
            if (w.mask) em = __ldg(w.mask + (t >> 5)) >> (t & 31) & 1;
          }
        } else if (rank == 0 && s0 == lo && (t < 0 || t >= a.vocab)) {
          report(a.err, SAR_ERR_BOUNDS, SITE_CONTROL_BIAS, e);
        }
      }
      sync();
    }
    // (spans and tiles start at multiples of 32 tokens)
    for (int t0 = s0; t0 < s1; t0 += kCtlTile) {
      const int i = (t0 - lo) / kCtlTile, t1 = min(s1, t0 + kCtlTile);
      alive &= mbar_wait(smem_u32(&full[i % kCtlStages]), (uint32_t)(i / kCtlStages) & 1u, a.err, SITE_CONTROL_PIPE,
                         alive ? kWaitLimitNs : 0);  // (going on keeps the warp together and the barriers matched)
      const uint8_t* st = stage_mem + (i % kCtlStages) * kStage;
      const T* xs = reinterpret_cast<const T*>(st);
      const uint16_t* ss = reinterpret_cast<const uint16_t*>(st + kState);
      const uint32_t* ms = reinterpret_cast<const uint32_t*>(st + kMask);
      const Placed at = placed[i % kCtlStages];
      auto mask_bits = [&](int t) {  // the mask from token t on, bit 0 first
        const int q = t >> 5;
        return (q >= at.m.lo && q < at.m.hi ? ms[q - at.m.lo] : __ldg(w.mask + q)) >> (t & 31);
      };
      auto listed_bits = [&](int t) { return listed[(t - s0) >> 5] >> (t & 31); };
      // a lone token (at a row's or a tile's ends)
      auto one = [&](int t) {
        float v = ctl_load<T>(x + t);
        if (!(b1 > b0 && (listed_bits(t) & 1))) {
          const uint32_t seen = w.state ? w.state[t] : 0;
          if (seen) v = penalised(v, seen, w);
          if (w.mask && !(mask_bits(t) & 1)) v = -INFINITY;
          best.take_later(v, t);
        }
        if (y) ctl_store<T>(y + t, v);
      };
      // Eight tokens at once: the row's switches and the lead are looked at once for
      // all of them (a token alone: 25 instructions each, which was the limit).
      int done = t0;  // tokens before it are worked on
      constexpr int kHalf = 4 * kCtlThreads;  // two groups of four to a thread
      for (; VEC && done + 2 * kHalf <= t1; done += 2 * kHalf) {
        const int p = done - t0 + tid * 4, t = t0 + p;
        float v[8];
        if constexpr (sizeof(T) == 4) {
          const float4 f = *reinterpret_cast<const float4*>(xs + p), g = *reinterpret_cast<const float4*>(xs + kHalf + p);
          v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w, v[4] = g.x, v[5] = g.y, v[6] = g.z, v[7] = g.w;
        } else {
          const uint2 f = *reinterpret_cast<const uint2*>(xs + p), g = *reinterpret_cast<const uint2*>(xs + kHalf + p);
          v[0] = Elem<T>::lo(f.x), v[1] = Elem<T>::hi(f.x), v[2] = Elem<T>::lo(f.y), v[3] = Elem<T>::hi(f.y);
          v[4] = Elem<T>::lo(g.x), v[5] = Elem<T>::hi(g.x), v[6] = Elem<T>::lo(g.y), v[7] = Elem<T>::hi(g.y);
        }
        uint32_t raw = 0, on = 0xffu;  // bit k: left to the list; allowed
        if (b1 > b0) raw = (listed_bits(t) & 0xfu) | (listed_bits(t + kHalf) & 0xfu) << 4;
        if (w.mask) on = (mask_bits(t) & 0xfu) | (mask_bits(t + kHalf) & 0xfu) << 4;
        if (w.state) {
          const uint2 f = *reinterpret_cast<const uint2*>(ss + p), g = *reinterpret_cast<const uint2*>(ss + kHalf + p);
          if (f.x | f.y | g.x | g.y) {  // (most of a vocabulary is unseen)
            const uint32_t s[4] = {f.x, f.y, g.x, g.y};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t seen = k & 1 ? s[k / 2] >> 16 : s[k / 2] & 0xffffu;
              if (__builtin_expect(seen != 0, 0) && !(raw >> k & 1)) v[k] = penalised(v[k], seen, w);
            }
          }
        }
        lead(v, on, raw, bar, best, [&](int k) { return t + (k & 3) + (k >> 2) * kHalf; });
        if (y) {
          if constexpr (sizeof(T) == 4) {
            __stcs(reinterpret_cast<float4*>(y + t), make_float4(v[0], v[1], v[2], v[3]));
            __stcs(reinterpret_cast<float4*>(y + t + kHalf), make_float4(v[4], v[5], v[6], v[7]));
          } else {
            __stcs(reinterpret_cast<uint2*>(y + t), make_uint2(Elem<T>::pack(v[0], v[1]), Elem<T>::pack(v[2], v[3])));
            __stcs(reinterpret_cast<uint2*>(y + t + kHalf), make_uint2(Elem<T>::pack(v[4], v[5]), Elem<T>::pack(v[6], v[7])));
          }
        }
      }
      if (done < t1) {
        constexpr int kU = 4;
        // what is in shared memory of both arrays; the few others, at the ends, one by one
        const int i0 = max(done, w.state ? max(at.x.lo, at.s.lo) : at.x.lo);
        const int i1 = max(i0, w.state ? min(at.x.hi, at.s.hi) : at.x.hi);
        if (done + tid < min(i0, t1)) one(done + tid);
        const T* xi = xs - at.x.lo;
        const uint16_t* si = ss - at.s.lo;
        for (int t = i0 + tid; t < i1; t += kU * kCtlThreads) {
          float v[kU];
          uint32_t s[kU], raw = 0, on = (1u << kU) - 1;
#pragma unroll
          for (int k = 0; k < kU; ++k) {
            const int tk = t + k * kCtlThreads;
            const bool in = tk < i1;
            v[k] = in ? ctl_load<T>(xi + tk) : -INFINITY;
            s[k] = in && w.state ? si[tk] : 0;
            if (!in) raw |= 1u << k;
          }
          if (b1 > b0) {
#pragma unroll
            for (int k = 0; k < kU; ++k)
              if (t + k * kCtlThreads < i1) raw |= (listed_bits(t + k * kCtlThreads) & 1) << k;
          }
          if (w.mask) {
            on = 0;
#pragma unroll
            for (int k = 0; k < kU; ++k)
              if (t + k * kCtlThreads < i1) on |= (mask_bits(t + k * kCtlThreads) & 1) << k;
          }
          if (s[0] | s[1] | s[2] | s[3]) {
#pragma unroll
            for (int k = 0; k < kU; ++k)
              if (__builtin_expect(s[k] != 0, 0) && !(raw >> k & 1)) v[k] = penalised(v[k], s[k], w);
          }
          lead(v, on, raw, bar, best, [&](int k) { return t + k * kCtlThreads; });
          if (y) {
#pragma unroll
            for (int k = 0; k < kU; ++k)
              if (t + k * kCtlThreads < i1) ctl_store<T>(y + t + k * kCtlThreads, v[k]);
          }
        }
        if (i1 + tid < t1) one(i1 + tid);
      }
      __syncwarp();
      bar = fmaxf(bar, warp_max(best.v));
      if ((tid & 31) == 0) mbar_arrive(smem_u32(&empty[i % kCtlStages]));  // the warp has read the stage
    }
    if (b1 > b0) {
      if (y) sync();  // y's listed tokens are written last
      // (where y is x its marked tokens still hold the logits)
      const int n = b1 - b0;
      for (int e = b0 + tid; e < b1; e += kCtlThreads) {
        const bool kept = e < b0 + kCtlThreads;
        const int t = kept ? et : __ldg(c.bias_tokens + e);
        if (t < s0 || t >= s1) continue;
        float sum = kept ? ev : __ldg(c.bias_values + e);
        if (twice[(t - s0) >> 5] >> (t & 31) & 1) {
          if (n > kCtlThreads) continue;  // (below)
          // its first entry's thread adds up the token's biases (no early end: the
          // loads of eight steps are under way together)
          bool first = true;
          const int me = e - b0;
#pragma unroll 8
          for (int f = 0; f < me; ++f) first &= list_t[f] != t;
          if (!first) continue;
#pragma unroll 8
          for (int f = me + 1; f < n; ++f) {
            const float more = __fadd_rn(sum, list_v[f]);
            sum = list_t[f] == t ? more : sum;
          }
        }
        if (!kept) {
          ex = ctl_load<T>(x + t);
          es = w.state ? w.state[t] : 0;
          em = w.mask ? __ldg(w.mask + (t >> 5)) >> (t & 31) & 1 : 1;
        }
        const float v = em ? __fadd_rn(es ? penalised(ex, es, w) : ex, sum) : -INFINITY;
        best.take(v, t);
        if (y) ctl_store<T>(y + t, v);
      }
      if (n > kCtlThreads) {
        const Best b = finish_repeated<T>(x, y, c.bias_tokens, c.bias_values, b0, b1, s0, s1, twice, list_t, list_v, w);
        best.take(b.v, b.i);
      }
    }
  }
  if (!a.picks) return;  // (every CTA of the cluster alike)
  if (!alive) best.v = INFINITY, best.i = -1;  // a row that was not read whole has no pick
  best.warp();
  if (tid < kCtlThreads && (tid & 31) == 0) {
    best_v[tid >> 5] = best.v;
    best_i[tid >> 5] = best.i;
  }
  __syncthreads();
  if (tid < 32) {
    best = Best();
    if (tid < kCtlThreads / 32) best.take(best_v[tid], best_i[tid]);
    best.warp();
    if (tid == 0) cta_best = best;
  }
  __syncwarp();
  cluster_sync();
  if (rank == 0 && tid < 32) {
    if (tid > 0 && tid < (int)gridDim.x) {
      const uint32_t at = cluster_addr(smem_u32(&cta_best), (uint32_t)tid);
      float v;
      int i;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at + (uint32_t)offsetof(Best, v)) : "memory");
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(i) : "r"(at + (uint32_t)offsetof(Best, i)) : "memory");
      best.take(v, i);
    }
    best.warp();
    if (tid == 0) {
      const bool any = best.i != 0x7fffffff;
      a.picks[r] = any ? best.i : -1;
      // (every CTA of the row has read its state)
      if (any && best.i >= 0 && c.count_picks && slot >= 0) state_count(c.state + (int64_t)slot * c.state_ld + best.i, false);
    }
  }
  __syncwarp();
  cluster_sync();  // rank 0 has read the others' shared memory
}

template <typename T>
int launch_control_t(const CtlArgs& a, int rows, int ctas, bool vec, cudaStream_t s) {
  auto fn = vec ? logits_control_kernel<T, true> : logits_control_kernel<T, false>;
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[2];
  lc.gridDim = dim3((unsigned)ctas, (unsigned)rows);
  lc.blockDim = dim3(kCtlThreads + 32);
  lc.dynamicSmemBytes = kCtlStages * (kCtlTile * sizeof(T) + kCtlTile * 2 + kCtlTile / 8);
  SAR_TRY(ensure_smem_attr(reinterpret_cast<const void*>(fn), (int)lc.dynamicSmemBytes, "logits control: set smem attribute"));
  lc.stream = s;
  lc.attrs = attr;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  lc.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&lc, fn, a);
  if (e != cudaSuccess) return cuda_error(e, "logits control launch");
  count_launches(1);
  return SAR_OK;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

// The controls' pointers and sizes, before anything is launched.
int check_controls(const sar_logit_controls* c, int vocab) {
  const bool penal = c->repetition || c->presence || c->frequency;
  if ((penal || c->count_picks) && !c->state)
    return set_error(SAR_ERR_INVALID_ARG, "logits control: penalties and counted picks need the token state");
  if (c->state && (!c->slots || c->n_slots < 1 || c->state_ld < vocab))
    return set_error(SAR_ERR_INVALID_ARG, "logits control: token state without slots, or narrower than the vocabulary");
  if (c->state && !aligned(c->state, 2)) return set_error(SAR_ERR_INVALID_ARG, "logits control: token state not aligned");
  const int lists = (c->bias_offsets != nullptr) + (c->bias_tokens != nullptr) + (c->bias_values != nullptr);
  if ((lists != 0 && lists != 3) || c->n_biases < 0)
    return set_error(SAR_ERR_INVALID_ARG, "logits control: biases need offsets, tokens and values");
  // (the kernel's steps past a list's end stay within 32 bits)
  if (c->n_biases > 1 << 30) return set_error(SAR_ERR_UNSUPPORTED, "logits control: more than 2^30 biases");
  if (c->mask && (c->n_masks < 1 || c->mask_ld < ((int64_t)vocab + 31) / 32))
    return set_error(SAR_ERR_INVALID_ARG, "logits control: mask rows shorter than the vocabulary");
  if (!c->mask && c->mask_rows) return set_error(SAR_ERR_INVALID_ARG, "logits control: mask rows without a mask");
  const void* words[] = {c->slots, c->repetition, c->presence, c->frequency, c->bias_offsets,
                         c->bias_tokens, c->bias_values, c->mask, c->mask_rows};
  for (const void* p : words)
    if (!aligned(p, 4)) return set_error(SAR_ERR_INVALID_ARG, "logits control: array not aligned to its element");
  return SAR_OK;
}

int launch_control(const void* x, int64_t ldx, int rows, int vocab, int type, const sar_logit_controls& c, void* y,
                   int64_t ldy, int32_t* picks, cudaStream_t s) {
  CtlArgs a = {};
  a.x = x;
  a.ldx = ldx;
  a.y = y;
  a.ldy = ldy;
  a.picks = picks;
  a.vocab = vocab;
  a.c = c;
  SAR_TRY(op_flags(&a.err));
  const int64_t size = type == SAR_TYPE_F32 ? 4 : 2;
  const bool vec = aligned(x, 16) && ldx * size % 16 == 0 && aligned(y, 16) && (!y || ldy * size % 16 == 0) &&
                   (!c.state || (aligned(c.state, 16) && c.state_ld % 8 == 0));
  // CTAs to a row: as many as stay resident at once (two to an SM), at least 4096
  // tokens each.  Beyond one wave every further CTA costs its start: 256
  // rows of 64000 with two to a row took longer than with one (see the kernel)
  int ctas = 1;
  while (ctas < 8 && 2l * rows * ctas <= kCtlPerSm * num_sms() && vocab > ctas * kCtlLeast) ctas *= 2;
  a.chunk = (int)((((int64_t)vocab + ctas - 1) / ctas + kCtlLeast - 1) / kCtlLeast * kCtlLeast);
  // (65535 rows to a launch)
  for (int r0 = 0; r0 < rows; r0 += 65535) {
    const int n = std::min(rows - r0, 65535);
    CtlArgs b = a;
    b.x = static_cast<const char*>(x) + (int64_t)r0 * ldx * size;
    if (y) b.y = static_cast<char*>(y) + (int64_t)r0 * ldy * size;
    if (picks) b.picks = picks + r0;
    if (c.slots) b.c.slots = c.slots + r0;
    if (c.repetition) b.c.repetition = c.repetition + r0;
    if (c.presence) b.c.presence = c.presence + r0;
    if (c.frequency) b.c.frequency = c.frequency + r0;
    if (c.bias_offsets) b.c.bias_offsets = c.bias_offsets + r0;
    if (c.mask_rows)
      b.c.mask_rows = c.mask_rows + r0;
    else if (c.mask)
      b.c.mask = c.mask + (int64_t)r0 * c.mask_ld, b.c.n_masks = c.n_masks - r0;
    int rc;
    if (type == SAR_TYPE_F32)
      rc = launch_control_t<float>(b, n, ctas, vec, s);
    else if (type == SAR_TYPE_BF16)
      rc = launch_control_t<__nv_bfloat16>(b, n, ctas, vec, s);
    else
      rc = launch_control_t<__half>(b, n, ctas, vec, s);
    if (rc != SAR_OK) return rc;
  }
  return SAR_OK;
}

}  // namespace sar

using sar::set_error;

extern "C" {

int sar_token_state_add(uint16_t* state, int64_t ld, int32_t n_slots, int32_t vocab, const int32_t* slots, int32_t n,
                        const int32_t* offsets, const int32_t* tokens, int32_t n_tokens, const int32_t* prompt_lens,
                        int32_t reset, void* stream) try {
  if (n_slots < 1 || vocab < 1 || ld < vocab || n < 0 || n_tokens < 0)
    return set_error(SAR_ERR_INVALID_ARG, "token_state_add: bad shape");
  if (n == 0 || (n_tokens == 0 && !reset)) return SAR_OK;
  if (!state || !slots || !offsets || (!tokens && n_tokens > 0))
    return set_error(SAR_ERR_INVALID_ARG, "token_state_add: null pointer");
  if (!sar::aligned(state, 2) || !sar::aligned(slots, 4) || !sar::aligned(offsets, 4) || !sar::aligned(tokens, 4) ||
      !sar::aligned(prompt_lens, 4))
    return set_error(SAR_ERR_INVALID_ARG, "token_state_add: array not aligned to its element");
  if (n > 65535) return set_error(SAR_ERR_UNSUPPORTED, "token_state_add: more than 65535 rows");
  // (the kernels' steps past a list's end stay within 32 bits)
  if (vocab > 1 << 30 || n_tokens > 1 << 30)
    return set_error(SAR_ERR_UNSUPPORTED, "token_state_add: vocabulary or tokens above 2^30");
  sar::StateArgs a = {state, ld, n_slots, vocab, slots, n, offsets, tokens, n_tokens, prompt_lens, 0, nullptr};
  a.vec = sar::aligned(state, 16) && ld % 8 == 0;
  SAR_TRY(sar::op_flags(&a.err));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (reset)
    e = sar::launch_pdl(sar::state_reset_kernel, dim3((unsigned)((vocab + (int64_t)sar::kStateSpan - 1) / sar::kStateSpan), (unsigned)n),
                        dim3(sar::kStateThreads), 0, s, a);
  else
    e = sar::launch_pdl(sar::state_append_kernel, dim3((unsigned)((std::max(n_tokens, n) + 255ll) / 256)), dim3(256), 0, s, a);
  if (e != cudaSuccess) return sar::cuda_error(e, "token state launch");
  sar::count_launches(1);
  return SAR_OK;
} catch (...) {
  return sar::entry_failed("token_state_add");
}

int sar_logits_control(const void* logits, int64_t ld, int32_t rows, int32_t vocab, int32_t type,
                       const sar_logit_controls* controls, void* out, int64_t ld_out, int32_t* tokens_out, void* stream) try {
  if (!controls || rows < 0 || vocab < 1 || ld < vocab || (out && ld_out < vocab))
    return set_error(SAR_ERR_INVALID_ARG, "logits control: bad shape");
  if (type != SAR_TYPE_F16 && type != SAR_TYPE_BF16 && type != SAR_TYPE_F32)
    return set_error(SAR_ERR_INVALID_ARG, "logits control: bad element type");
  if (rows == 0) return SAR_OK;  // (its slots and picks may be arrays without an address)
  if (!out && !tokens_out) return set_error(SAR_ERR_INVALID_ARG, "logits control: nothing to write");
  if (controls->count_picks && !tokens_out)
    return set_error(SAR_ERR_INVALID_ARG, "logits control: counted picks without picks");
  if (vocab > (1 << 30) || rows > (1 << 30))
    return set_error(SAR_ERR_UNSUPPORTED, "logits control: vocabulary or rows above 2^30");
  SAR_TRY(sar::check_controls(controls, vocab));
  if (!logits) return set_error(SAR_ERR_INVALID_ARG, "logits control: null logits");
  const uintptr_t size = type == SAR_TYPE_F32 ? 4 : 2;
  if (!sar::aligned(logits, size) || !sar::aligned(out, size) || !sar::aligned(tokens_out, 4))
    return set_error(SAR_ERR_INVALID_ARG, "logits control: buffer not aligned to its element");
  return sar::launch_control(logits, ld, rows, vocab, type, *controls, out, ld_out, tokens_out,
                             static_cast<cudaStream_t>(stream));
} catch (...) {
  return sar::entry_failed("logits_control");
}

}  // extern "C"
