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
// (from L2 after the first).  Shared-memory atomics on whole numbers: the result
// does not depend on their order.
__global__ void __launch_bounds__(kStateThreads) state_reset_kernel(const StateArgs a) {
  __shared__ uint32_t cnt[kStateSpan];
  __shared__ int again;
  pdl_wait();
  pdl_launch_dependents();
  const int r = blockIdx.y, lo = blockIdx.x * kStateSpan, hi = min(a.vocab, lo + kStateSpan);
  const int slot = a.slots[r];
  const bool first_cta = blockIdx.x == 0;
  if (threadIdx.x == 0) again = 0;
  for (int i = threadIdx.x; i < kStateSpan; i += kStateThreads) cnt[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < r; i += kStateThreads)
    if (a.slots[i] == slot) again = 1;
  __syncthreads();
  if (slot < 0 || slot >= a.n_slots || again) {
    if (first_cta && threadIdx.x == 0) report(a.err, SAR_ERR_BOUNDS, SITE_STATE_SLOT, r);
    return;
  }
  const int b = a.offsets[r], e = a.offsets[r + 1];
  if (b < 0 || e < b || e > a.n_tokens) {
    if (first_cta && threadIdx.x == 0) report(a.err, SAR_ERR_BOUNDS, SITE_STATE_OFFSET, r);
    return;
  }
  const int made = b + (a.prompt_lens ? max(0, a.prompt_lens[r]) : 0);  // (past e: a prompt only)
  for (int i = b + (int)threadIdx.x; i < e; i += kStateThreads) {
    const int t = __ldg(a.tokens + i);
    if (t >= lo && t < hi) {
      if (i < made || made < b)
        atomicOr(&cnt[t - lo], 0x80000000u);
      else
        atomicAdd(&cnt[t - lo], 1u);
    } else if (first_cta && (t < 0 || t >= a.vocab)) {
      report(a.err, SAR_ERR_BOUNDS, SITE_STATE_TOKEN, i);
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

// An appending call: one thread per token, its row found by bisection.
__global__ void __launch_bounds__(256) state_append_kernel(const StateArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= a.n_tokens) return;
  int lo = 0, hi = a.n;  // the last row that begins at or before i
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.offsets[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  const int b = a.offsets[lo];
  if (i < b || i >= a.offsets[lo + 1]) return;  // a token of no row
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

constexpr int kCtlThreads = 512;
constexpr int kCtlSpan = 32768;              // tokens per pass: two bitmaps of 4 KB
constexpr int kCtlTile = 8 * kCtlThreads;    // tokens per CTA and step

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
};

// The penalties, in the order and with the roundings the header gives (no fused
// multiply-add: f * count is rounded before it is taken off).
__device__ __forceinline__ float penalised(float x, uint32_t s, const RowCtl& w) {
  if (s == 0) return x;
  const uint32_t made = s & 0x7fffu;
  x = x > 0.f ? __fdiv_rn(x, w.rep) : __fmul_rn(x, w.rep);
  x = __fsub_rn(x, __fmul_rn(w.freq, (float)made));
  return made ? __fsub_rn(x, w.pres) : x;
}

// The larger logit, then the lower token; NaN and -inf never come here.
struct Best {
  float v = -INFINITY;
  int i = 0x7fffffff;
  __device__ __forceinline__ void take(float x, int t) {
    if (x > v || (x == v && t < i && x > -INFINITY)) {
      v = x;
      i = t;
    }
  }
};

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

// One pass over the logits: a cluster of CTAs shares each row, every CTA takes
// one stretch of the vocabulary and the stretches' best tokens meet through
// distributed shared memory, so that a lone row is read by as many SMs as the
// cluster has CTAs, and one launch without a workspace does penalties, biases,
// mask, store and pick.
//
// Biases come as a list per row.  Their tokens are marked in a bitmap of the
// stretch; the dense pass leaves marked tokens as they are, and the list's
// threads then finish one each: penalties from the original logit, the token's
// biases added up in list order (a second bitmap marks tokens that are listed
// again: only those search the list), mask.
//
// VEC: a thread takes 8 neighbouring tokens with 16-byte accesses; otherwise
// (rows at odd addresses) 8 tokens kCtlThreads apart, a warp's still adjacent.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kCtlThreads) logits_control_kernel(const CtlArgs a) {
  __shared__ uint32_t listed[kCtlSpan / 32], twice[kCtlSpan / 32];
  __shared__ float best_v[kCtlThreads / 32];
  __shared__ int best_i[kCtlThreads / 32];
  __shared__ Best cta_best;
  pdl_wait();
  pdl_launch_dependents();
  const int r = blockIdx.y, rank = blockIdx.x, tid = threadIdx.x;
  const bool tells = rank == 0 && tid == 0;
  const sar_logit_controls& c = a.c;
  RowCtl w;
  int slot = -1;
  if (c.state) {
    slot = c.slots[r];
    if (slot >= c.n_slots || slot < -1) {
      if (tells) report(a.err, SAR_ERR_BOUNDS, SITE_CONTROL_SLOT, r);
      slot = -1;
    }
    if (slot >= 0 && (c.repetition || c.presence || c.frequency)) {
      w.state = c.state + (int64_t)slot * c.state_ld;
      if (c.repetition) w.rep = c.repetition[r];
      if (c.presence) w.pres = c.presence[r];
      if (c.frequency) w.freq = c.frequency[r];
    }
  }
  if (c.mask) {
    const int m = c.mask_rows ? c.mask_rows[r] : r;
    if (m >= c.n_masks || m < -1) {
      if (tells) report(a.err, SAR_ERR_BOUNDS, SITE_CONTROL_MASK, r);
    } else if (m >= 0) {
      w.mask = c.mask + (int64_t)m * c.mask_ld;
    }
  }
  int b0 = 0, b1 = 0;
  if (c.bias_offsets) {
    b0 = c.bias_offsets[r];
    b1 = c.bias_offsets[r + 1];
    if (b0 < 0 || b1 < b0 || b1 > c.n_biases) {
      if (tells) report(a.err, SAR_ERR_BOUNDS, SITE_CONTROL_BIAS, r);
      b0 = b1 = 0;
    }
  }
  const T* x = static_cast<const T*>(a.x) + (int64_t)r * a.ldx;
  T* y = a.y ? static_cast<T*>(a.y) + (int64_t)r * a.ldy : nullptr;
  const int lo = rank * a.chunk, hi = min(a.vocab, lo + a.chunk);
  Best best;
  for (int s0 = lo; s0 < hi; s0 += kCtlSpan) {
    const int s1 = min(hi, s0 + kCtlSpan);
    if (b1 > b0) {
      __syncthreads();  // the last span's bitmaps are done with
      for (int i = tid; i < kCtlSpan / 32; i += kCtlThreads) listed[i] = twice[i] = 0;
      __syncthreads();
      for (int e = b0 + tid; e < b1; e += kCtlThreads) {
        const int t = __ldg(c.bias_tokens + e);
        if (t >= s0 && t < s1) {
          const uint32_t bit = 1u << (t & 31);
          if (atomicOr(&listed[(t - s0) >> 5], bit) & bit) atomicOr(&twice[(t - s0) >> 5], bit);
        } else if (rank == 0 && s0 == lo && (t < 0 || t >= a.vocab)) {
          report(a.err, SAR_ERR_BOUNDS, SITE_CONTROL_BIAS, e);
        }
      }
      __syncthreads();
    }
    // (s0 and every tile start are multiples of 32)
    for (int t0 = s0; t0 < s1; t0 += kCtlTile) {
      auto token = [&](int k) { return VEC ? t0 + tid * 8 + k : t0 + k * kCtlThreads + tid; };
      float v[8];
      uint32_t s[8];
      uint32_t on = 0, raw = 0;  // bit k: allowed; left to the list
      const bool full = VEC && token(7) < s1;
      if (full) {
        const int t = token(0);
        if constexpr (sizeof(T) == 4) {
          const float4 p = __ldcs(reinterpret_cast<const float4*>(x + t)), q = __ldcs(reinterpret_cast<const float4*>(x + t) + 1);
          v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w, v[4] = q.x, v[5] = q.y, v[6] = q.z, v[7] = q.w;
        } else {
          const uint4 p = __ldcs(reinterpret_cast<const uint4*>(x + t));
          const uint32_t u[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[2 * k] = Elem<T>::lo(u[k]);
            v[2 * k + 1] = Elem<T>::hi(u[k]);
          }
        }
        if (w.state) {
          const uint4 p = *reinterpret_cast<const uint4*>(w.state + t);
          const uint32_t u[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            s[2 * k] = u[k] & 0xffffu;
            s[2 * k + 1] = u[k] >> 16;
          }
        }
        on = w.mask ? __ldg(w.mask + (t >> 5)) >> (t & 31) & 0xffu : 0xffu;
        if (b1 > b0) raw = listed[(t - s0) >> 5] >> (t & 31) & 0xffu;
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int t = token(k);
          if (t < s1) {
            v[k] = ctl_load<T>(x + t);
            if (w.state) s[k] = w.state[t];
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int t = token(k);
          if (t < s1) {
            on |= (w.mask ? __ldg(w.mask + (t >> 5)) >> (t & 31) & 1u : 1u) << k;
            if (b1 > b0) raw |= (listed[(t - s0) >> 5] >> (t & 31) & 1u) << k;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (raw >> k & 1) continue;
        if (w.state && (full || token(k) < s1)) v[k] = penalised(v[k], s[k], w);
        if (!(on >> k & 1)) v[k] = -INFINITY;
        if (full || token(k) < s1) best.take(v[k], token(k));
      }
      if (y) {
        if (full) {
          T* d = y + token(0);
          if constexpr (sizeof(T) == 4) {
            __stcs(reinterpret_cast<float4*>(d), make_float4(v[0], v[1], v[2], v[3]));
            __stcs(reinterpret_cast<float4*>(d) + 1, make_float4(v[4], v[5], v[6], v[7]));
          } else {
            __stcs(reinterpret_cast<uint4*>(d), make_uint4(Elem<T>::pack(v[0], v[1]), Elem<T>::pack(v[2], v[3]),
                                                           Elem<T>::pack(v[4], v[5]), Elem<T>::pack(v[6], v[7])));
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (token(k) < s1) ctl_store<T>(y + token(k), v[k]);
        }
      }
    }
    if (b1 > b0) {
      __syncthreads();  // y's marked tokens hold the logits (y may be x)
      for (int e = b0 + tid; e < b1; e += kCtlThreads) {
        const int t = __ldg(c.bias_tokens + e);
        if (t < s0 || t >= s1) continue;
        float sum = __ldg(c.bias_values + e);
        if (twice[(t - s0) >> 5] >> (t & 31) & 1) {
          bool first = true;
          for (int f = b0; f < e; ++f) first = first && __ldg(c.bias_tokens + f) != t;
          if (!first) continue;  // its first entry's thread adds it
          for (int f = e + 1; f < b1; ++f)
            if (__ldg(c.bias_tokens + f) == t) sum = __fadd_rn(sum, __ldg(c.bias_values + f));
        }
        float v = ctl_load<T>(x + t);
        if (w.state) v = penalised(v, w.state[t], w);
        v = __fadd_rn(v, sum);
        if (w.mask && !(__ldg(w.mask + (t >> 5)) >> (t & 31) & 1)) v = -INFINITY;
        best.take(v, t);
        if (y) ctl_store<T>(y + t, v);
      }
    }
  }
  if (!a.picks) return;  // (every CTA of the cluster alike)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float v = __shfl_xor_sync(0xffffffffu, best.v, o);
    const int i = __shfl_xor_sync(0xffffffffu, best.i, o);
    best.take(v, i);
  }
  if ((tid & 31) == 0) {
    best_v[tid >> 5] = best.v;
    best_i[tid >> 5] = best.i;
  }
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kCtlThreads / 32; ++i) best.take(best_v[i], best_i[i]);
    cta_best = best;
  }
  __syncwarp();
  cluster_sync();
  if (tells) {
    for (int k = 1; k < (int)gridDim.x; ++k) {
      const uint32_t at = cluster_addr(smem_u32(&cta_best), (uint32_t)k);
      float v;
      int i;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at + (uint32_t)offsetof(Best, v)) : "memory");
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(i) : "r"(at + (uint32_t)offsetof(Best, i)) : "memory");
      best.take(v, i);
    }
    const bool any = best.i != 0x7fffffff;
    a.picks[r] = any ? best.i : -1;
    // (every CTA of the row has read its state)
    if (any && c.count_picks && slot >= 0) state_count(c.state + (int64_t)slot * c.state_ld + best.i, false);
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
  lc.blockDim = dim3(kCtlThreads);
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
  // CTAs to a row: enough to fill the SMs twice, at least one tile of tokens each
  int ctas = 1;
  while (ctas < 8 && (long)rows * ctas < 2l * num_sms() && vocab > ctas * kCtlTile) ctas *= 2;
  a.chunk = (int)((((int64_t)vocab + ctas - 1) / ctas + kCtlTile - 1) / kCtlTile * kCtlTile);
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
                        int32_t reset, void* stream) {
  if (n_slots < 1 || vocab < 1 || ld < vocab || n < 0 || n_tokens < 0)
    return set_error(SAR_ERR_INVALID_ARG, "token_state_add: bad shape");
  if (n == 0 || (n_tokens == 0 && !reset)) return SAR_OK;
  if (!state || !slots || !offsets || (!tokens && n_tokens > 0))
    return set_error(SAR_ERR_INVALID_ARG, "token_state_add: null pointer");
  if (!sar::aligned(state, 2) || !sar::aligned(slots, 4) || !sar::aligned(offsets, 4) || !sar::aligned(tokens, 4) ||
      !sar::aligned(prompt_lens, 4))
    return set_error(SAR_ERR_INVALID_ARG, "token_state_add: array not aligned to its element");
  if (n > 65535) return set_error(SAR_ERR_UNSUPPORTED, "token_state_add: more than 65535 rows");
  sar::StateArgs a = {state, ld, n_slots, vocab, slots, n, offsets, tokens, n_tokens, prompt_lens, 0, nullptr};
  a.vec = sar::aligned(state, 16) && ld % 8 == 0;
  SAR_TRY(sar::op_flags(&a.err));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (reset)
    e = sar::launch_pdl(sar::state_reset_kernel, dim3((unsigned)((vocab + (int64_t)sar::kStateSpan - 1) / sar::kStateSpan), (unsigned)n),
                        dim3(sar::kStateThreads), 0, s, a);
  else
    e = sar::launch_pdl(sar::state_append_kernel, dim3((unsigned)((n_tokens + 255ll) / 256)), dim3(256), 0, s, a);
  if (e != cudaSuccess) return sar::cuda_error(e, "token state launch");
  sar::count_launches(1);
  return SAR_OK;
}

int sar_logits_control(const void* logits, int64_t ld, int32_t rows, int32_t vocab, int32_t type,
                       const sar_logit_controls* controls, void* out, int64_t ld_out, int32_t* tokens_out, void* stream) {
  if (!controls || rows < 0 || vocab < 1 || ld < vocab || (out && ld_out < vocab))
    return set_error(SAR_ERR_INVALID_ARG, "logits control: bad shape");
  if (type != SAR_TYPE_F16 && type != SAR_TYPE_BF16 && type != SAR_TYPE_F32)
    return set_error(SAR_ERR_INVALID_ARG, "logits control: bad element type");
  if (!out && !tokens_out) return set_error(SAR_ERR_INVALID_ARG, "logits control: nothing to write");
  if (controls->count_picks && !tokens_out)
    return set_error(SAR_ERR_INVALID_ARG, "logits control: counted picks without picks");
  if (vocab > (1 << 30)) return set_error(SAR_ERR_UNSUPPORTED, "logits control: vocabulary above 2^30");
  SAR_TRY(sar::check_controls(controls, vocab));
  if (rows == 0) return SAR_OK;
  if (!logits) return set_error(SAR_ERR_INVALID_ARG, "logits control: null logits");
  const uintptr_t size = type == SAR_TYPE_F32 ? 4 : 2;
  if (!sar::aligned(logits, size) || !sar::aligned(out, size) || !sar::aligned(tokens_out, 4))
    return set_error(SAR_ERR_INVALID_ARG, "logits control: buffer not aligned to its element");
  return sar::launch_control(logits, ld, rows, vocab, type, *controls, out, ld_out, tokens_out,
                             static_cast<cudaStream_t>(stream));
}

}  // extern "C"
