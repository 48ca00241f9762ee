// Block tables and slot maps of a paged KV cache from the requests' lengths.
//
// With held = ceil(len / page) and need = ceil((len + new) / page) - held of each
// request, three prefix sums say everything: rows (whose they are), pages taken and
// pages given back.  The free list is a stack; the t-th page taken is entry
// have - 1 - t of the list with the pages given back behind its end, so every
// table entry, slot and list entry has a closed form, and no thread waits for
// another's page.
//
// One CTA, or a cluster of 8 whose CTAs form the same sums and share out the
// entries: all of it reads a few hundred KB from L2 at most, so the time is a chain
// of latencies (lengths, two block-wide sums, list entry, store): 6.2 us for one request,
// 10.9 for 256 that decode or begin, 12.4 for 64 chunks of up to 2048 rows.  What is read and
// may be written over (lengths, the count) is in shared memory before the cluster
// passes its barrier; the rest is disjoint: entries of the list are read below the
// old count and written from there on, tables are read for pages given back (or
// held) and written behind those held.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "tc05.cuh"

namespace sar {

namespace {

constexpr int kMapThreads = 1024;
constexpr int kMapCtas = 8;     // CTAs of a large call's cluster
constexpr int kMapAlone = 1024; // rows up to which one CTA takes the call
constexpr int kMapMost = 8192;  // requests: four shared-memory words each

struct MapArgs {
  sar_page_map_args m;
  int shift;  // log2 page_size
  int vec;    // positions and slots are 16-byte aligned
  int* err;
};

// Inclusive sums of (a, b) over the block; `warps` is scratch, one pair per warp.
__device__ __forceinline__ void block_scan(int64_t& a, int& b, int64_t (*warps)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, a, o);
    const int y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) a += x, b += y;
  }
  if (lane == 31) warps[warp][0] = a, warps[warp][1] = b;
  __syncthreads();
  if (warp == 0) {
    int64_t x = lane < kMapThreads / 32 ? warps[lane][0] : 0, y = lane < kMapThreads / 32 ? warps[lane][1] : 0;
#pragma unroll
    for (int o = 1; o < kMapThreads / 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) x += u, y += v;
    }
    if (lane < kMapThreads / 32) warps[lane][0] = x, warps[lane][1] = y;
  }
  __syncthreads();
  if (warp > 0) a += warps[warp - 1][0], b += (int)warps[warp - 1][1];
}

// The last i with at[i] <= x, of a non-falling at[0 .. n] with at[0] <= x < at[n].
__device__ __forceinline__ int owner(const int* at, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kMapThreads) page_map_kernel(const MapArgs a) {
  extern __shared__ int sh[];
  __shared__ int64_t warps[kMapThreads / 32][2];
  __shared__ int64_t carry_a;
  __shared__ int carry_b, taken_s;
  const sar_page_map_args& m = a.m;
  const int n = m.n;
  int* row_at = sh;                 // [n + 1], clamped to max_rows
  int* take_at = row_at + n + 1;    // [n + 1]
  int* give_at = take_at + n + 1;   // [n + 1]
  int* len_s = give_at + n + 1;     // [n]: length; ~length where the request gets nothing
  const int ps = m.page_size, shift = a.shift;
  const unsigned rank = blockIdx.x, ctas = gridDim.x;
  pdl_wait();
  pdl_launch_dependents();
  const int f_raw = *m.free_count;
  const int f = min(max(f_raw, 0), m.num_pages);
  const int64_t most = (int64_t)m.bt_cols << shift;  // (not the stride: behind the columns lies what is not ours)
  const bool first_cta = rank == 0;
  if (first_cta && threadIdx.x == 0 && f != f_raw) report(a.err, SAR_ERR_BOUNDS, SITE_MAP_REQUEST, -1);

  // rows and pages given back
  if (threadIdx.x == 0) carry_a = 0, carry_b = 0, taken_s = 0, row_at[0] = take_at[0] = give_at[0] = 0;
  __syncthreads();
  for (int i0 = 0; i0 < n; i0 += kMapThreads) {
    const int i = i0 + threadIdx.x;
    int len = 0, add = 0, give = 0;
    if (i < n) {
      len = m.lens[i];
      add = m.new_lens[i];
      const bool bad = len < 0 || len > most || add < -1 || (int64_t)len + add > most;
      if (bad) {
        if (first_cta) report(a.err, SAR_ERR_BOUNDS, SITE_MAP_REQUEST, i);
        add = 0;
        len = max(len, 0);
      }
      if (add < 0) give = (int)(((int64_t)len + ps - 1) >> shift), add = 0;
      len_s[i] = len;
    }
    int64_t x = add;
    int y = give;
    block_scan(x, y, warps);
    x += carry_a;
    y += carry_b;
    if (i < n) {
      // rows that pass max_rows belong to requests that get nothing: add is kept
      // for the page sums below where they fit
      row_at[i + 1] = (int)min(x, (int64_t)m.max_rows);
      give_at[i + 1] = y;
      take_at[i + 1] = x <= m.max_rows ? add : add > 0 ? -1 : 0;
    }
    __syncthreads();
    if (threadIdx.x == kMapThreads - 1) carry_a = x, carry_b = y;
    __syncthreads();
  }
  // (n * bt_stride <= 2^30 bounds every sum of pages)
  const int have = f + (n > 0 ? give_at[n] : 0);
  if (threadIdx.x == 0) carry_b = 0;
  __syncthreads();
  for (int i0 = 0; i0 < n; i0 += kMapThreads) {
    const int i = i0 + threadIdx.x;
    int take = 0, fits = 1;
    if (i < n) {
      const int add = take_at[i + 1], len = len_s[i];
      fits = add >= 0;
      if (add > 0) take = (int)((((int64_t)len + add + ps - 1) >> shift) - (((int64_t)len + ps - 1) >> shift));
    }
    int64_t none = 0;
    int y = take;
    block_scan(none, y, warps);
    y += carry_b;
    if (i < n) {
      take_at[i + 1] = y;
      const bool pages = take == 0 || y <= have;
      if (!fits || !pages) {
        if (first_cta) {
          if (!fits)
            report(a.err, SAR_ERR_BOUNDS, SITE_MAP_REQUEST, i);
          else
            report(a.err, SAR_ERR_NO_PAGES, SITE_MAP_PAGES, i);
        }
        len_s[i] = ~len_s[i];
      } else if (take > 0) {
        atomicMax(&taken_s, y);
      }
    }
    __syncthreads();
    if (threadIdx.x == kMapThreads - 1) carry_b = y;
    __syncthreads();
  }
  const int taken = taken_s;
  const int left = min(have - taken, m.num_pages);
  if (first_cta && threadIdx.x == 0 && left != have - taken) report(a.err, SAR_ERR_BOUNDS, SITE_MAP_REQUEST, -1);
  if (ctas > 1) cluster_sync();  // every CTA has read what is written over from here on

  const unsigned gt = rank * kMapThreads + threadIdx.x, gn = ctas * kMapThreads;
  // entry x of the free list with the pages given back behind it
  auto listed = [&](int x) -> int {
    if (x < f) return m.free_pages[x];
    const int i = owner(give_at, n, x - f);
    return m.block_tables[(int64_t)i * m.bt_stride + (x - f - give_at[i])];
  };
  auto in_pool = [&](int page) -> bool {
    if (page >= 0 && page < m.num_pages) return true;
    report(a.err, SAR_ERR_BOUNDS, SITE_MAP_PAGE, page);
    return false;
  };
  // Rows of chunks, four to a thread, are mostly one request's, in one page, and then take
  // one search and one look-up (64 chunks of up to 2048 rows: 12.4 us; 18.4 with a row at a
  // time).  Where there is a thread for every row, a row each: single tokens'
  // look-ups do not wait for one another (256 mixed requests: 10.9 us; 18 with four).
  const int live = n > 0 ? row_at[n] : 0;
  const int each = m.max_rows > 2 * (int)gn ? 4 : 1;
  for (int r0 = each * (int)gt; r0 < m.max_rows; r0 += each * (int)gn) {
    int pos[4], slot[4], i = -1, page = -1, of = -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = r0 + k;
      pos[k] = 0;
      slot[k] = -1;
      if (r >= live || k >= each) continue;
      if (i < 0 || r >= row_at[i + 1]) {
        i = owner(row_at, n, r);
        of = -1;
      }
      const bool ok = len_s[i] >= 0;
      const int len = ok ? len_s[i] : ~len_s[i];
      pos[k] = len + (r - row_at[i]);
      if (!ok) continue;
      const int held = (int)(((int64_t)len + ps - 1) >> shift), b = pos[k] >> shift;
      if (b != of) {
        of = b;
        page = b < held ? m.block_tables[(int64_t)i * m.bt_stride + b] : listed(have - 1 - (take_at[i] + b - held));
        if (!in_pool(page)) page = -1;
      }
      if (page >= 0) slot[k] = (page << shift) + (pos[k] & (ps - 1));
    }
    if (a.vec && each == 4 && r0 + 4 <= m.max_rows) {
      *reinterpret_cast<int4*>(m.positions + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<int4*>(m.slots + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < each && r0 + k < m.max_rows) m.positions[r0 + k] = pos[k], m.slots[r0 + k] = slot[k];
    }
  }
  for (int i = (int)gt; i <= n; i += (int)gn) {
    m.row_offsets[i] = row_at[i];
    if (i == n) continue;
    const bool ok = len_s[i] >= 0;
    const int len = ok ? len_s[i] : ~len_s[i];
    // (a request that has ended without pages had no tokens)
    m.lens_out[i] = give_at[i + 1] > give_at[i] ? 0 : ok ? len + (row_at[i + 1] - row_at[i]) : len;
  }
  for (int t = (int)gt; t < taken; t += (int)gn) {
    const int i = owner(take_at, n, t);
    const int held = (int)(((int64_t)len_s[i] + ps - 1) >> shift);
    m.block_tables[(int64_t)i * m.bt_stride + held + (t - take_at[i])] = listed(have - 1 - t);
  }
  for (int x = f + (int)gt; x < left; x += (int)gn) {
    const int page = listed(x);
    in_pool(page);
    m.free_pages[x] = page;
  }
  if (gt == 0) *m.free_count_out = left;
}

bool on4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

}  // namespace
}  // namespace sar

using sar::set_error;

extern "C" int sar_page_map(const sar_page_map_args* args, void* stream) try {
  if (!args) return set_error(SAR_ERR_INVALID_ARG, "page_map: null arguments");
  const sar_page_map_args& m = *args;
  if (m.n < 0 || m.bt_stride < 1 || m.num_pages < 1 || m.max_rows < 0 || m.bt_cols < 0 || m.bt_cols > m.bt_stride)
    return set_error(SAR_ERR_INVALID_ARG, "page_map: bad sizes");
  if (m.page_size != 16 && m.page_size != 32 && m.page_size != 64)
    return set_error(SAR_ERR_UNSUPPORTED, "page_map: pages of 16, 32 or 64 tokens");
  if (m.n > sar::kMapMost) return set_error(SAR_ERR_UNSUPPORTED, "page_map: more than 8192 requests");
  if ((int64_t)m.n * m.bt_stride > 1 << 30 || m.max_rows > 1 << 30 || (int64_t)m.num_pages * m.page_size > INT32_MAX ||
      m.num_pages > 1 << 30 || (int64_t)m.bt_stride * m.page_size > INT32_MAX)
    return set_error(SAR_ERR_UNSUPPORTED, "page_map: tables, rows or slots above their limits");
  const void* need[] = {m.free_pages, m.free_count, m.free_count_out, m.row_offsets};
  for (const void* p : need)
    if (!p) return set_error(SAR_ERR_INVALID_ARG, "page_map: null pointer");
  if (m.n > 0 && (!m.lens || !m.new_lens || !m.lens_out || !m.block_tables))
    return set_error(SAR_ERR_INVALID_ARG, "page_map: null pointer");
  if (m.max_rows > 0 && (!m.positions || !m.slots)) return set_error(SAR_ERR_INVALID_ARG, "page_map: null pointer");
  const void* all[] = {m.lens, m.new_lens, m.lens_out, m.block_tables, m.free_pages, m.free_count, m.free_count_out,
                       m.row_offsets, m.positions, m.slots};
  for (const void* p : all)
    if (!sar::on4(p)) return set_error(SAR_ERR_INVALID_ARG, "page_map: array not aligned to its element");
  sar::MapArgs a = {m, m.page_size == 16 ? 4 : m.page_size == 32 ? 5 : 6, 0, nullptr};
  if (a.m.bt_cols == 0) a.m.bt_cols = m.bt_stride;
  a.vec = ((reinterpret_cast<uintptr_t>(m.positions) | reinterpret_cast<uintptr_t>(m.slots)) & 15) == 0;
  SAR_TRY(sar::op_flags(&a.err));
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[2];
  const unsigned ctas = m.max_rows > sar::kMapAlone ? sar::kMapCtas : 1;
  lc.gridDim = dim3(ctas);
  lc.blockDim = dim3(sar::kMapThreads);
  lc.dynamicSmemBytes = (size_t)(4 * m.n + 3) * 4;
  SAR_TRY(sar::ensure_smem_attr(reinterpret_cast<const void*>(&sar::page_map_kernel), (4 * sar::kMapMost + 3) * 4,
                                "page map: set smem attribute"));
  lc.stream = static_cast<cudaStream_t>(stream);
  lc.attrs = attr;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = sar::pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  lc.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&lc, sar::page_map_kernel, a);
  if (e != cudaSuccess) return sar::cuda_error(e, "page map launch");
  sar::count_launches(1);
  return SAR_OK;
} catch (...) {
  return sar::entry_failed("page_map");
}
