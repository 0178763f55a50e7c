// Block tables, slot map and free-page ring of a paged KV cache, from request lengths.
//
// For every request s with n_s = max(add_s, 0) new tokens, h_s = ceil(len_s / ps) pages held and
// g_s = ceil((len_s + n_s) / ps) - h_s pages wanted:
//   cu_new = exclusive scan of n, off = exclusive scan of g,
//   table[s][h_s + j] = ring[(head + off_s + j) mod P],            j < g_s
//   slot[cu_new_s + j] = table[s][(len_s + j) / ps] * ps + (len_s + j) mod ps,
// and the pages of a request that ends (add_s < 0) go behind the ring's last free page.  The ring
// is a queue: what a call takes (front) and what it gives back (behind the end) do not overlap where
// the free pages and those held are no more than the pool, and a call for which they are more is
// refused: some page is then listed twice.  So nothing has to be ordered between the two and the
// results do not depend on timing.
//
// Latency bound: a few bytes per request.  Every CTA of a cluster scans all requests (in chunks of its
// size; several chunks take a first pass for the totals, which decide whether the call changes
// anything); the pages and tokens are then spread over the cluster's threads, each of which finds its
// request by bisection in the scanned offsets in shared memory.  Lengths and the ring's state may be
// updated in place, so they are written behind a barrier of the cluster.  4.2 us for one token of 64
// requests, 10.0 us for 128K tokens of 16 prompts in pages of 16, 8.1 us for 20011 tokens of 1000 requests
// (0.1 to 0.2 of it to count the pages held).
#include "moba.h"
#include "cache.cuh"
#include "sm100.cuh"

namespace moba {
namespace {

constexpr int kTabThreads = 1024;

struct Growth {
  int32_t len, have;  // cached tokens, pages held
  int32_t len_out;    // tokens after the call
  int32_t n;          // new tokens
  int32_t need;       // pages to take
  int32_t back;       // pages to give back
  int bad;            // status bits
};

__device__ __forceinline__ Growth growth_of(const CacheGeom& g, int lps, const int32_t* add, const int32_t* lens, int s) {
  Growth r{0, 0, 0, 0, 0, 0, 0};
  if (s >= g.B) return r;
  const int32_t len = lens[s], a = add[s];
  r.len = r.len_out = len;
  if ((uint32_t)len > (uint32_t)g.max_len) {
    r.bad = kTabState;
    return r;
  }
  r.have = (len + g.ps - 1) >> lps;
  if (a < 0) {
    r.back = r.have;
    r.len_out = 0;
  } else if (a > g.max_len - len) {
    r.bad = kTabTooLong;
  } else {
    r.n = a;
    r.need = ((len + a + g.ps - 1) >> lps) - r.have;
    r.len_out = len + a;
  }
  return r;
}

struct Triple {
  long long n;
  int32_t need, back;
};

__device__ __forceinline__ Triple add3(const Triple& a, const Triple& b) {
  return {a.n + b.n, a.need + b.need, a.back + b.back};
}

__device__ __forceinline__ Triple shfl_up3(const Triple& x, int off) {
  return {__shfl_up_sync(0xffffffffu, x.n, off), __shfl_up_sync(0xffffffffu, x.need, off),
          __shfl_up_sync(0xffffffffu, x.back, off)};
}
__device__ __forceinline__ Triple warp_scan(Triple x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const Triple o = shfl_up3(x, off);
    if (lane >= off) x = add3(x, o);
  }
  return x;
}

// Exclusive scan over the block; *total gets the sum.
__device__ __forceinline__ Triple block_scan(Triple x, Triple* warp_sums, Triple* total) {
  static_assert(kTabThreads == 1024, "one warp scans the warps' sums");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Triple inc = warp_scan(x);
  __syncthreads();  // warp_sums of an earlier scan is read
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) warp_sums[lane] = warp_scan(warp_sums[lane]);
  __syncthreads();
  const Triple before = warp > 0 ? warp_sums[warp - 1] : Triple{0, 0, 0};
  *total = warp_sums[kTabThreads / 32 - 1];
  return {before.n + inc.n - x.n, before.need + inc.need - x.need, before.back + inc.back - x.back};
}

// Last index j < n with off[j] <= x (off is nondecreasing, off[0] <= x).
__device__ __forceinline__ int owner_of(const int32_t* off, int n, int32_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kTabThreads)
    cache_tables_kernel(CacheGeom g, const int32_t* add, const int32_t* lens, int32_t* tables, int32_t* free_pages,
                        const int32_t* free_state, int32_t* lens_out, int32_t* free_state_out, int32_t* cu_new,
                        int32_t* slots, int32_t max_tokens, int32_t* status) {
  __shared__ Triple warp_sums[kTabThreads / 32];
  __shared__ int32_t s_tok[kTabThreads], s_need[kTabThreads], s_back[kTabThreads];  // chunk offsets
  __shared__ int32_t s_len[kTabThreads], s_held[kTabThreads / 32];
  const int tid = threadIdx.x, rank = blockIdx.x, lps = 31 - __clz(g.ps);
  const bool one = g.B <= kTabThreads;  // a single chunk
  const int32_t first = rank * kTabThreads + tid, step = gridDim.x * kTabThreads;  // of pages and tokens
  const int32_t head = free_state[0], count = free_state[1];
  const uint32_t P = (uint32_t)g.P;
  auto ring = [&](uint32_t at) { return at >= P ? at - P : at; };  // at < 2 P <= 2^32
  // ---- totals: they decide whether anything changes
  Triple total{0, 0, 0}, off{0, 0, 0}, t{0, 0, 0};
  Growth r;
  int bad = 0;
  int32_t held = 0;  // pages of all requests: at most the entries of the block tables
  for (int b0 = 0; b0 < g.B; b0 += kTabThreads) {
    r = growth_of(g, lps, add, lens, b0 + tid);
    bad |= r.bad;
    held += r.have;
    off = block_scan({r.n, r.need, r.back}, warp_sums, &t);
    total = add3(total, t);
  }
  held = __reduce_add_sync(0xffffffffu, held);
  if ((tid & 31) == 0) s_held[tid >> 5] = held;
  // the four bits of all threads
  bad = (__syncthreads_or(bad & kTabState) ? kTabState : 0) | (__syncthreads_or(bad & kTabTooLong) ? kTabTooLong : 0);
  held = __reduce_add_sync(0xffffffffu, s_held[tid & 31]);
  if ((uint32_t)head >= P || (uint32_t)count > P) bad |= kTabState;
  else if (total.need > count) bad |= kTabNoPages;
  // more pages than there are: what comes back might overrun the free pages, which are read meanwhile, and a
  // page that two requests hold would come back while one of them still reads it
  else if ((int64_t)count + held > g.P) bad |= kTabState;
  if (total.n > max_tokens) bad |= kTabSlots;
  const bool go = bad == 0;
  // ---- pages and tokens
  Triple base{0, 0, 0};
  for (int b0 = 0; b0 < g.B; b0 += kTabThreads) {
    const int s = b0 + tid, live = min(kTabThreads, g.B - b0);
    if (!one) {
      r = growth_of(g, lps, add, lens, s);
      off = block_scan({r.n, r.need, r.back}, warp_sums, &t);
    }
    if (rank == 0 && s < g.B) cu_new[s] = go ? (int32_t)(base.n + off.n) : 0;
    if (!go) continue;
    s_tok[tid] = (int32_t)off.n;
    s_need[tid] = off.need;
    s_back[tid] = off.back;
    s_len[tid] = r.len;
    __syncthreads();
    // r-th page that the chunk takes; % never: what a call takes or gives is at most the ring
    auto taken = [&](int32_t i) { return free_pages[ring((uint32_t)head + (uint32_t)(base.need + i))]; };
    for (int32_t i = first; i < t.need; i += step) {
      const int j = owner_of(s_need, live, i);
      tables[(int64_t)(b0 + j) * g.MP + ((s_len[j] + g.ps - 1) >> lps) + (i - s_need[j])] = taken(i);
    }
    const uint32_t end = ring((uint32_t)head + (uint32_t)count);
    for (int32_t i = first; i < t.back; i += step) {
      const int j = owner_of(s_back, live, i);
      free_pages[ring(end + (uint32_t)(base.back + i))] = tables[(int64_t)(b0 + j) * g.MP + (i - s_back[j])];
    }
    for (int64_t i = first; i < t.n; i += step) {
      const int j = owner_of(s_tok, live, (int32_t)i);
      const int32_t pos = s_len[j] + ((int32_t)i - s_tok[j]), nth = (pos >> lps) - ((s_len[j] + g.ps - 1) >> lps);
      // a new page is read where the entry above comes from
      const int32_t page = nth < 0 ? tables[(int64_t)(b0 + j) * g.MP + (pos >> lps)] : taken(s_need[j] + nth);
      slots[base.n + i] = page_ok(g, page) ? (page << lps) + (pos & (g.ps - 1)) : -1;
    }
    base = add3(base, t);
  }
  for (int64_t i = base.n + first; i < max_tokens; i += step) slots[i] = -1;
  if (gridDim.x > 1) cluster_barrier(); else __syncthreads();  // lens and free_state are read
  if (rank > 0) return;
  for (int b0 = 0; b0 < g.B; b0 += kTabThreads) {
    if (!one) r = growth_of(g, lps, add, lens, b0 + tid);
    if (b0 + tid < g.B) lens_out[b0 + tid] = go ? r.len_out : r.len;
  }
  if (tid == 0) {
    cu_new[g.B] = (int32_t)base.n;
    *status = bad;
    free_state_out[0] = go ? (int32_t)ring((uint32_t)head + (uint32_t)base.need) : head;
    free_state_out[1] = go ? count - base.need + base.back : count;
  }
}

}  // namespace

cudaError_t launch_cache_tables(const CacheGeom& g, const int32_t* add, const int32_t* lens, int32_t* tables,
                                int32_t* free_pages, const int32_t* free_state, int32_t* lens_out,
                                int32_t* free_state_out, int32_t* cu_new, int32_t* slots, int32_t max_tokens,
                                int32_t* status, cudaStream_t st) {
  // one CTA writes a decode step's slots at once; a prompt's are worth a cluster: 64 requests with 64, 1024,
  // 2048 and 4096 tokens take 4.2, 4.5, 5.3 and 6.7 us with one, 4.5, 4.9, 4.9 and 4.9 with 8
  const unsigned c = max_tokens > kTabThreads ? 8 : 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(c);
  cfg.blockDim = dim3(kTabThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = c;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_tables_kernel, g, add, lens, tables, free_pages, free_state, lens_out,
                            free_state_out, cu_new, slots, max_tokens, status);
}

}  // namespace moba
