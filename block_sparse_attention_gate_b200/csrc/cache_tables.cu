// Block tables, slot map and free-page ring of a paged KV cache, from request lengths.
//
// For every request s with n_s = max(add_s, 0) new tokens, h_s = ceil(len_s / ps) pages held and
// g_s = ceil((len_s + n_s) / ps) - h_s pages wanted:
//   cu_new = exclusive scan of n, off = exclusive scan of g,
//   table[s][h_s + j] = ring[(head + off_s + j) mod P],            j < g_s
//   slot[cu_new_s + j] = table[s][(len_s + j) / ps] * ps + (len_s + j) mod ps,
// and the pages of a request that ends (add_s < 0) go behind the ring's last free page.  The ring
// is a queue: what a call takes (front) and what it gives back (behind the end) never overlap, so
// nothing has to be ordered between the two and the results do not depend on timing.
//
// Latency bound: a few bytes per request.  One CTA scans the requests in chunks of its size (a
// first pass for the totals, which decide whether the call changes anything at all, a second one
// that writes); pages and tokens are then spread over all threads, each of which finds its
// request by bisection in the chunk's scanned offsets in shared memory.
#include "moba.h"
#include "cache.cuh"

namespace moba {
namespace {

constexpr int kTabThreads = 1024;

struct Growth {
  int32_t len, have;  // cached tokens, pages held
  int32_t n;          // new tokens
  int32_t need;       // pages to take
  int32_t back;       // pages to give back
  int bad;            // status bits
};

__device__ __forceinline__ Growth growth_of(const CacheGeom& g, const int32_t* add, const int32_t* lens, int s) {
  Growth r{0, 0, 0, 0, 0, 0};
  if (s >= g.B) return r;
  const int32_t len = lens[s], a = add[s];
  if ((uint32_t)len > (uint32_t)g.max_len) {
    r.bad = kTabState;
    return r;
  }
  r.len = len;
  r.have = (len + g.ps - 1) / g.ps;
  if (a < 0) {
    r.back = r.have;
  } else if (a > g.max_len - len) {
    r.bad = kTabTooLong;
  } else {
    r.n = a;
    r.need = (len + a + g.ps - 1) / g.ps - r.have;
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

// Exclusive scan over the block; *total gets the sum.
__device__ __forceinline__ Triple block_scan(Triple x, Triple* warp_sums, Triple* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Triple inc = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    Triple o;
    o.n = __shfl_up_sync(0xffffffffu, inc.n, off);
    o.need = __shfl_up_sync(0xffffffffu, inc.need, off);
    o.back = __shfl_up_sync(0xffffffffu, inc.back, off);
    if (lane >= off) inc = add3(inc, o);
  }
  __syncthreads();  // warp_sums of an earlier scan is read
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  Triple before{0, 0, 0}, sum{0, 0, 0};
#pragma unroll 8
  for (int w = 0; w < kTabThreads / 32; ++w) {
    if (w == warp) before = sum;
    sum = add3(sum, warp_sums[w]);
  }
  *total = sum;
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
  __shared__ int32_t s_len[kTabThreads];
  __shared__ int s_bad;
  const int tid = threadIdx.x;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  const int32_t head = free_state[0], count = free_state[1];
  // ---- totals: they decide whether anything changes
  Triple total{0, 0, 0};
  int bad = 0;
  for (int b0 = 0; b0 < g.B; b0 += kTabThreads) {
    const Growth r = growth_of(g, add, lens, b0 + tid);
    bad |= r.bad;
    Triple t;
    block_scan({r.n, r.need, r.back}, warp_sums, &t);
    total = add3(total, t);
  }
  if (bad) atomicOr(&s_bad, bad);
  __syncthreads();
  bad = s_bad;
  if ((uint32_t)head >= (uint32_t)g.P || (uint32_t)count > (uint32_t)g.P) bad |= kTabState;
  else if (total.need > count) bad |= kTabNoPages;
  else if ((int64_t)count - total.need + total.back > g.P) bad |= kTabState;
  if (total.n > max_tokens) bad |= kTabSlots;
  const bool go = bad == 0;
  // ---- write
  Triple base{0, 0, 0};
  for (int b0 = 0; b0 < g.B; b0 += kTabThreads) {
    const int s = b0 + tid, live = min(kTabThreads, g.B - b0);
    Growth r = growth_of(g, add, lens, s);
    if (!go) r.n = r.need = r.back = 0;
    Triple t;
    const Triple off = block_scan({r.n, r.need, r.back}, warp_sums, &t);
    s_tok[tid] = (int32_t)off.n;
    s_need[tid] = off.need;
    s_back[tid] = off.back;
    s_len[tid] = r.len;
    if (s < g.B) {
      cu_new[s] = (int32_t)(base.n + off.n);
      lens_out[s] = !go ? lens[s] : add[s] < 0 ? 0 : r.len + r.n;
    }
    __syncthreads();
    for (int32_t i = tid; i < t.need; i += kTabThreads) {
      const int j = owner_of(s_need, live, i);
      const int32_t have = (s_len[j] + g.ps - 1) / g.ps;
      const int32_t page = free_pages[((int64_t)head + base.need + i) % g.P];
      tables[(int64_t)(b0 + j) * g.MP + have + (i - s_need[j])] = page;
    }
    for (int32_t i = tid; i < t.back; i += kTabThreads) {
      const int j = owner_of(s_back, live, i);
      free_pages[((int64_t)head + count + base.back + i) % g.P] = tables[(int64_t)(b0 + j) * g.MP + (i - s_back[j])];
    }
    __syncthreads();  // the new table entries are visible to the whole CTA
    for (int32_t i = tid; i < (int32_t)t.n; i += kTabThreads) {
      const int j = owner_of(s_tok, live, i);
      const int32_t pos = s_len[j] + (i - s_tok[j]);
      const int32_t page = tables[(int64_t)(b0 + j) * g.MP + pos / g.ps];
      slots[base.n + i] = page_ok(g, page) ? page * g.ps + pos % g.ps : -1;
    }
    base = add3(base, t);
  }
  for (int64_t i = base.n + tid; i < max_tokens; i += kTabThreads) slots[i] = -1;
  if (tid == 0) {
    cu_new[g.B] = (int32_t)base.n;
    *status = bad;
    free_state_out[0] = go ? (int32_t)(((int64_t)head + base.need) % g.P) : head;
    free_state_out[1] = go ? count - base.need + base.back : count;
  }
}

}  // namespace

cudaError_t launch_cache_tables(const CacheGeom& g, const int32_t* add, const int32_t* lens, int32_t* tables,
                                int32_t* free_pages, const int32_t* free_state, int32_t* lens_out,
                                int32_t* free_state_out, int32_t* cu_new, int32_t* slots, int32_t max_tokens,
                                int32_t* status, cudaStream_t st) {
  cache_tables_kernel<<<1, kTabThreads, 0, st>>>(g, add, lens, tables, free_pages, free_state, lens_out,
                                                 free_state_out, cu_new, slots, max_tokens, status);
  return cudaGetLastError();
}

}  // namespace moba
