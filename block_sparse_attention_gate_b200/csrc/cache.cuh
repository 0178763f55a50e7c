// Internal definitions of the paged 8-bit KV cache: geometry, launchers, code conversions.
#pragma once

#include <cuda_fp8.h>

#include <atomic>

#include "moba.h"

#include "moba_internal.cuh"

namespace moba {

// Bits that the cache kernels OR into the device error word (bit 0 is the bounded wait).
enum : int { kErrBadPage = 2 };

// Bits of the status word that cache_tables writes.
enum : int { kTabNoPages = 1, kTabTooLong = 2, kTabSlots = 4, kTabState = 8 };

// Geometry of a paged cache as the kernels see it (passed by value).
struct CacheGeom {
  int32_t B;           // request slots
  int32_t max_len;     // longest request
  int32_t MP;          // pages of the longest request: row length of the block tables
  int32_t MB;          // MoBA blocks of the longest request
  int32_t P;           // pages in the pool
  int32_t ps;          // tokens of a page
  int32_t Hq, Hkv, G, D;
  int32_t bs;          // tokens of a MoBA block (a multiple of ps)
  int32_t k;           // blocks a query takes, its own included
  int32_t fmt;         // moba_cache_format
  float scale;         // softmax scale
  float scale_log2;    // softmax scale * log2(e)
  int* err;            // device error word, never null
};

// Bytes of one (page, KV head) slab of codes, and where it starts in the pool.
__device__ __forceinline__ size_t slab_offset(const CacheGeom& g, int32_t page, int head) {
  return ((size_t)page * g.Hkv + head) * ((size_t)g.ps * g.D);
}

__device__ __forceinline__ bool page_ok(const CacheGeom& g, int32_t page) {
  return (uint32_t)page < (uint32_t)g.P;
}

// Cached length of a request; a length outside [0, max_len] counts as 0 (nothing is touched).
__device__ __forceinline__ int32_t cached_len(const CacheGeom& g, const int32_t* lens, int s) {
  const int32_t n = __ldg(lens + s);
  return (uint32_t)n <= (uint32_t)g.max_len ? n : 0;
}

// Two codes (low and high byte of c) as values.
template <int kFmt>
__device__ __forceinline__ float2 codes2_to_float2(uint32_t c) {
  if constexpr (kFmt == MOBA_CACHE_E4M3) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xffffu), __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
  } else {
    return make_float2((float)(int8_t)(c & 0xffu), (float)(int8_t)((c >> 8) & 0xffu));
  }
}

// Two values as codes: nearest, ties to even, clamped to the largest code.
template <int kFmt>
__device__ __forceinline__ uint32_t float2_to_codes2(float a, float b) {
  if constexpr (kFmt == MOBA_CACHE_E4M3) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  } else {
    const int x = min(max(__float2int_rn(a), -127), 127), y = min(max(__float2int_rn(b), -127), 127);
    return (uint32_t)(x & 0xff) | ((uint32_t)(y & 0xff) << 8);
  }
}

// A block that heads of one tile of 8 chose: byte h of slots is head h's slot, 0xff if it did not.
struct __align__(16) CacheSeg {
  int32_t block;
  int32_t keys;        // of the block: bs, or those up to the newest token
  uint32_t slots[2];
};

// Work space of one decode call (device pointers), and how its blocks are cut.  An entry of the work
// list is a (request, KV head, tile of 8 heads), its units are chunks of CK keys.
struct CacheDecodeWork {
  uint64_t* score;   // [B, Hq, MB] gate scores, as ordered keys
  CacheSeg* segs;    // [entries, max_segs] distinct blocks, the own one last
  int32_t* units;    // [entries] chunks in all
  float* part_o;     // [B, Hq, k, NC, D] partial sums of weighted values
  float4* part_ml;   // [B, Hq, k, NC] references r and u (log2 units), sum of the softmax
  int32_t* sel;      // [B, Hq, k] (used when the caller passes none)
  int32_t max_segs, CK, NC;
  size_t bytes;
};

int cache_chunk_keys(const CacheGeom& g);
// Raises a kernel's limit of dynamic shared memory, once for each device (a kernel takes the same
// amount in every launch).
template <auto kKernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};  // a bit for each device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

cudaError_t launch_cache_tables(const CacheGeom& g, const int32_t* add, const int32_t* lens, int32_t* tables,
                                int32_t* free_pages, const int32_t* free_state, int32_t* lens_out,
                                int32_t* free_state_out, int32_t* cu_new, int32_t* slots, int32_t max_tokens,
                                int32_t* status, cudaStream_t st);
cudaError_t launch_cache_append(const CacheGeom& g, const __nv_bfloat16* K, int64_t k_stride, const __nv_bfloat16* V,
                                int64_t v_stride, int32_t max_tokens, const int32_t* cu_new, const int32_t* lens,
                                const int32_t* slots, const int32_t* tables, uint8_t* Kc, uint8_t* Vc, float* Ks,
                                float* Vs, float* Kbar, cudaStream_t st);
cudaError_t launch_cache_decode(const CacheGeom& g, const __nv_bfloat16* Q, const uint8_t* Kc, const uint8_t* Vc,
                                const float* Ks, const float* Vs, const float* Kbar, const int32_t* lens,
                                const int32_t* tables, int32_t* sel, const CacheDecodeWork& w, __nv_bfloat16* O,
                                float* LSE, cudaStream_t st);

}  // namespace moba
