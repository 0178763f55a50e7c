// New keys and values into a paged 8-bit cache, with a scale for each page and KV head.
//
// For the new rows X of one (page, KV head) with `off` older rows before them:
//   t     = least number of 8 significant bits with t * qmax >= max(2^-96, max |x| over finite x)
//   scale = off > 0 ? max(old scale, t) : t             (qmax: 448 for e4m3, 127 for int8)
//   code  = rn(x / scale), clamped;   older codes, when the scale grew: rn(code * old / scale).
// Scales are kept to 8 significant bits, as bf16 values have: a quotient of two such numbers is
// either exactly half-way between two codes or at least 2^-17 (relative) away from there, so the
// fp32 quotient never lands on the wrong side and codes equal those of the exact formula.
//
// A MoBA block whose last token this call writes gets its pooled key: the mean of the block's
// stored (dequantised) keys, read back from the pages; the gate then ranks what attention sees.
//
// Bound by HBM for prompts (bf16 in, codes out: 6 bytes for each element of K and V together), by
// latency for single tokens.  One CTA per (request, KV head, K or V) takes the request's touched
// pages one after the other.
#include "moba.h"
#include <float.h>

#include "cache.cuh"

namespace moba {
namespace {

constexpr int kAppThreads = 256;
constexpr float kTiny = 0x1p-96f;  // keeps scales and quotients far from the subnormal range

// max over the block (every thread gets it); red holds one value a warp.
__device__ __forceinline__ float block_max(float x, float* red) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  x = red[0];
#pragma unroll
  for (int w = 1; w < kAppThreads / 32; ++w) x = fmaxf(x, red[w]);
  return x;
}

// Least number of 8 significant bits that takes magnitude a to the largest code.
template <int kFmt>
__device__ __forceinline__ float scale_for(float a) {
  constexpr float qmax = kFmt == MOBA_CACHE_E4M3 ? 448.f : 127.f;
  a = fmaxf(a, kTiny);
  const uint32_t down = __float_as_uint(__fdiv_rn(a, qmax)) & 0xffff0000u;
  // 8 bits times 7 bits: the product is exact
  return __uint_as_float(__uint_as_float(down) * qmax < a ? down + 0x10000u : down);
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= FLT_MAX ? a : 0.f;  // NaN fails the comparison too
}

// Rows [0, nr) of src (token stride `stride` elements) into rows [off, off + nr) of a slab.
template <int kD, int kFmt>
__device__ __forceinline__ void quantise_rows(const __nv_bfloat16* __restrict__ src, int64_t stride, int nr, int off,
                                              uint8_t* slab, float* scale_ptr, float* red) {
  constexpr int kVec = kD / 8;                        // 16-byte vectors of a row
  constexpr int kIt = 128 * kVec / kAppThreads;       // for the largest page
  uint4 x[kIt];
  float a = 0.f;
#pragma unroll
  for (int it = 0; it < kIt; ++it) {
    const int i = it * kAppThreads + (int)threadIdx.x, r = i / kVec, v = i % kVec;
    if (r < nr) {
      x[it] = __ldg(reinterpret_cast<const uint4*>(src + (int64_t)r * stride) + v);
      const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&x[it]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = __bfloat1622float2(h[e]);
        a = fmaxf(a, fmaxf(finite_abs(f.x), finite_abs(f.y)));
      }
    }
  }
  a = block_max(a, red);
  const float old = off > 0 ? *scale_ptr : 0.f;
  float scale = scale_for<kFmt>(a);
  if (off > 0 && old > scale) scale = old;
  __syncthreads();  // every thread has read the old scale
  if (threadIdx.x == 0) *scale_ptr = scale;
  if (off > 0 && old < scale) {
    uint2* rows = reinterpret_cast<uint2*>(slab);
    for (int i = threadIdx.x; i < off * kVec; i += kAppThreads) {
      const uint2 c = rows[i];
      uint32_t in[2] = {c.x, c.y}, out[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 lo = codes2_to_float2<kFmt>(in[e]), hi = codes2_to_float2<kFmt>(in[e] >> 16);
        out[e] = float2_to_codes2<kFmt>(__fdiv_rn(lo.x * old, scale), __fdiv_rn(lo.y * old, scale)) |
                 float2_to_codes2<kFmt>(__fdiv_rn(hi.x * old, scale), __fdiv_rn(hi.y * old, scale)) << 16;
      }
      rows[i] = make_uint2(out[0], out[1]);
    }
  }
#pragma unroll
  for (int it = 0; it < kIt; ++it) {
    const int i = it * kAppThreads + (int)threadIdx.x, r = i / kVec, v = i % kVec;
    if (r < nr) {
      const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&x[it]);
      uint32_t out[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 lo = __bfloat1622float2(h[2 * e]), hi = __bfloat1622float2(h[2 * e + 1]);
        out[e] = float2_to_codes2<kFmt>(__fdiv_rn(lo.x, scale), __fdiv_rn(lo.y, scale)) |
                 float2_to_codes2<kFmt>(__fdiv_rn(hi.x, scale), __fdiv_rn(hi.y, scale)) << 16;
      }
      reinterpret_cast<uint2*>(slab + (size_t)(off + r) * kD)[v] = make_uint2(out[0], out[1]);
    }
  }
}

// Mean of block b's stored keys of one head (the whole CTA; every token is in the cache).
template <int kD, int kFmt>
__device__ __forceinline__ void pool_cached_block(const CacheGeom& g, const int32_t* __restrict__ table, int b,
                                                  int head, const uint8_t* Kc, const float* Ks, float* out,
                                                  float (*red)[kD + 4]) {
  constexpr int kVec = kD / 16;                      // 16-code vectors of a row
  constexpr int kGroups = kAppThreads / kVec;        // rows in flight
  const int v = threadIdx.x % kVec, r0 = threadIdx.x / kVec;
  float acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int t = r0; t < g.bs; t += kGroups) {
    const int pos = b * g.bs + t;
    const int32_t page = __ldg(table + pos / g.ps);
    if (!page_ok(g, page)) {
      atomicOr(g.err, kErrBadPage);
      continue;
    }
    const float sc = Ks[(size_t)page * g.Hkv + head];
    const uint4 c = reinterpret_cast<const uint4*>(Kc + slab_offset(g, page, head) + (size_t)(pos % g.ps) * kD)[v];
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 lo = codes2_to_float2<kFmt>(w[e]), hi = codes2_to_float2<kFmt>(w[e] >> 16);
      acc[4 * e] = fmaf(lo.x, sc, acc[4 * e]);
      acc[4 * e + 1] = fmaf(lo.y, sc, acc[4 * e + 1]);
      acc[4 * e + 2] = fmaf(hi.x, sc, acc[4 * e + 2]);
      acc[4 * e + 3] = fmaf(hi.y, sc, acc[4 * e + 3]);
    }
  }
  // row groups of one warp share a lane pattern: fold them first, then the warps in order
#pragma unroll
  for (int off = kVec; off < 32; off <<= 1)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], off);
  __syncthreads();
  if ((threadIdx.x & 31) < kVec)
#pragma unroll
    for (int e = 0; e < 16; ++e) red[threadIdx.x >> 5][v * 16 + e] = acc[e];
  __syncthreads();
  if (threadIdx.x < kD) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kAppThreads / 32; ++w) sum += red[w][threadIdx.x];
    out[threadIdx.x] = sum / (float)g.bs;
  }
}

template <int kD, int kFmt>
__global__ void __launch_bounds__(kAppThreads)
    cache_append_kernel(CacheGeom g, const __nv_bfloat16* __restrict__ K, int64_t k_stride,
                        const __nv_bfloat16* __restrict__ V, int64_t v_stride, int32_t max_tokens,
                        const int32_t* __restrict__ cu_new, const int32_t* __restrict__ lens,
                        const int32_t* __restrict__ slots, const int32_t* __restrict__ tables, uint8_t* Kc,
                        uint8_t* Vc, float* Ks, float* Vs, float* Kbar) {
  __shared__ float red[kAppThreads / 32];
  __shared__ float pool_red[kAppThreads / 32][kD + 4];
  const int head = blockIdx.x, s = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const int32_t t0 = max(__ldg(cu_new + s), 0), t1 = min(__ldg(cu_new + s + 1), max_tokens);
  const int32_t len = cached_len(g, lens, s), n = t1 - t0, start = len - n;
  if (n <= 0 || start < 0) return;
  const __nv_bfloat16* src = (is_v ? V : K) + (size_t)head * kD;
  const int64_t stride = is_v ? v_stride : k_stride;
  for (int32_t pos = start; pos < len;) {
    const int off = pos % g.ps, nr = min(g.ps - off, len - pos);
    const int32_t t = t0 + (pos - start), slot = __ldg(slots + t);
    const int32_t page = slot / g.ps;
    if (slot >= 0 && slot % g.ps == off && page_ok(g, page)) {
      const size_t at = (size_t)page * g.Hkv + head;
      quantise_rows<kD, kFmt>(src + (int64_t)t * stride, stride, nr, off, (is_v ? Vc : Kc) + slab_offset(g, page, head),
                              (is_v ? Vs : Ks) + at, red);
    } else if (slot >= 0 && threadIdx.x == 0) {
      atomicOr(g.err, kErrBadPage);
    }
    pos += nr;
  }
  if (is_v) return;
  __syncthreads();  // the codes are visible to the whole CTA
  for (int b = start / g.bs; b < len / g.bs; ++b)
    pool_cached_block<kD, kFmt>(g, tables + (size_t)s * g.MP, b, head, Kc, Ks,
                                Kbar + (((size_t)s * g.MB + b) * g.Hkv + head) * kD, pool_red);
}

}  // namespace

cudaError_t launch_cache_append(const CacheGeom& g, const __nv_bfloat16* K, int64_t k_stride, const __nv_bfloat16* V,
                                int64_t v_stride, int32_t max_tokens, const int32_t* cu_new, const int32_t* lens,
                                const int32_t* slots, const int32_t* tables, uint8_t* Kc, uint8_t* Vc, float* Ks,
                                float* Vs, float* Kbar, cudaStream_t st) {
  const dim3 grid((unsigned)g.Hkv, (unsigned)g.B, 2);
  auto go = [&](auto kernel) {
    kernel<<<grid, kAppThreads, 0, st>>>(g, K, k_stride, V, v_stride, max_tokens, cu_new, lens, slots, tables, Kc, Vc,
                                         Ks, Vs, Kbar);
    return cudaGetLastError();
  };
  if (g.D == 64)
    return g.fmt == MOBA_CACHE_E4M3 ? go(cache_append_kernel<64, MOBA_CACHE_E4M3>) : go(cache_append_kernel<64, MOBA_CACHE_INT8>);
  return g.fmt == MOBA_CACHE_E4M3 ? go(cache_append_kernel<128, MOBA_CACHE_E4M3>) : go(cache_append_kernel<128, MOBA_CACHE_INT8>);
}

}  // namespace moba
