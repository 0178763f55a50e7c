// Gated decode over a paged 8-bit KV cache: one new query per request (the newest cached token,
// at position len - 1, in block i = (len - 1) / bs) attends to its own block up to itself and to
// the top_k - 1 earlier blocks with the largest <q, Kbar[b]>, ties to the lower block:
//   z_j = scale * <q, code_j> * Ks[page(j)],  O = sum_j softmax(z)_j * code'_j * Vs[page(j)],
//   LSE = log sum_j exp(z_j).   A request of length 0 gets O = 0, LSE = -inf, no blocks.
// The gate's outcome is discrete, so its scores are summed in 64 bits (bf16 times fp32 is exact
// there): the choice is that of the exact scores but for ties to 2^-50.
#include <float.h>

#include "cache.cuh"

namespace moba {
namespace {

constexpr float kLn2C = 0.6931471805599453f;

__device__ __forceinline__ bool ranks_before(double sa, int32_t ba, double sb, int32_t bb) {
  return sa > sb || (sa == sb && ba < bb);
}

// One CTA per (request, KV head): scores of the group's heads, then one warp a head picks.
template <int kD>
__global__ void __launch_bounds__(256)
    cache_gate_kernel(CacheGeom g, const __nv_bfloat16* __restrict__ Q, const float* __restrict__ Kbar,
                      const int32_t* __restrict__ lens, double* score, int32_t* __restrict__ sel) {
  constexpr int kDL = kD / 32;
  const int gk = blockIdx.x, s = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t len = cached_len(g, lens, s);
  const int i = len > 0 ? (len - 1) / g.bs : -1;
  for (int b = warp; b < i; b += 8) {
    float kb[kDL];
#pragma unroll
    for (int x = 0; x < kDL; ++x) kb[x] = __ldg(Kbar + (((size_t)s * g.MB + b) * g.Hkv + gk) * kD + lane + 32 * x);
    for (int hh = 0; hh < g.G; ++hh) {
      const size_t row = (size_t)s * g.Hq + gk * g.G + hh;
      double acc = 0.0;
#pragma unroll
      for (int x = 0; x < kDL; ++x)
        acc = fma((double)__bfloat162float(Q[row * kD + lane + 32 * x]), (double)kb[x], acc);
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
      if (lane == 0) score[row * g.MB + b] = acc == acc ? acc : -INFINITY;  // NaN ranks last
    }
  }
  __syncthreads();
  const int m = min(g.k - 1, max(i, 0));
  for (int hh = warp; hh < g.G; hh += 8) {
    const size_t row = (size_t)s * g.Hq + gk * g.G + hh;
    int32_t* out = sel + row * g.k;
    if (lane == 0) out[0] = i;
    double last = INFINITY;
    int32_t last_b = -1;
    for (int q = 0; q < m; ++q) {
      double bs_ = -INFINITY;
      int32_t bb = INT32_MAX;
      for (int b = lane; b < i; b += 32) {
        const double v = score[row * g.MB + b];
        if (ranks_before(last, last_b, v, b) && ranks_before(v, b, bs_, bb)) { bs_ = v; bb = b; }
      }
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) {
        const double os = __shfl_xor_sync(0xffffffffu, bs_, off);
        const int32_t ob = __shfl_xor_sync(0xffffffffu, bb, off);
        if (ranks_before(os, ob, bs_, bb)) { bs_ = os; bb = ob; }
      }
      if (lane == 0) out[1 + q] = bb;
      last = bs_;
      last_b = bb;
    }
    for (int q = 1 + m + lane; q < g.k; q += 32) out[q] = -1;
  }
}

// One CTA per (slot, query head, request): a warp takes every fourth key, a lane D/32 dimensions.
template <int kD, int kFmt>
__global__ void __launch_bounds__(128)
    cache_attn_kernel(CacheGeom g, const __nv_bfloat16* __restrict__ Q, const uint8_t* __restrict__ Kc,
                      const uint8_t* __restrict__ Vc, const float* __restrict__ Ks, const float* __restrict__ Vs,
                      const int32_t* __restrict__ lens, const int32_t* __restrict__ tables,
                      const int32_t* __restrict__ sel, float* __restrict__ part_o, float* __restrict__ part_lse) {
  constexpr int kDL = kD / 32;
  __shared__ float red_o[4][kD], red_m[4], red_l[4];
  const int slot = blockIdx.x, h = blockIdx.y, s = blockIdx.z, gk = h / g.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t unit = ((size_t)s * g.Hq + h) * g.k + slot;
  const int32_t b = __ldg(sel + unit);
  if (b < 0) return;
  const int32_t len = cached_len(g, lens, s), n = min(g.bs, len - b * g.bs);
  float q[kDL], o[kDL], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int x = 0; x < kDL; ++x) {
    q[x] = __bfloat162float(Q[((size_t)s * g.Hq + h) * kD + lane * kDL + x]) * g.scale_log2;
    o[x] = 0.f;
  }
  for (int j = warp; j < n; j += 4) {
    const int pos = b * g.bs + j;
    const int32_t page = __ldg(tables + (size_t)s * g.MP + pos / g.ps);
    if (!page_ok(g, page)) {
      if (lane == 0) atomicOr(g.err, kErrBadPage);
      continue;
    }
    const size_t at = slab_offset(g, page, gk) + (size_t)(pos % g.ps) * kD + lane * kDL;
    float z = 0.f, v[kDL];
#pragma unroll
    for (int x = 0; x < kDL; x += 2) {
      const float2 k2 = codes2_to_float2<kFmt>(*reinterpret_cast<const uint16_t*>(Kc + at + x));
      const float2 v2 = codes2_to_float2<kFmt>(*reinterpret_cast<const uint16_t*>(Vc + at + x));
      z = fmaf(q[x], k2.x, fmaf(q[x + 1], k2.y, z));
      v[x] = v2.x;
      v[x + 1] = v2.y;
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
    z *= __ldg(Ks + (size_t)page * g.Hkv + gk);
    const float vs = __ldg(Vs + (size_t)page * g.Hkv + gk);
    const float m_new = fmaxf(m, z), alpha = m == m_new ? 1.f : exp2f(m - m_new), p = exp2f(z - m_new);
    l = l * alpha + p;
#pragma unroll
    for (int x = 0; x < kDL; ++x) o[x] = fmaf(p * vs, v[x], o[x] * alpha);
    m = m_new;
  }
  if (lane == 0) {
    red_m[warp] = m;
    red_l[warp] = l;
  }
#pragma unroll
  for (int x = 0; x < kDL; ++x) red_o[warp][lane * kDL + x] = o[x];
  __syncthreads();
  if (threadIdx.x < kD) {
    float M = -INFINITY, L = 0.f, acc = 0.f;
    for (int w = 0; w < 4; ++w) M = fmaxf(M, red_m[w]);
    for (int w = 0; w < 4; ++w) {
      const float c = red_m[w] == -INFINITY && M != red_m[w] ? 0.f : exp2f(red_m[w] - M);
      if (red_l[w] == 0.f) continue;  // no key of this warp
      L = fmaf(red_l[w], c, L);
      acc = fmaf(red_o[w][threadIdx.x], c, acc);
    }
    part_o[unit * kD + threadIdx.x] = L > 0.f || L != L ? acc / L : 0.f;
    if (threadIdx.x == 0) part_lse[unit] = L > 0.f || L != L ? M + log2f(L) : -INFINITY;
  }
}

// The slots of a (request, head) merged by online softmax; part_lse in log2 units.
template <int kD>
__global__ void __launch_bounds__(128)
    cache_merge_kernel(CacheGeom g, const int32_t* __restrict__ sel, const float* __restrict__ part_o,
                       const float* __restrict__ part_lse, __nv_bfloat16* __restrict__ O, float* __restrict__ LSE) {
  constexpr int kDL = kD / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t row = (size_t)blockIdx.x * 4 + warp;
  if (row >= (size_t)g.B * g.Hq) return;
  float M = -INFINITY, L = 0.f, acc[kDL];
#pragma unroll
  for (int x = 0; x < kDL; ++x) acc[x] = 0.f;
  for (int q = 0; q < g.k; ++q)
    if (__ldg(sel + row * g.k + q) >= 0) M = fmaxf(M, __ldg(part_lse + row * g.k + q));
  for (int q = 0; q < g.k; ++q) {
    if (__ldg(sel + row * g.k + q) < 0) continue;
    const float t = __ldg(part_lse + row * g.k + q);
    if (t == -INFINITY) continue;  // no key in this block
    const float w = exp2f(t - M);
    L += w;
#pragma unroll
    for (int x = 0; x < kDL; ++x) acc[x] = fmaf(w, __ldg(part_o + (row * g.k + q) * kD + lane * kDL + x), acc[x]);
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
  for (int x = 0; x < kDL; x += 2)
    *reinterpret_cast<__nv_bfloat162*>(O + row * kD + lane * kDL + x) = __floats2bfloat162_rn(acc[x] * inv, acc[x + 1] * inv);
  if (lane == 0) LSE[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2C;
}

template <int kD, int kFmt>
cudaError_t launch_decode_t(const CacheGeom& g, const __nv_bfloat16* Q, const uint8_t* Kc, const uint8_t* Vc,
                            const float* Ks, const float* Vs, const float* Kbar, const int32_t* lens,
                            const int32_t* tables, int32_t* sel, const CacheDecodeWork& w, __nv_bfloat16* O,
                            float* LSE, cudaStream_t st) {
  cache_gate_kernel<kD><<<dim3((unsigned)g.Hkv, (unsigned)g.B), 256, 0, st>>>(g, Q, Kbar, lens, w.score, sel);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cache_attn_kernel<kD, kFmt><<<dim3((unsigned)g.k, (unsigned)g.Hq, (unsigned)g.B), 128, 0, st>>>(
      g, Q, Kc, Vc, Ks, Vs, lens, tables, sel, w.part_o, w.part_lse);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const size_t rows = (size_t)g.B * g.Hq;
  cache_merge_kernel<kD><<<(unsigned)((rows + 3) / 4), 128, 0, st>>>(g, sel, w.part_o, w.part_lse, O, LSE);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_decode(const CacheGeom& g, const __nv_bfloat16* Q, const uint8_t* Kc, const uint8_t* Vc,
                                const float* Ks, const float* Vs, const float* Kbar, const int32_t* lens,
                                const int32_t* tables, int32_t* sel, const CacheDecodeWork& w, __nv_bfloat16* O,
                                float* LSE, cudaStream_t st) {
  auto go = [&](auto fn) { return fn(g, Q, Kc, Vc, Ks, Vs, Kbar, lens, tables, sel, w, O, LSE, st); };
  if (g.D == 64)
    return g.fmt == MOBA_CACHE_E4M3 ? go(launch_decode_t<64, MOBA_CACHE_E4M3>) : go(launch_decode_t<64, MOBA_CACHE_INT8>);
  return g.fmt == MOBA_CACHE_E4M3 ? go(launch_decode_t<128, MOBA_CACHE_E4M3>) : go(launch_decode_t<128, MOBA_CACHE_INT8>);
}

}  // namespace moba
