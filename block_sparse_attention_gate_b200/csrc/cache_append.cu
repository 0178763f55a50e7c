// New keys and values into a paged 8-bit cache, with a scale for each page and KV head.
//
// For the new rows X of one (page, KV head) with `off` older rows before them:
//   t     = least number of 8 significant bits with t * qmax >= max(2^-96, max |x| over finite x)
//   scale = off > 0 ? max(old scale, t) : t             (qmax: 448 for e4m3, 127 for int8)
//   code  = rn(x / scale), clamped;   older codes, when the scale grew: rn(code * old / scale).
// Scales are kept to 8 significant bits, as bf16 values have: a quotient of two such numbers is
// either exactly half-way between two codes or at least 2^-17 (relative) away from there, so fp32
// arithmetic can place every code where the exact formula places it.
//
// A MoBA block whose last token this call writes gets its pooled key: the mean of the block's
// stored (dequantised) keys, so that the gate ranks what attention sees.
//
// Bound by HBM for prompts (bf16 in, codes out: 6 bytes for each element of K and V together), by
// latency for single tokens.  Two forms of one body:
//   cache_append_kernel : a CTA for each (request, KV head, K or V) takes the request's touched
//                         pages one after the other: for requests with few new tokens (2.7 us for
//                         single tokens of 8, 5.8 us for 64 of which some complete a block of 512,
//                         45 us where all 64 complete a block of 2048 of 8 heads of 128).
//   cache_prompt_kernel : for requests with the tokens of kLongPages pages or more, a cluster of up to 8
//                         CTAs for each (touched MoBA block, some KV heads, K or half of V); its CTAs
//                         share the block's pages and add up the pooled key on the way (54769 tokens, 8
//                         heads of 128, pages of 64: 336 MB in 63 us, 5.4 TB/s).
#include <float.h>

#include "cache.cuh"
#include "sm100.cuh"

namespace moba {
namespace {

constexpr int kStepThreads = 256;  // of cache_append_kernel
constexpr int kMaxWarps = kStepThreads / 32;
constexpr int kLongPages = 4;
constexpr int64_t kMostCtas = 8192;  // of a launch of which most may have nothing to do
constexpr float kTiny = 0x1p-96f;  // keeps scales and quotients far from the subnormal range
// Pooled keys are added up under this power of two (exact, down to the smallest scale), so that the sum of
// up to 8192 keys is finite where their mean is.
constexpr float kPoolUnit = 0x1p-14f;
constexpr uint32_t kInfBits = 0x7f80;  // magnitude bits of a bf16 infinity; NaN lies above

template <int kFmt>
__device__ constexpr float qmax_of() {
  return kFmt == MOBA_CACHE_E4M3 ? 448.f : 127.f;
}

// Least number of 8 significant bits that takes magnitude a to the largest code.
template <int kFmt>
__device__ __forceinline__ float scale_for(float a) {
  constexpr float qmax = qmax_of<kFmt>();
  a = fmaxf(a, kTiny);
  // a first guess, at most one step off; 8 bits times at most 7 bits: the products are exact
  uint32_t c = __float_as_uint(a * (1.f / qmax)) & 0xffff0000u;
  if (__uint_as_float(c) * qmax < a) c += 0x10000u;
  if (__uint_as_float(c - 0x10000u) * qmax >= a) c -= 0x10000u;
  return __uint_as_float(c);
}

// Quotients x / s for x and s of 8 significant bits, close enough to be rounded to a code.  `up` is
// 1 / s raised by 2^-21 (and off by at most 2^-23, the reciprocal's own error), so the product lies
// above the quotient by less than 2^-20 of it, and cutting it to 19 bits (steps of 2^-18) gives back
// a quotient that lies half-way between codes (at most 9 bits) exactly, while any other stays on its
// side of the half-way points, from which 2^-17 separate it.  Finite x only.  Half a multiplication
// (two at a time) and one logic operation each, where a division takes about ten.
__device__ __forceinline__ float raised_reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r * (1.f + 0x1p-21f);
}
__device__ __forceinline__ float2 quotients(float x, float y, float up) {
  mul2(x, y, x, y, up, up);
  return make_float2(__uint_as_float(__float_as_uint(x) & ~31u), __uint_as_float(__float_as_uint(y) & ~31u));
}

// Four values as codes.  kClean: finite, with magnitudes up to the largest code.
template <int kFmt, bool kClean>
__device__ __forceinline__ uint32_t codes4(float2 a, float2 b) {
  if constexpr (kFmt == MOBA_CACHE_E4M3) {
    uint32_t r;
    asm("{.reg .b16 l, h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};}" : "=r"(r) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
  } else if constexpr (kClean) {
    // adding 1.5 * 2^23 rounds to an integer, ties to even, and leaves it in the low byte
    constexpr float kMagic = 12582912.f;
    add2(a.x, a.y, a.x, a.y, kMagic, kMagic);
    add2(b.x, b.y, b.x, b.y, kMagic, kMagic);
    return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                       __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
  } else {
    return float2_to_codes2<kFmt>(a.x, a.y) | float2_to_codes2<kFmt>(b.x, b.y) << 16;
  }
}

// The larger magnitude of each half; NaN stays (signs are left to the caller).
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{.reg .b32 x, y;\n\tabs.bf16x2 x, %1;\n\tabs.bf16x2 y, %2;\n\tmax.NaN.bf16x2 %0, x, y;}" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ float2 bf16x2_to_float2(uint32_t x) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

// Eight values over the scale as codes; a page with an infinity or NaN (not kClean) is divided plainly.
template <int kFmt, bool kClean>
__device__ __forceinline__ uint2 quantise8(const uint4& x, float scale, float up) {
  auto q = [&](uint32_t w) {
    const float2 f = bf16x2_to_float2(w);
    return kClean ? quotients(f.x, f.y, up) : make_float2(__fdiv_rn(f.x, scale), __fdiv_rn(f.y, scale));
  };
  return make_uint2(codes4<kFmt, kClean>(q(x.x), q(x.y)), codes4<kFmt, kClean>(q(x.z), q(x.w)));
}

// Sums of codes in the thread's kN columns: exact for int8, in fp32 for e4m3.
template <int kFmt, int kN>
struct CodeSums {
  float f[kFmt == MOBA_CACHE_E4M3 ? kN : 1];
  int i[kFmt == MOBA_CACHE_INT8 ? kN : 1];

  __device__ __forceinline__ CodeSums() : f{}, i{} {}
  // columns [kAt, kAt + 4)
  template <int kAt>
  __device__ __forceinline__ void add4(uint32_t c) {
    if constexpr (kFmt == MOBA_CACHE_E4M3) {
      asm("{.reg .b16 l, h, e, o;\n\t.reg .b32 p;\n\tmov.b32 {l, h}, %4;\n\t"
          "cvt.rn.f16x2.e4m3x2 p, l;\n\tmov.b32 {e, o}, p;\n\tadd.f32.f16 %0, e, %0;\n\tadd.f32.f16 %1, o, %1;\n\t"
          "cvt.rn.f16x2.e4m3x2 p, h;\n\tmov.b32 {e, o}, p;\n\tadd.f32.f16 %2, e, %2;\n\tadd.f32.f16 %3, o, %3;}"
          : "+f"(f[kAt]), "+f"(f[kAt + 1]), "+f"(f[kAt + 2]), "+f"(f[kAt + 3]) : "r"(c));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) i[kAt + e] = __dp4a((int)c, 1 << 8 * e, i[kAt + e]);
    }
  }
  __device__ __forceinline__ float sum(int e) const {
    if constexpr (kFmt == MOBA_CACHE_E4M3) return f[e]; else return (float)i[e];
  }
};

// Largest magnitude (bf16 bits) over the block; red holds one value a warp and is used by one call
// out of two, so that one barrier a call is enough.
template <int kThreads>
__device__ __forceinline__ uint32_t block_max(uint32_t x, uint32_t* red) {
  x = __reduce_max_sync(0xffffffffu, x);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  x = red[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) x = max(x, red[w]);
  return x;
}

// Shared memory of a CTA.
template <int kD>
struct AppendSmem {
  uint32_t red[2][kMaxWarps];
  float pool[kMaxWarps][kD];
  float part[kD];  // this CTA's share of a pooled key
};

// The rows of one (page, KV head): thread holds vector v (8 columns) of rows r + it * kRows.
template <int kD, int kFmt, int kIt, int kThreads>
struct PageRows {
  static constexpr int kVec = kD / 8, kRows = kThreads / kVec;
  uint4 x[kIt];

  // Asynchronously into a stage of the thread's own in shared memory (rows behind nr as zeros), and
  // from there: no thread reads what another one copied, so no barrier is needed.
  static __device__ __forceinline__ void prefetch(uint32_t stage, const __nv_bfloat16* __restrict__ src, int64_t stride,
                                                  int nr) {
    const int v = threadIdx.x % kVec, r = threadIdx.x / kVec;
    const __nv_bfloat16* p = src + (int64_t)r * stride + v * 8;
    stage += threadIdx.x * 16;
    if (nr == kIt * kRows) {
#pragma unroll
      for (int it = 0; it < kIt; ++it, p += kRows * stride) cp_async_16(stage + it * kThreads * 16, p, 16);
    } else {
#pragma unroll
      for (int it = 0; it < kIt; ++it, p += kRows * stride) {
        const bool live = r + it * kRows < nr;
        cp_async_16(stage + it * kThreads * 16, live ? p : src, live ? 16 : 0);
      }
    }
  }
  __device__ __forceinline__ void take(uint32_t stage) {
#pragma unroll
    for (int it = 0; it < kIt; ++it) x[it] = ld_shared_16(stage + (it * kThreads + threadIdx.x) * 16);
  }

  __device__ __forceinline__ void load(const __nv_bfloat16* __restrict__ src, int64_t stride, int nr) {
    const int v = threadIdx.x % kVec, r = threadIdx.x / kVec;
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      x[it] = make_uint4(0, 0, 0, 0);
      if (r + it * kRows < nr)
        x[it] = __ldg(reinterpret_cast<const uint4*>(src + (int64_t)(r + it * kRows) * stride) + v);
    }
  }

  // kFull: every row of the page, at offset 0.
  template <bool kPool, bool kClean, bool kFull>
  __device__ __forceinline__ void write(int nr, uint8_t* dst, float scale, CodeSums<kFmt, 8>& sum) {
    const float up = raised_reciprocal(scale);
    uint2* out = reinterpret_cast<uint2*>(dst) + threadIdx.x;  // rows are kVec vectors apart
#pragma unroll
    for (int it = 0; it < kIt; ++it)
      if (kFull || (int)threadIdx.x / kVec + it * kRows < nr) {
        const uint2 c = quantise8<kFmt, kClean>(x[it], scale, up);
        out[it * kThreads] = c;
        if constexpr (kPool) {
          sum.template add4<0>(c.x);
          sum.template add4<4>(c.y);
        }
      }
  }

  // Into rows [off, off + nr) of the slab.  kPool: sum += codes of the new rows.  Returns the scale.
  template <bool kPool>
  __device__ __forceinline__ float store(int nr, int off, uint8_t* slab, float* scale_ptr, uint32_t (*red)[kMaxWarps],
                                         int& turn, CodeSums<kFmt, 8>& sum) {
    uint32_t big2 = 0;  // two magnitudes side by side
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      big2 = max_abs_bf16x2(max_abs_bf16x2(big2, x[it].x), x[it].y);
      big2 = max_abs_bf16x2(max_abs_bf16x2(big2, x[it].z), x[it].w);
    }
    big2 &= 0x7fff7fffu;
    uint32_t big = block_max<kThreads>(max(big2 & 0xffffu, big2 >> 16), red[turn ^= 1]);
    const bool clean = big < kInfBits;
    if (!clean) {  // the scale is that of the finite values
      big = 0;
#pragma unroll
      for (int it = 0; it < kIt; ++it) {
        const uint32_t w[4] = {x[it].x, x[it].y, x[it].z, x[it].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t lo = w[e] & 0x7fffu, hi = (w[e] >> 16) & 0x7fffu;
          big = max(big, max(lo < kInfBits ? lo : 0u, hi < kInfBits ? hi : 0u));
        }
      }
      big = block_max<kThreads>(big, red[turn ^= 1]);
    }
    float scale = scale_for<kFmt>(__uint_as_float(big << 16));
    if (off > 0) {
      const float old = *scale_ptr;
      if (old > scale) scale = old;
      __syncthreads();  // every thread has read the old scale
      if (old < scale) {
        uint2* rows = reinterpret_cast<uint2*>(slab);
        for (int i = threadIdx.x; i < off * kVec; i += kThreads) {
          const uint2 c = rows[i];
          const uint32_t in[2] = {c.x, c.y};
          uint32_t out[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 lo = codes2_to_float2<kFmt>(in[e]), hi = codes2_to_float2<kFmt>(in[e] >> 16);
            // the product is exact (at most 15 bits), the quotient as close as one of 8-bit numbers needs
            out[e] = codes4<kFmt, false>(make_float2(__fdiv_rn(lo.x * old, scale), __fdiv_rn(lo.y * old, scale)),
                                         make_float2(__fdiv_rn(hi.x * old, scale), __fdiv_rn(hi.y * old, scale)));
          }
          rows[i] = make_uint2(out[0], out[1]);
        }
      }
    }
    if (threadIdx.x == 0) *scale_ptr = scale;
    uint8_t* dst = slab + (size_t)off * kD;
    if (!clean) write<kPool, false, false>(nr, dst, scale, sum);
    else if (nr == kIt * kRows) write<kPool, true, true>(nr, dst, scale, sum);
    else write<kPool, true, false>(nr, dst, scale, sum);
    return scale;
  }
};

// acc += kPoolUnit * scale * (sum of the stored codes of a whole page), as the rows above are spread.
template <int kD, int kFmt, int kThreads>
__device__ __forceinline__ void add_stored_page(const CacheGeom& g, const uint8_t* slab, float scale, float (&acc)[8]) {
  constexpr int kVec = kD / 8, kRows = kThreads / kVec;
  CodeSums<kFmt, 8> sum;
#pragma unroll 8
  for (int r = threadIdx.x / kVec; r < g.ps; r += kRows) {
    const uint2 c = reinterpret_cast<const uint2*>(slab + (size_t)r * kD)[threadIdx.x % kVec];
    sum.template add4<0>(c.x);
    sum.template add4<4>(c.y);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = fmaf(sum.sum(e), scale * kPoolUnit, acc[e]);
}

// The CTA's sums of its columns (kN of them in each lane): part[d] for all d < kD, visible after the
// caller's next barrier.
template <int kD, int kN, int kThreads>
__device__ __forceinline__ void fold_columns(float (&acc)[kN], AppendSmem<kD>& sm) {
  constexpr int kVec = kD / kN;
#pragma unroll
  for (int off = kVec; off < 32; off <<= 1)
#pragma unroll
    for (int e = 0; e < kN; ++e) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], off);
  __syncthreads();  // an earlier fold is read
  if ((threadIdx.x & 31) < kVec)
#pragma unroll
    for (int e = 0; e < kN; ++e) sm.pool[threadIdx.x >> 5][(threadIdx.x & 31) * kN + e] = acc[e];
  __syncthreads();
  if (threadIdx.x < kD) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += sm.pool[w][threadIdx.x];
    sm.part[threadIdx.x] = s;
  }
}

// One side (K or V) of an append.
struct AppendSide {
  const __nv_bfloat16* src;
  int64_t stride;
  uint8_t* codes;
  float* scales;
};

// Page that a request's run of new tokens in one page goes to, by the slot of the first of them, which has
// to be at that token's offset in a page of the pool; -1 if the run is left out.  The other slots of a run
// follow from it and are not read.
__device__ __forceinline__ int32_t page_of_slot(const CacheGeom& g, int32_t slot, int off) {
  if (slot < 0) return -1;
  if (slot % g.ps == off && page_ok(g, slot / g.ps)) return slot / g.ps;
  if (threadIdx.x == 0) atomicOr(g.err, kErrBadPage);
  return -1;
}

template <int kD, int kFmt>
__global__ void __launch_bounds__(kStepThreads)
    cache_append_kernel(CacheGeom g, AppendSide sk, AppendSide sv, int32_t max_tokens, int32_t too_long,
                        const int32_t* __restrict__ cu_new, const int32_t* __restrict__ lens,
                        const int32_t* __restrict__ slots, const int32_t* __restrict__ tables, float* Kbar) {
  __shared__ AppendSmem<kD> sm;
  const int head = blockIdx.x, s = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const AppendSide a = is_v ? sv : sk;
  const int32_t t0 = max(__ldg(cu_new + s), 0), t1 = min(__ldg(cu_new + s + 1), max_tokens);
  const int32_t len = cached_len(g, lens, s), n = t1 - t0, start = len - n;
  if (n <= 0 || start < 0 || n >= too_long) return;
  int turn = 0;
  for (int32_t pos = start; pos < len;) {
    const int off = pos % g.ps, nr = min(g.ps - off, len - pos);
    const int32_t t = t0 + (pos - start), page = page_of_slot(g, __ldg(slots + t), off);
    if (page >= 0) {
      PageRows<kD, kFmt, 128 * kD / 8 / kStepThreads, kStepThreads> rows;  // any page size
      CodeSums<kFmt, 8> unused;
      rows.load(a.src + (size_t)head * kD + (int64_t)t * a.stride, a.stride, nr);
      rows.template store<false>(nr, off, a.codes + slab_offset(g, page, head), a.scales + (size_t)page * g.Hkv + head,
                                 sm.red, turn, unused);
    }
    pos += nr;
  }
  if (is_v) return;
  __syncthreads();  // the codes and scales are visible to the whole CTA
  // a warp takes every eighth page of a completed block, 32 rows of it at a time
  constexpr int kVec = kD / 16, kRows = 32 / kVec;
  const int warp = threadIdx.x >> 5, v = (threadIdx.x & 31) % kVec, r0 = (threadIdx.x & 31) / kVec;
  for (int b = start / g.bs; b < len / g.bs; ++b) {
    float acc[16] = {};
    for (int pi = b * (g.bs / g.ps) + warp; pi < (b + 1) * (g.bs / g.ps); pi += kStepThreads / 32) {
      const int32_t page = __ldg(tables + (size_t)s * g.MP + pi);
      if (!page_ok(g, page)) {
        if ((threadIdx.x & 31) == 0) atomicOr(g.err, kErrBadPage);
        continue;
      }
      const float scale = a.scales[(size_t)page * g.Hkv + head] * kPoolUnit;
      const uint4* src = reinterpret_cast<const uint4*>(a.codes + slab_offset(g, page, head)) + v;
      CodeSums<kFmt, 16> sum;
#pragma unroll 8
      for (int r = r0; r < g.ps; r += kRows) {
        const uint4 c = src[r * kVec];
        sum.template add4<0>(c.x);
        sum.template add4<4>(c.y);
        sum.template add4<8>(c.z);
        sum.template add4<12>(c.w);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[e] = fmaf(sum.sum(e), scale, acc[e]);
    }
    fold_columns<kD, 16, kStepThreads>(acc, sm);
    if (threadIdx.x < kD)
      Kbar[(((size_t)s * g.MB + b) * g.Hkv + head) * kD + threadIdx.x] = sm.part[threadIdx.x] / (kPoolUnit * (float)g.bs);
  }
}

// A long request's new tokens, and which of its touched MoBA blocks a work item is.
struct LongRun {
  int32_t s, t0, start, len, block;
};

// Work items are the touched blocks of the long requests, in the order of the requests: a scan of how
// many each has, a thread a request, until the item's is found (run->s < 0: there are fewer).
template <int kThreads>
__device__ __forceinline__ void find_run(const CacheGeom& g, const int32_t* __restrict__ cu_new,
                                         const int32_t* __restrict__ lens, int32_t max_tokens, int32_t too_short, int item,
                                         int32_t (*sums)[kThreads / 32], LongRun* run) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) run->s = -1;
  int32_t before = 0;
  int turn = 0;
  for (int s0 = 0; s0 < g.B && before <= item; s0 += kThreads) {
    const int s = s0 + (int)threadIdx.x;
    LongRun r{s, 0, 0, 0, 0};
    int32_t count = 0;
    if (s < g.B) {
      r.t0 = max(__ldg(cu_new + s), 0);
      const int32_t n = min(__ldg(cu_new + s + 1), max_tokens) - r.t0;
      r.len = cached_len(g, lens, s);
      r.start = r.len - n;
      if (n > too_short && r.start >= 0) count = (r.len - 1) / g.bs - r.start / g.bs + 1;
    }
    int32_t inc = count;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int32_t o = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += o;
    }
    turn ^= 1;  // sums of two rounds ago are read
    if (lane == 31) sums[turn][warp] = inc;
    __syncthreads();
    int32_t at = before + inc - count;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) at += sums[turn][w];
      before += sums[turn][w];
    }
    if (item >= at && item < at + count) {
      r.block = r.start / g.bs + (item - at);
      *run = r;
    }
  }
  __syncthreads();
}

__host__ __device__ constexpr int prompt_threads(int ps) { return ps == 128 ? 256 : 128; }

// kPS: tokens of a page; kAhead: pages on their way while one is written.
template <int kD, int kFmt, int kPS, int kAhead>
__global__ void __launch_bounds__(prompt_threads(kPS), kPS == 128 ? 3 : 6)
    cache_prompt_kernel(CacheGeom g, AppendSide sk, AppendSide sv, int32_t max_tokens, int32_t too_short, int ranks,
                        int heads, const int32_t* __restrict__ cu_new, const int32_t* __restrict__ lens,
                        const int32_t* __restrict__ slots, const int32_t* __restrict__ tables, float* Kbar) {
  constexpr int kPromptThreads = prompt_threads(kPS), kIt = kPS * (kD / 8) / kPromptThreads;
  using Rows = PageRows<kD, kFmt, kIt, kPromptThreads>;
  constexpr uint32_t kStageBytes = kIt * kPromptThreads * 16;
  g.ps = kPS;
  __shared__ AppendSmem<kD> sm;
  extern __shared__ __align__(16) uint8_t stages[];
  const int item = blockIdx.x / ranks, rank = blockIdx.x % ranks;
  const bool is_v = blockIdx.z != 0;
  const AppendSide a = is_v ? sv : sk;
  __shared__ LongRun run;
  __shared__ int32_t sums[2][kPromptThreads / 32];
  find_run<kPromptThreads>(g, cu_new, lens, max_tokens, too_short, item, sums, &run);
  const int32_t s = run.s, t0 = run.t0, start = run.start, len = run.len, b = run.block;
  if (s < 0) return;  // the same for the whole cluster
  const bool pool = !is_v && (int64_t)(b + 1) * g.bs <= len;
  const int R = g.bs / g.ps, per = (R + ranks - 1) / ranks;
  int p0 = b * R + rank * per, p1 = b * R + min(R, (rank + 1) * per);
  if (is_v) {  // in halves: the short CTAs come last and fill the last round of CTAs (3 % of a long prompt)
    const int half = (max(p1 - p0, 0) + 1) / 2;
    if (blockIdx.z == 1) p1 = min(p1, p0 + half); else p0 += half;
  }
  // new rows of page ordinal p: packed row of the first, how many, and the older rows before them
  auto rows_of = [&](int p, int32_t& t, int& nr, int& off) {
    const int32_t lo = max(start, p * g.ps), hi = min(len, (p + 1) * g.ps);
    t = t0 + (lo - start);
    off = lo - p * g.ps;
    nr = p < p1 ? max(hi - lo, 0) : 0;
  };
  const uint32_t ring = smem_u32(stages);
  int turn = 0;
  // slot of a page's first new token, and the page that the block table names (the pooled key is that of
  // these pages), read one page ahead and looked at only when it is their turn
  auto slot_of = [&](int p) -> int32_t {
    int32_t t;
    int nr, off;
    rows_of(p, t, nr, off);
    return nr > 0 ? __ldg(slots + t) : -1;
  };
  auto listed_at = [&](int p) -> int32_t { return pool && p < p1 ? __ldg(tables + (size_t)s * g.MP + p) : -1; };
  for (int head = blockIdx.y * heads; head < min(g.Hkv, (int)(blockIdx.y + 1) * heads); ++head) {
    const __nv_bfloat16* src = a.src + (size_t)head * kD;
    auto prefetch = [&](int p, int stage) {
      int32_t t;
      int nr, off;
      rows_of(p, t, nr, off);
      if (nr > 0) Rows::prefetch(ring + stage * kStageBytes, src + (int64_t)t * a.stride, a.stride, nr);
      cp_async_commit();
    };
#pragma unroll
    for (int q = 0; q < kAhead; ++q) prefetch(p0 + q, q);
    int stage = 0;
    int32_t slot = slot_of(p0), listed = listed_at(p0);
    float acc[8] = {};
    for (int p = p0; p < p1; ++p) {
      prefetch(p + kAhead, stage == 0 ? kAhead : stage - 1);  // the stage that the last page left
      const int32_t slot_n = slot_of(p + 1), listed_n = listed_at(p + 1);
      int32_t t;
      int nr, off;
      rows_of(p, t, nr, off);
      const int32_t page = page_of_slot(g, slot, off);
      if (pool && !page_ok(g, listed)) {
        if (threadIdx.x == 0) atomicOr(g.err, kErrBadPage);
        listed = -1;
      }
      cp_async_wait<kAhead>();
      Rows rows;
      if (page >= 0) rows.take(ring + stage * kStageBytes);
      float* sp = a.scales + (size_t)max(page, 0) * g.Hkv + head;
      uint8_t* slab = a.codes + slab_offset(g, max(page, 0), head);
      if (pool && page >= 0 && page == listed && off == 0) {
        CodeSums<kFmt, 8> sum;
        const float scale = rows.template store<true>(nr, off, slab, sp, sm.red, turn, sum);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = fmaf(sum.sum(e), scale * kPoolUnit, acc[e]);
      } else {
        CodeSums<kFmt, 8> unused;
        if (page >= 0) rows.template store<false>(nr, off, slab, sp, sm.red, turn, unused);
        if (pool) {  // older rows are in the page: read all of it back
          __syncthreads();
          if (listed >= 0)
            add_stored_page<kD, kFmt, kPromptThreads>(g, a.codes + slab_offset(g, listed, head),
                                                      a.scales[(size_t)listed * g.Hkv + head], acc);
        }
      }
      slot = slot_n;
      listed = listed_n;
      stage = stage == kAhead ? 0 : stage + 1;
    }
    if (!pool) continue;  // the same for the whole cluster
    fold_columns<kD, 8, kPromptThreads>(acc, sm);
    cluster_barrier();
    if (rank == 0 && threadIdx.x < kD) {
      float total = sm.part[threadIdx.x];
      for (int r = 1; r < ranks; ++r) total += ld_cluster_f32(&sm.part[threadIdx.x], r);
      Kbar[(((size_t)s * g.MB + b) * g.Hkv + head) * kD + threadIdx.x] = total / (kPoolUnit * (float)g.bs);
    }
    cluster_barrier();  // no CTA goes on while its share is read
  }
}

template <int kD, int kFmt, int kPS, int kAhead>
cudaError_t launch_prompt(const CacheGeom& g, const AppendSide& sk, const AppendSide& sv, int32_t max_tokens,
                          int32_t too_short, const int32_t* cu_new, const int32_t* lens, const int32_t* slots,
                          const int32_t* tables, float* Kbar, cudaStream_t st) {
  // n tokens touch at most n / bs + 2 blocks
  const int64_t runs = too_short > 0 ? max_tokens / (too_short + 1) : g.B;
  const int64_t items = max_tokens / g.bs + 2 * (runs < g.B ? runs : g.B);
  // CTAs of a cluster: at least 128 rows each, and at most 4 once there are several rounds of CTAs (each
  // begins with a few loads one behind the other, which longer runs of pages spread): prompts of 128K
  // tokens took 77 us with 4, 80 with 8 and 82 with 2; 8K tokens 6.8 with 8 and 8.2 with 4
  const int most = items * g.Hkv * 2 * 8 > 4 * 148 * 6 ? 4 : 8;
  int ranks = 1;
  while (ranks < most && 2 * ranks * 128 <= g.bs) ranks *= 2;
  // heads of a CTA: one, but more where most of the items may turn out not to be there, as even an empty
  // CTA takes 1.5 ns to start
  int heads = 1;
  while (heads < g.Hkv && items * ranks * ((g.Hkv + heads - 1) / heads) * 3 > kMostCtas) heads *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(items * ranks), (unsigned)((g.Hkv + heads - 1) / heads), 3);
  cfg.blockDim = dim3(prompt_threads(kPS));
  cfg.dynamicSmemBytes = (kAhead + 1) * kPS * kD * 2;
  cfg.stream = st;
  const cudaError_t e = allow_smem<cache_prompt_kernel<kD, kFmt, kPS, kAhead>>((int)cfg.dynamicSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_prompt_kernel<kD, kFmt, kPS, kAhead>, g, sk, sv, max_tokens, too_short, ranks,
                            heads, cu_new, lens, slots,
                            tables, Kbar);
}

template <int kD, int kFmt>
cudaError_t launch_append_t(const CacheGeom& g, const AppendSide& sk, const AppendSide& sv, int32_t max_tokens,
                            const int32_t* cu_new, const int32_t* lens, const int32_t* slots, const int32_t* tables,
                            float* Kbar, cudaStream_t st) {
  // Where a request has two pages of new tokens on average, all go as prompts; else those with fewer than
  // kLongPages one page after the other and then the others, where there can be any.  Up to 4 tokens a slot
  // count as decode steps and drafts, without long runs: the second launch would cost them 2 to 3 us (10.1
  // and 12.8 for 256 tokens in one of 256 slots).  A long run among so many slots is slow by that: 1024
  // tokens in one of 256 slots 25 us, 13 with the second launch; 4000 in one of 1000 101 and 37.
  // Pages of 64, 8 heads of 128, us one page after the other / all as prompts / by this rule: 1 request with
  // 256 tokens 11.6 / 7.7 / 7.7; 24 with 300 31 / 27 / 27; 64 with 600 76 / 75 / 75; 64 with 16 8.9 / 33 /
  // 11.4; one with 8000 beside 63 with one 181 / 42 / 26.  The rule also loses where many requests have a few
  // pages each: 32 with 128 15 / 26 / 26, 64 with 256 41 / 53 / 53.  Limits of 8 pages for full grids give 19
  // and 48 us there, but 35 for 24 with 300 and 35 instead of 31 for 32 with 256.
  const int32_t tokens = kLongPages * g.ps;
  const bool prompts = max_tokens >= 2 * (int64_t)g.ps * g.B;
  const bool few = max_tokens < tokens || max_tokens <= 4 * (int64_t)g.B;
  if (!prompts) {
    cache_append_kernel<kD, kFmt><<<dim3((unsigned)g.Hkv, (unsigned)g.B, 2), kStepThreads, 0, st>>>(
        g, sk, sv, max_tokens, few ? INT32_MAX : tokens, cu_new, lens, slots, tables, Kbar);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || few) return e;
  }
  const int32_t too_short = prompts ? 0 : tokens - 1;
  auto go = [&](auto fn) { return fn(g, sk, sv, max_tokens, too_short, cu_new, lens, slots, tables, Kbar, st); };
  switch (g.ps) {  // 24 to 64 KB of shared memory: 3 or more CTAs on an SM
    case 16: return go(launch_prompt<kD, kFmt, 16, 4>);
    case 32: return go(launch_prompt<kD, kFmt, 32, 2>);
    case 64: return go(launch_prompt<kD, kFmt, 64, 1>);
    default: return go(launch_prompt<kD, kFmt, 128, 1>);
  }
}

}  // namespace

cudaError_t launch_cache_append(const CacheGeom& g, const __nv_bfloat16* K, int64_t k_stride, const __nv_bfloat16* V,
                                int64_t v_stride, int32_t max_tokens, const int32_t* cu_new, const int32_t* lens,
                                const int32_t* slots, const int32_t* tables, uint8_t* Kc, uint8_t* Vc, float* Ks,
                                float* Vs, float* Kbar, cudaStream_t st) {
  const AppendSide sk{K, k_stride, Kc, Ks}, sv{V, v_stride, Vc, Vs};
  auto go = [&](auto fn) { return fn(g, sk, sv, max_tokens, cu_new, lens, slots, tables, Kbar, st); };
  if (g.D == 64)
    return g.fmt == MOBA_CACHE_E4M3 ? go(launch_append_t<64, MOBA_CACHE_E4M3>) : go(launch_append_t<64, MOBA_CACHE_INT8>);
  return g.fmt == MOBA_CACHE_E4M3 ? go(launch_append_t<128, MOBA_CACHE_E4M3>) : go(launch_append_t<128, MOBA_CACHE_INT8>);
}

}  // namespace moba
