// Gated decode over a paged 8-bit KV cache: one new query per request (the newest cached token,
// at position len - 1, in block i = (len - 1) / bs) attends to its own block up to itself and to
// the top_k - 1 earlier blocks with the largest <q, Kbar[b]>, ties to the lower block:
//   z_j = scale * <q, code_j> * Ks[page(j)],  O = sum_j softmax(z)_j * code'_j * Vs[page(j)],
//   LSE = log sum_j exp(z_j).   A request of length 0 gets O = 0, LSE = -inf, no blocks.
//
//   cache_gate_kernel: scores and choice of every head of a (request, KV head), and the list of the
//                      distinct blocks that those heads chose.
//   cache_attn_kernel: each distinct block is read once for all the heads (up to 8) that chose it, in
//                      chunks of CK keys spread evenly over the warps of a persistent grid.
//   cache_merge_kernel: the chunks' partial results of a (request, head), by online softmax, always
//                      cut and added up in the same order: a row does not depend on other requests.
//
// Bound by HBM: the chosen blocks' codes, 2 D bytes a key and KV head.
#include <cudaTypedefs.h>
#include <float.h>

#include <type_traits>

#include "cache.cuh"
#include "sm100.cuh"

namespace moba {
namespace {

constexpr float kLn2C = 0.6931471805599453f;

// ------------------------------------------------------------------------------------ gate
//
// The gate's outcome is discrete, so its scores are summed in 64 bits (bf16 times fp32 is exact
// there): the choice is that of the exact scores but for ties to about 2^-50.

constexpr int kGateWarps = 8;
constexpr int kGateRows = 8;   // blocks that a warp scores at a time

// Order of scores as unsigned numbers: NaN last, -0 as +0.  No score maps to 0.
__device__ __forceinline__ uint64_t score_key(double x) {
  x = x == x ? x + 0.0 : -INFINITY;
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  return u >> 63 ? ~u : u | 1ull << 63;
}

// Sums of kN values over the warp's lanes, all at once: lane x returns the sum of v[x / (32 / kN)].
// Each of the first steps halves the values that a lane still carries.
template <int kN>
__device__ __forceinline__ double warp_sums(double (&v)[kN]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    const int half = kN * off / 32;  // values left after this step
    if (half >= 1) {
      const bool up = (lane & off) != 0;
#pragma unroll
      for (int x = 0; x < half; ++x) {
        const double give = up ? v[x] : v[x + half], keep = up ? v[x + half] : v[x];
        v[x] = keep + __shfl_xor_sync(0xffffffffu, give, off);
      }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
    }
  }
  return v[0];
}

// The best key of the lanes' best (key, block), ties to the lower block; the block that has it.
__device__ __forceinline__ int32_t warp_best(uint64_t key, int32_t b) {
  const uint32_t hi = (uint32_t)(key >> 32), top = __reduce_max_sync(0xffffffffu, hi);
  const uint32_t lo = hi == top ? (uint32_t)key : 0u, low = __reduce_max_sync(0xffffffffu, lo);
  return (int32_t)__reduce_min_sync(0xffffffffu, hi == top && lo == low ? (uint32_t)b : 0xffffffffu);
}

// The m best of up to 32 * kN keys, each lane holding kN; the q-th goes to lane 1 + q.  A round is a
// chain of comparisons in the lane and three warp reductions, so it pays to hold no more than needed:
// 11 rounds over 59 blocks took 3 us of the gate with 16 keys a lane.
template <int kN>
__device__ __forceinline__ void pick_best(const uint64_t* keys, int n, int m, int32_t& mine) {
  const int lane = threadIdx.x & 31;
  uint64_t held[kN];
#pragma unroll
  for (int x = 0; x < kN; ++x) held[x] = x * 32 + lane < n ? keys[x * 32 + lane] : 0;
  for (int q = 0; q < m; ++q) {
    uint64_t best = held[0];
    int at = 0;
#pragma unroll
    for (int x = 1; x < kN; ++x)
      if (held[x] > best) best = held[x], at = x;
    const int32_t bb = warp_best(best, at * 32 + lane);
    if (lane == 1 + q) mine = bb;
#pragma unroll
    for (int x = 0; x < kN; ++x)
      if (x * 32 + lane == bb) held[x] = 0;
  }
}

// The cluster of a (request, KV head): its CTAs share the earlier blocks' scores (kH heads and 8
// blocks a warp at a time, a lane per D / 32 dimensions), then CTA 0 chooses, a warp a head, and
// lists the distinct blocks of every 8 heads.  Bound by latency: three loads one behind the other, the
// fp64 sums and the choice take 5 us for eight requests of 63 blocks and 8 KV heads, 6 us for one of 511
// blocks on clusters of 8 (with 4, 2 and 1 CTAs the whole decode step takes 2, 6 and 12 us longer).
template <int kD, int kH>
__global__ void __launch_bounds__(kGateWarps * 32)
    cache_gate_kernel(CacheGeom g, const __nv_bfloat16* __restrict__ Q, const float* __restrict__ Kbar,
                      const int32_t* __restrict__ lens, int32_t* __restrict__ sel, CacheDecodeWork w) {
  constexpr int kDL = kD / 32;
  __shared__ int32_t s_sel[8][kMaxTopK], s_first[kGateWarps];
  const int rank = blockIdx.x, gk = blockIdx.y, s = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  launch_dependents();  // the attention kernel may be set up meanwhile
  const int32_t len = cached_len(g, lens, s);
  const int i = len > 0 ? (len - 1) / g.bs : -1;
  const int rows = gridDim.x * kGateWarps * kGateRows;
  const size_t row0 = (size_t)s * g.Hq + (size_t)gk * g.G;
  for (int h0 = 0; h0 < g.G; h0 += kH) {
    double q[kH][kDL];
#pragma unroll
    for (int h = 0; h < kH; ++h)
#pragma unroll
      for (int x = 0; x < kDL; ++x)
        q[h][x] = h0 + h < g.G ? (double)__bfloat162float(Q[(row0 + h0 + h) * kD + lane * kDL + x]) : 0.0;
    for (int b0 = (rank * kGateWarps + warp) * kGateRows; b0 < i; b0 += rows) {
      float kb[kGateRows][kDL];
#pragma unroll
      for (int r = 0; r < kGateRows; ++r) {
        const float* src = Kbar + (((size_t)s * g.MB + b0 + r) * g.Hkv + gk) * kD + lane * kDL;
        if (b0 + r < i) {
          if constexpr (kDL == 4) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(src));
            kb[r][0] = f.x, kb[r][1] = f.y, kb[r][2] = f.z, kb[r][3] = f.w;
          } else {
            const float2 f = __ldg(reinterpret_cast<const float2*>(src));
            kb[r][0] = f.x, kb[r][1] = f.y;
          }
        } else {
#pragma unroll
          for (int x = 0; x < kDL; ++x) kb[r][x] = 0.f;
        }
      }
      double v[kGateRows * kH];
#pragma unroll
      for (int r = 0; r < kGateRows; ++r)
#pragma unroll
        for (int h = 0; h < kH; ++h) {
          double acc = 0.0;
#pragma unroll
          for (int x = 0; x < kDL; ++x) acc = fma(q[h][x], (double)kb[r][x], acc);
          v[r * kH + h] = acc;
        }
      const uint64_t key = score_key(warp_sums<kGateRows * kH>(v));
      const int x = lane / (4 / kH), r = x / kH, h = x % kH;
      if (lane % (4 / kH) == 0 && b0 + r < i && h0 + h < g.G) w.score[(row0 + h0 + h) * g.MB + b0 + r] = key;
    }
  }
  if (gridDim.x > 1) cluster_barrier(); else __syncthreads();
  if (rank != 0) return;
  const int m = min(g.k - 1, max(i, 0)), HT = (g.G + 7) / 8;
  for (int ht = 0; ht < HT; ++ht) {
    const int hh = ht * 8 + warp, heads = min(8, g.G - ht * 8);
    if (hh < g.G) {
      const uint64_t* sc = w.score + (row0 + hh) * g.MB;
      int32_t mine = lane == 0 ? i : -1;  // this lane's entry of the row of sel
      if (m == 0) {
      } else if (i <= 32) {
        pick_best<1>(sc, i, m, mine);
      } else if (i <= 64) {
        pick_best<2>(sc, i, m, mine);
      } else if (i <= 128) {
        pick_best<4>(sc, i, m, mine);
      } else if (i <= 512) {
        pick_best<16>(sc, i, m, mine);
      } else {  // too many to hold: each round looks for the best behind the last one
        uint64_t last = ~0ull;
        int32_t last_b = -1;
        for (int q = 0; q < m; ++q) {
          uint64_t best = 0;
          int32_t bb = 0;
#pragma unroll 8
          for (int b = lane; b < i; b += 32) {
            const uint64_t v = sc[b];
            if ((v < last || (v == last && b > last_b)) && v > best) best = v, bb = b;
          }
          const int32_t won = warp_best(best, bb);
          last = __shfl_sync(0xffffffffu, best, won & 31);
          last_b = won;
          if (lane == 1 + q) mine = won;
        }
      }
      if (lane < g.k) {
        sel[(row0 + hh) * g.k + lane] = mine;
        s_sel[warp][lane] = mine;
      }
    }
    __syncthreads();
    // a thread for each chosen (head, slot) pair, head by head: the first pair with a block describes it
    const size_t idx = ((size_t)s * g.Hkv + gk) * HT + ht;
    CacheSeg* segs = w.segs + idx * w.max_segs;
    const int e = threadIdx.x, eh = m > 0 ? e / m : 8, ej = 1 + e - eh * m;
    bool first = eh < heads;
    CacheSeg seg{0, g.bs, {~0u, ~0u}};
    if (first) {
      seg.block = s_sel[eh][ej];
      for (int oh = 0; oh < heads; ++oh)
        for (int oj = 1; oj <= m; ++oj)
          if (s_sel[oh][oj] == seg.block) {
            if (oh < eh) first = false;  // a head chooses a block once
            const uint32_t keep = ~(0xffu << 8 * (oh & 3)), put = (uint32_t)oj << 8 * (oh & 3);
            if (oh < 4) seg.slots[0] = (seg.slots[0] & keep) | put; else seg.slots[1] = (seg.slots[1] & keep) | put;
          }
    }
    const uint32_t firsts = __ballot_sync(0xffffffffu, first);
    if (lane == 0) s_first[warp] = __popc(firsts);
    __syncthreads();
    int at = __popc(firsts & ((1u << lane) - 1)), count = 0;
#pragma unroll
    for (int x = 0; x < kGateWarps; ++x) {
      if (x < warp) at += s_first[x];
      count += s_first[x];
    }
    if (first) segs[at] = seg;
    if (threadIdx.x == 0) {  // last the own block, every head's slot 0; heads beyond the group take nothing
      CacheSeg own{i, len - max(i, 0) * g.bs, {~0u, ~0u}};
      for (int h = 0; h < heads; ++h) own.slots[h >> 2] &= ~(0xffu << 8 * (h & 3));
      if (i >= 0) segs[count] = own;
      w.units[idx] = count * w.NC + (own.keys + w.CK - 1) / w.CK;  // 0 where the request is empty
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------------------- attention
//
// Every warp works alone: it has a ring of kStages tiles of 32 keys (keys and values, by TMA) and its
// share of the units (chunks of CK keys of a distinct block).  One query for each of up to 8 heads:
// S = K Q^T and O += V^T P on mma.m16n8k16, with keys (dimensions) as the 16 rows and the heads as the
// 8 columns, so that the codes, converted in registers to fp16 (exact), are the large operand.  tcgen05
// has nothing to win here: its operands would have to be converted and written back to shared memory
// first, and these instructions are busy for 18 % of the time that the codes take to arrive.
//  - Q is scaled by a power of two for each head and held in fp16: exact down to 2^-32 of the head's
//    largest element.
//  - The sum of the softmax takes 2^(z_j - r) in fp32, with r the maximum of z_j so far, or up to 8 less.
//  - The value scale enters through the exponent, w_j = 2^((z_j - r) + (log2 Vs - u)) with u the maximum
//    of (z_j - r) + log2 Vs so far, or up to 8 less: fp16 weights are relative to the largest
//    CONTRIBUTION, however far the pages' scales lie apart (rounding 2^-11 of each weight).  log2 Vs may
//    lie anywhere from -105 (a page of zeros) to 121, so relative to that the sum would overflow or vanish.
//    z_j is rounded before r is taken off, which is then exact for the largest z_j, whatever their size.
//  - The k index of the products runs through a lane's own bytes, so both operands come out of the
//    swizzled tiles by 16-byte reads without bank conflicts; only the weights change places between
//    lanes (movmatrix).
// Measured (32/8 heads of 128, blocks of 2048, top_k 3, e4m3): 281 MB of eight 128K caches in 53 us (5.4
// TB/s, start and tail included), 2.3 GB of 64 of them at 6.2 TB/s, what a copy reaches.  At D 64 there is
// half the memory traffic for a key's conversions and softmax, and their latencies bound it: 156 MB of 37
// ragged int8 caches in 48 us, issue slots 47 % busy with three warps on a scheduler.

constexpr float kNoScore = -1e38f;  // reference before the first key: finite, below every score that counts
constexpr int kPiece = 256;     // keys whose pages a warp holds at a time (at most 16 pages)

template <int kD>
struct AttnLayout {
  static constexpr int kTile = 32;                          // keys of a stage
  static constexpr int kWarps = kD == 64 ? 12 : 8;
  static constexpr int kStages = kD == 64 ? 4 : 3;
  static constexpr int kHalf = kTile * kD;                  // codes of K (or V) of a stage
  static constexpr int kRing = kStages * 2 * kHalf;         // of a warp
  static constexpr int kBar = kWarps * kRing;              // after the rings
  static constexpr int kPrefix = kBar + kWarps * kStages * 8;
  static constexpr int kMaxPrefix = kWarps * 32 * 6;    // units are scanned in so many groups
  static constexpr int kBytes = kPrefix + (kMaxPrefix + 1) * 4 + kWarps * 4;
  static constexpr int kAlloc = kBytes + 1024;
};

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) { return __byte_perm(a, b, s); }

// Codes in the low (high) two bytes of x as a pair of fp16.
template <int kFmt>
__device__ __forceinline__ uint32_t half2_lo(uint32_t x) {
  uint32_t r;
  if constexpr (kFmt == MOBA_CACHE_E4M3) {
    asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(r) : "r"(x));
  } else {
    // byte + 128 as the low bits of 1024 + u, minus 1152
    const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&(r = prmt(x, 0x64646464u, 0x4140))),
                              __floats2half2_rn(1152.f, 1152.f));
    r = *reinterpret_cast<const uint32_t*>(&v);
  }
  return r;
}
template <int kFmt>
__device__ __forceinline__ uint32_t half2_hi(uint32_t x) {
  uint32_t r;
  if constexpr (kFmt == MOBA_CACHE_E4M3) {
    asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;}" : "=r"(r) : "r"(x));
  } else {
    const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&(r = prmt(x, 0x64646464u, 0x4342))),
                              __floats2half2_rn(1152.f, 1152.f));
    r = *reinterpret_cast<const uint32_t*>(&v);
  }
  return r;
}
// Codes as they come, made ready for half2_lo / half2_hi.
template <int kFmt>
__device__ __forceinline__ uint32_t ready(uint32_t x) {
  return kFmt == MOBA_CACHE_E4M3 ? x : x ^ 0x80808080u;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A run of at most kPiece keys of one unit (uniform over the warp).
struct Piece {
  int idx;                // entry of the work list
  int s, gk, ht;
  int32_t block;
  int chunk;              // of the block
  int key0, n, left;      // first key in the block, keys here, keys of the unit behind this piece
  uint32_t slots[2];
  bool begins;            // first piece of its unit
};

template <int kD, int kFmt>
__global__ void __launch_bounds__(AttnLayout<kD>::kWarps * 32, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, CacheGeom g,
                      const __nv_bfloat16* __restrict__ Q, const float* __restrict__ Ks, const float* __restrict__ Vs,
                      const int32_t* __restrict__ lens, const int32_t* __restrict__ tables, CacheDecodeWork w, int NI,
                      bool own_only) {
  using L = AttnLayout<kD>;
  constexpr int kStages = L::kStages, kTile = L::kTile, kMT = kTile / 16;
  constexpr int kW = kD / 16;   // k steps of K Q^T = 16-row tiles of V^T
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * L::kRing;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar) + warp * kStages;
  int32_t* prefix = reinterpret_cast<int32_t*>(smem + L::kPrefix);
  int32_t* wsum = prefix + L::kMaxPrefix + 1;

  if (lane == 0) {
    for (int q = 0; q < kStages; ++q) mbar_init(&full[q], 1);
    fence_mbar_init();
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  launch_dependents();
  wait_for_primary();  // the gate's results (at once where there is none)

  int32_t todo;       // units of this warp that are not opened yet
  int n_idx, n_unit;  // the next of them: entry and number in it,
  int n_at, n_chunk;  // which is a chunk of the entry's n_at-th block
  int4 n_seg = make_int4(0, 0, 0, 0);
  // Where no request can have an earlier block to choose, there is no gate (own_only): an entry's only
  // block follows from the length.
  const int HT = (g.G + 7) / 8;
  auto length_of = [&](int idx) { return cached_len(g, lens, idx / (HT * g.Hkv)); };
  auto own_keys = [&](int32_t len) { return len > 0 ? len - (len - 1) / g.bs * g.bs : 0; };
  auto units_in = [&](int idx) { return own_only ? (own_keys(length_of(idx)) + w.CK - 1) / w.CK : __ldcg(w.units + idx); };
  auto fetch_seg = [&]() {
    if (own_only) {
      const int32_t len = length_of(n_idx);
      const int heads = min(8, g.G - n_idx % HT * 8);
      n_seg = make_int4((len - 1) / g.bs, own_keys(len), heads >= 4 ? 0 : (int)(~0u << 8 * heads),
                        heads >= 8 ? 0 : heads <= 4 ? -1 : (int)(~0u << 8 * (heads - 4)));
    } else {
      n_seg = __ldcg(reinterpret_cast<const int4*>(w.segs + (size_t)n_idx * w.max_segs + n_at));
    }
  };
  const int64_t W = (int64_t)gridDim.x * L::kWarps, wid = (int64_t)blockIdx.x * L::kWarps + warp;
  const int per = (NI + L::kMaxPrefix - 1) / L::kMaxPrefix, groups = (NI + per - 1) / per;
  auto units_of = [&](int idx) { return per == 1 ? prefix[idx + 1] - prefix[idx] : units_in(idx); };
  // ---- which units: where there is a warp for every one that an entry can have, each warp (spread over
  // the SMs) looks at its own; else the warps take equal runs of those that there are
  const int most = w.max_segs * w.NC;
  if ((int64_t)NI * most <= W) {
    __syncwarp();  // the barriers
    const int u = warp * (int)gridDim.x + (int)blockIdx.x;
    n_idx = u / most;
    n_unit = u - n_idx * most;
    if (n_idx >= NI) return;
    n_at = n_unit / w.NC;
    n_chunk = n_unit - n_at * w.NC;
    fetch_seg();
    todo = n_unit < units_in(n_idx);
    if (todo == 0) return;
  } else {
    // units before each group of `per` entries
    constexpr int kEach = L::kMaxPrefix / (L::kWarps * 32);
    int32_t cnt[kEach], sum = 0;
#pragma unroll
    for (int x = 0; x < kEach; ++x) {
      const int gr = threadIdx.x * kEach + x;
      cnt[x] = 0;
      if (gr < groups)
        for (int y = gr * per; y < min(NI, (gr + 1) * per); ++y) cnt[x] += units_in(y);
      sum += cnt[x];
    }
    int32_t inc = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int32_t o = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += o;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int32_t before = inc - sum;
    for (int q = 0; q < warp; ++q) before += wsum[q];
#pragma unroll
    for (int x = 0; x < kEach; ++x) {
      prefix[threadIdx.x * kEach + x] = before;
      before += cnt[x];
    }
    if (threadIdx.x == L::kWarps * 32 - 1) prefix[L::kMaxPrefix] = before;
    __syncthreads();
    const int32_t total = prefix[L::kMaxPrefix];
    todo = (int32_t)((wid + 1) * total / W) - (int32_t)(wid * total / W);
    if (todo == 0) return;
    const int32_t u = (int32_t)(wid * total / W);
    int lo = 0, hi = groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= u) lo = mid; else hi = mid - 1;
    }
    n_idx = lo * per;
    n_unit = u - prefix[lo];
    for (int32_t c; n_unit >= (c = units_of(n_idx));) n_unit -= c, ++n_idx;
    n_at = n_unit / w.NC;
    n_chunk = n_unit - n_at * w.NC;
    fetch_seg();
  }

  // ---- work ahead: the description of the unit after the next piece is on its way while that piece's
  // pages are, so that none of these loads is waited for
  // The piece after p into o (p: the last one, or idx -1); false behind the warp's last one.
  auto advance = [&](const Piece& p, Piece& o) -> bool {
    if (p.left > 0) {
      o = p;
      o.key0 = p.key0 + p.n;
      o.n = min(p.left, kPiece);
      o.left = p.left - o.n;
      o.begins = false;
      return true;
    }
    if (todo == 0) return false;
    o.idx = n_idx;
    o.s = p.s, o.gk = p.gk, o.ht = p.ht;
    if (n_idx != p.idx) {
      const int sg = n_idx / HT;
      o.ht = n_idx - sg * HT;
      o.s = sg / g.Hkv;
      o.gk = sg - o.s * g.Hkv;
    }
    o.chunk = n_chunk;
    o.block = n_seg.x;
    o.slots[0] = (uint32_t)n_seg.z;
    o.slots[1] = (uint32_t)n_seg.w;
    o.key0 = o.chunk * w.CK;
    const int n = min(w.CK, n_seg.y - o.key0);
    o.n = min(n, kPiece);
    o.left = n - o.n;
    o.begins = true;
    ++n_unit;
    if (++n_chunk == w.NC) n_chunk = 0, ++n_at;
    if (--todo > 0) {
      while (n_unit >= units_of(n_idx)) n_unit = n_at = n_chunk = 0, ++n_idx;
      fetch_seg();
    }
    return true;
  };
  const int lps = 31 - __clz(g.ps);
  // Keys of a piece are counted from the start of its first page (offset_of keys before its own first).
  auto offset_of = [&](const Piece& p) { return p.key0 & (g.ps - 1); };
  // The lane-th page of a piece (-1: none), not yet looked at.
  auto pages_of = [&](const Piece& p) -> int32_t {
    return lane << lps < offset_of(p) + p.n ? __ldg(tables + (size_t)p.s * g.MP + ((p.block * g.bs + p.key0) >> lps) + lane) : -1;
  };
  // Bad pages become -1 and are reported; the others' scales are fetched.  True if there are any.
  auto look_at = [&](const Piece& p, int32_t& page, float& ks, float& vs) -> bool {
    const bool bad = lane << lps < offset_of(p) + p.n && !page_ok(g, page);
    ks = 0.f, vs = 1.f;
    if (page_ok(g, page)) {
      ks = __ldg(Ks + (size_t)page * g.Hkv + p.gk);
      vs = __ldg(Vs + (size_t)page * g.Hkv + p.gk);
    } else {
      if (bad) atomicOr(g.err, kErrBadPage);
      page = -1;
    }
    return __any_sync(0xffffffffu, bad);
  };
  const int box = min(g.ps, kTile);
  int wr = 0;  // stage that the next copy goes to
  auto copy_box = [&](const Piece& p, int32_t page, int key, uint8_t* dst) {
    const int row = (p.key0 + key) & (g.ps - 1), slab = page * g.Hkv + p.gk;
    tma_load_3d(dst, &tmK, &full[wr], 0, row, slab);
    tma_load_3d(dst + L::kHalf, &tmV, &full[wr], 0, row, slab);
  };
  auto issue = [&](const Piece& p, int32_t page, int tile) {
    uint8_t* dst = ring + wr * 2 * L::kHalf;
    const int key = tile * kTile;
    const int32_t p0 = __shfl_sync(0xffffffffu, page, (offset_of(p) + key) >> lps & 31);
    if (box == kTile) {  // a tile lies in one page
      if (lane == 0) {
        if (p0 >= 0) {
          mbar_expect_tx(&full[wr], 2 * kTile * kD);
          copy_box(p, p0, key, dst);
        } else {
          mbar_arrive(&full[wr]);
        }
      }
    } else {             // pages of 16: two boxes
      int32_t p1 = __shfl_sync(0xffffffffu, page, (offset_of(p) + key + box) >> lps & 31);
      if (key + box >= p.n) p1 = -1;
      if (lane == 0) {
        const int boxes = (p0 >= 0) + (p1 >= 0);
        if (boxes) mbar_expect_tx(&full[wr], boxes * 2 * box * kD); else mbar_arrive(&full[wr]);
        if (p0 >= 0) copy_box(p, p0, key, dst);
        if (p1 >= 0) copy_box(p, p1, key + box, dst + box * kD);
      }
    }
    if (++wr == kStages) wr = 0;
  };
  auto tiles_of = [](const Piece& p) { return (p.n + kTile - 1) / kTile; };

  Piece cur, nxt;
  nxt.idx = -1;
  nxt.left = 0;
  advance(nxt, cur);
  int32_t page_c = pages_of(cur), page_n = -1;
  float ks, vs, ks_n = 0.f, vs_n = 1.f;
  bool odd = look_at(cur, page_c, ks, vs), odd_n = false;
  int issued_c = 0, issued_n = 0, flying = 0;
  for (; issued_c < min(tiles_of(cur), kStages); ++issued_c, ++flying) issue(cur, page_c, issued_c);
  bool more = advance(cur, nxt), looked = false, ok = true;
  if (more) page_n = pages_of(nxt);
  int rd = 0;
  uint32_t parity = 0;

  uint32_t qb[kW][2];
  float sf[2];                  // of heads 2t, 2t + 1: softmax scale over Q's power of two, log2 units
  int q_idx = -1;
  float o[kW][4], l[2];         // l: sum of the softmax
  float r[2], u[2];             // references (below)
  bool fresh = true;            // nothing is added up yet

  while (true) {
    if (cur.begins) {
      if (q_idx != cur.idx) {
        // Q of head gq, dimensions [t * kD / 4, (t + 1) * kD / 4), as the products' second operand
        q_idx = cur.idx;
        const int h = cur.ht * 8 + gq;
        const bool live = h < g.G;
        const uint2* src = reinterpret_cast<const uint2*>(Q + ((size_t)cur.s * g.Hq + (size_t)cur.gk * g.G + h) * kD) + t * kW;
        uint2 raw[kW];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < kW; ++j) {
          raw[j] = live ? __ldg(src + j) : make_uint2(0, 0);
          top = max(max(top, max(raw[j].x & 0x7fffu, (raw[j].x >> 16) & 0x7fffu)),
                    max(raw[j].y & 0x7fffu, (raw[j].y >> 16) & 0x7fffu));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // largest element to [2^14, 2^15); an infinity or NaN stays what it is
        const int ex = (int)(top >> 7), sh = ex == 255 ? 0 : min(141 - ex, 126);
        const float f = __int_as_float((127 + sh) << 23);
#pragma unroll
        for (int j = 0; j < kW; ++j) {
          const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[j].x));
          const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[j].y));
          qb[j][0] = pack_half2(lo.x * f, lo.y * f);
          qb[j][1] = pack_half2(hi.x * f, hi.y * f);
        }
        const float mine = g.scale_log2 * __int_as_float((127 - sh) << 23);
        sf[0] = __shfl_sync(0xffffffffu, mine, 8 * t);      // a lane of head 2t
        sf[1] = __shfl_sync(0xffffffffu, mine, 8 * t + 4);
      }
#pragma unroll
      for (int j = 0; j < kW; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[j][x] = 0.f;
      r[0] = r[1] = kNoScore;
      u[0] = u[1] = l[0] = l[1] = 0.f;
      fresh = true;
    }
    const float lvs = log2f(vs);
    const int tiles = tiles_of(cur);
    // One tile.  kOdd: some of its keys do not count (behind the newest token, or on a bad page).
    auto take = [&](auto odd_tile, int tile) {
      constexpr bool kOdd = decltype(odd_tile)::value;
      const uint8_t* kst = ring + rd * 2 * L::kHalf;
      const uint8_t* vst = kst + L::kHalf;
      float c[kMT][4];
      // ---- S = K Q^T: keys gq and gq + 8 of each 16, heads 2t and 2t + 1
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        uint32_t kw[2][kW];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int r = mt * 16 + x * 8 + gq;
          if constexpr (kD == 128) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4 v = *reinterpret_cast<const uint4*>(kst + r * 128 + (((2 * t + h) ^ (r & 7)) << 4));
              kw[x][4 * h] = v.x, kw[x][4 * h + 1] = v.y, kw[x][4 * h + 2] = v.z, kw[x][4 * h + 3] = v.w;
            }
          } else {
            const uint4 v = *reinterpret_cast<const uint4*>(kst + r * 64 + ((t ^ ((r >> 1) & 3)) << 4));
            kw[x][0] = v.x, kw[x][1] = v.y, kw[x][2] = v.z, kw[x][3] = v.w;
          }
        }
        float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kW; ++j) {
          const uint32_t a = ready<kFmt>(kw[0][j]), b = ready<kFmt>(kw[1][j]);
          mma_f16(j & 1 ? c1 : c0, half2_lo<kFmt>(a), half2_lo<kFmt>(b), half2_hi<kFmt>(a), half2_hi<kFmt>(b), qb[j][0],
                  qb[j][1]);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) c[mt][x] = c0[x] + c1[x];
      }
      // the values are fetched ahead of their use
      uint32_t v[kMT][4][kW / 2];  // keys 2t, 2t + 1, 2t + 8, 2t + 9 of each 16
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = mt * 16 + 2 * t + (x & 1) + 8 * (x >> 1);
          if constexpr (kD == 128) {
            const uint4 u = *reinterpret_cast<const uint4*>(vst + r * 128 + ((gq ^ (r & 7)) << 4));
            v[mt][x][0] = u.x, v[mt][x][1] = u.y, v[mt][x][2] = u.z, v[mt][x][3] = u.w;
          } else {
            const uint2 u = *reinterpret_cast<const uint2*>(vst + r * 64 + (((gq >> 1) ^ ((r >> 1) & 3)) << 4) + (gq & 1) * 8);
            v[mt][x][0] = u.x, v[mt][x][1] = u.y;
          }
        }
      // ---- online softmax: z = c * f, in place of c
      int live[kMT] = {};  // keys of each 16 that count
      float f0, f1, lv[kMT], zx0 = -INFINITY, zx1 = -INFINITY;
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        const int key = tile * kTile + mt * 16, pi = (offset_of(cur) + key) >> lps & 31;
        if (mt > 0 && box == kTile) {  // the same page
          lv[mt] = lv[0];
        } else {
          const float k1 = __shfl_sync(0xffffffffu, ks, pi);
          lv[mt] = __shfl_sync(0xffffffffu, lvs, pi);
          f0 = k1 * sf[0];
          f1 = k1 * sf[1];
        }
        if constexpr (kOdd) {
          const int32_t pg = __shfl_sync(0xffffffffu, page_c, pi);
          live[mt] = pg >= 0 ? min(16, cur.n - key) : 0;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          c[mt][x] = __fmul_rn(c[mt][x], x & 1 ? f1 : f0);
          if (kOdd && (x < 2 ? gq : gq + 8) >= live[mt]) c[mt][x] = -INFINITY;  // masked
        }
        zx0 = max3(zx0, c[mt][0], c[mt][2]);
        zx1 = max3(zx1, c[mt][1], c[mt][3]);
      }
      // r and u are maxima of earlier keys, not the largest so far: weights up to 2^kSlack are as good in fp16
      // and fp32, and the exact maxima over the lanes are only needed when a key may leave that range
      constexpr float kSlack = 8.f;
      const float lv_max = kMT > 1 && box != kTile ? fmaxf(lv[0], lv[kMT - 1]) : lv[0];
      if (__any_sync(0xffffffffu, zx0 - r[0] > fminf(u[0] - lv_max, 0.f) + kSlack ||
                                      zx1 - r[1] > fminf(u[1] - lv_max, 0.f) + kSlack)) {
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) {
          zx0 = fmaxf(zx0, __shfl_xor_sync(0xffffffffu, zx0, off));
          zx1 = fmaxf(zx1, __shfl_xor_sync(0xffffffffu, zx1, off));
        }
        zx0 = fmaxf(zx0, r[0]);
        zx1 = fmaxf(zx1, r[1]);
        float ux0 = -INFINITY, ux1 = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
          ux0 = fmaxf(ux0, fmaxf(c[mt][0] - zx0, c[mt][2] - zx0) + lv[mt]);
          ux1 = fmaxf(ux1, fmaxf(c[mt][1] - zx1, c[mt][3] - zx1) + lv[mt]);
        }
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) {
          ux0 = fmaxf(ux0, __shfl_xor_sync(0xffffffffu, ux0, off));
          ux1 = fmaxf(ux1, __shfl_xor_sync(0xffffffffu, ux1, off));
        }
        const float d0 = r[0] - zx0, d1 = r[1] - zx1;  // the old references under the new r
        ux0 = fmaxf(ux0, d0 + u[0]);
        ux1 = fmaxf(ux1, d1 + u[1]);
        if (!fresh) {
          const float a0 = ex2(d0 + u[0] - ux0), a1 = ex2(d1 + u[1] - ux1);
          l[0] *= ex2(d0);
          l[1] *= ex2(d1);
#pragma unroll
          for (int j = 0; j < kW; ++j) {
            o[j][0] *= a0;
            o[j][1] *= a1;
            o[j][2] *= a0;
            o[j][3] *= a1;
          }
        }
        r[0] = zx0;
        r[1] = zx1;
        u[0] = ux0;
        u[1] = ux1;
      }
      fresh = false;
      // ---- O += V^T P: dimensions of group gq, heads 2t and 2t + 1
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
        for (int x = 0; x < 4; ++x) c[mt][x] -= r[x & 1];
        l[0] += ex2(c[mt][0]) + ex2(c[mt][2]);
        l[1] += ex2(c[mt][1]) + ex2(c[mt][3]);
        const float w0 = lv[mt] - u[0], w1 = lv[mt] - u[1];
        const uint32_t p0 = transpose8(pack_half2(ex2(c[mt][0] + w0), ex2(c[mt][1] + w1)));
        const uint32_t p1 = transpose8(pack_half2(ex2(c[mt][2] + w0), ex2(c[mt][3] + w1)));
        if constexpr (kOdd) {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (2 * t + (x & 1) + 8 * (x >> 1) >= live[mt]) {  // whatever stands there must not meet a weight of 0
#pragma unroll
              for (int j = 0; j < kW / 2; ++j) v[mt][x][j] = 0;
            }
        }
#pragma unroll
        for (int j = 0; j < kW / 2; ++j) {
          const uint32_t a = ready<kFmt>(v[mt][0][j]), b = ready<kFmt>(v[mt][1][j]);
          const uint32_t d = ready<kFmt>(v[mt][2][j]), e = ready<kFmt>(v[mt][3][j]);
          const uint32_t x0 = prmt(a, b, 0x5140), x1 = prmt(a, b, 0x7362), y0 = prmt(d, e, 0x5140), y1 = prmt(d, e, 0x7362);
          mma_f16(o[2 * j], half2_lo<kFmt>(x0), half2_hi<kFmt>(x0), half2_lo<kFmt>(y0), half2_hi<kFmt>(y0), p0, p1);
          mma_f16(o[2 * j + 1], half2_lo<kFmt>(x1), half2_hi<kFmt>(x1), half2_lo<kFmt>(y1), half2_hi<kFmt>(y1), p0, p1);
        }
      }
    };
    for (int tile = 0; tile < tiles; ++tile) {
      ok = mbar_wait_warp(&full[rd], parity, g.err);
      if (!ok) break;
      if (odd || (tile + 1) * kTile > cur.n) take(std::true_type{}, tile); else take(std::false_type{}, tile);
      __syncwarp();  // the stage is read
      if (++rd == kStages) rd = 0, parity ^= 1;
      --flying;
      if (issued_c < tiles) issue(cur, page_c, issued_c++), ++flying;
      else if (more) {
        if (!looked) odd_n = look_at(nxt, page_n, ks_n, vs_n), looked = true;
        if (issued_n < tiles_of(nxt)) issue(nxt, page_n, issued_n++), ++flying;
      }
    }
    if (!ok) break;
    if (cur.left == 0) {
      // ---- partial result of the unit
      float ls[2] = {l[0], l[1]};
#pragma unroll
      for (int off = 4; off <= 16; off <<= 1) {
        ls[0] += __shfl_xor_sync(0xffffffffu, ls[0], off);
        ls[1] += __shfl_xor_sync(0xffffffffu, ls[1], off);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 2 * t + e;
        const uint32_t slot = ((t < 2 ? cur.slots[0] : cur.slots[1]) >> 8 * (h & 3)) & 0xffu;
        if (slot != 0xffu) {
          const size_t row = (size_t)cur.s * g.Hq + (size_t)cur.gk * g.G + cur.ht * 8 + h;
          const size_t part = (row * g.k + slot) * w.NC + cur.chunk;
          float4* dst = reinterpret_cast<float4*>(w.part_o + part * kD + gq * (kD / 8));
#pragma unroll
          for (int j = 0; j < kW; j += 2) dst[j / 2] = make_float4(o[j][e], o[j][2 + e], o[j + 1][e], o[j + 1][2 + e]);
          if (gq == 0) w.part_ml[part] = make_float4(r[e], u[e], ls[e], 0.f);
        }
      }
    }
    if (!more) break;
    if (!looked) odd_n = look_at(nxt, page_n, ks_n, vs_n);
    cur = nxt;
    odd = odd_n;
    page_c = page_n;
    ks = ks_n;
    vs = vs_n;
    issued_c = issued_n;
    issued_n = 0;
    for (; flying < kStages && issued_c < tiles_of(cur); ++flying) issue(cur, page_c, issued_c++);
    more = advance(cur, nxt);
    looked = false;
    if (more) page_n = pages_of(nxt);
  }
  if (!ok)  // a wait gave up: leave no copy behind
    for (; flying > 0; --flying) {
      mbar_wait_warp(&full[rd], parity, g.err);
      if (++rd == kStages) rd = 0, parity ^= 1;
    }
}

// Partial results of a (request, head), merged by online softmax (log2 units) by kWarps warps: warp x
// takes every kWarps-th part.  Bound by the latency of two rounds of loads: about 4 us.
constexpr int kMergeWarps = 8;  // of a CTA
constexpr int kMergeRows = 8;   // partial rows of a warp on their way at a time

template <int kD, int kWarps>
__global__ void __launch_bounds__(kMergeWarps * 32)
    cache_merge_kernel(CacheGeom g, const int32_t* __restrict__ lens, CacheDecodeWork w, bool own_only,
                       int32_t* __restrict__ sel, __nv_bfloat16* __restrict__ O, float* __restrict__ LSE) {
  constexpr int kDL = kD / 32;
  __shared__ float s_acc[kMergeWarps][kD], s_l[kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % kWarps;
  const size_t row = (size_t)blockIdx.x * (kMergeWarps / kWarps) + warp / kWarps;
  const bool live = row < (size_t)g.B * g.Hq;
  // the step's first kernel starts when all earlier work has ended, so the lengths may be read before the wait
  const int32_t len = live ? cached_len(g, lens, (int)(row / g.Hq)) : 0;
  const int own = len > 0 ? (len - 1) / g.bs : 0, own_chunks = (len - own * g.bs + w.CK - 1) / w.CK;
  const int n = own_chunks + min(g.k - 1, own) * w.NC;  // slots are filled from the front
  const int mine = n > part ? (n - part + kWarps - 1) / kWarps : 0;  // parts of this warp
  const float4* ml = w.part_ml + row * g.k * w.NC;
  const float* po = w.part_o + row * g.k * w.NC * kD + lane * kDL;
  auto at = [&](int x) { return x < own_chunks ? x : w.NC + (x - own_chunks); };
  float f[kMergeRows][kDL];
  auto fetch = [&](int x1) {  // this warp's rows [x1, x1 + kMergeRows)
#pragma unroll
    for (int x = 0; x < kMergeRows; ++x)
      if (x1 + x < mine) {
        const float* src = po + (size_t)at(part + (x1 + x) * kWarps) * kD;
        if constexpr (kDL == 4) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
          f[x][0] = v.x, f[x][1] = v.y, f[x][2] = v.z, f[x][3] = v.w;
        } else {
          const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
          f[x][0] = v.x, f[x][1] = v.y;
        }
      }
  };
  wait_for_primary();
  fetch(0);  // while the weights are found
  // R: largest r; U: largest (r - R) + u, the reference of acc.  Up to 64 parts are read once for both.
  float4 held[2];
#pragma unroll
  for (int x = 0; x < 2; ++x)
    held[x] = lane + 32 * x < n ? __ldcg(ml + at(lane + 32 * x)) : make_float4(kNoScore, 0.f, 0.f, 0.f);
  float R = fmaxf(held[0].x, held[1].x);
  for (int x = lane + 64; x < n; x += 32) R = fmaxf(R, __ldcg(ml + at(x)).x);
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) R = fmaxf(R, __shfl_xor_sync(0xffffffffu, R, off));
  float U = fmaxf((held[0].x - R) + held[0].y, (held[1].x - R) + held[1].y);
  for (int x = lane + 64; x < n; x += 32) {
    const float4 v = __ldcg(ml + at(x));
    U = fmaxf(U, (v.x - R) + v.y);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) U = fmaxf(U, __shfl_xor_sync(0xffffffffu, U, off));
  float L = 0.f, acc[kDL];
#pragma unroll
  for (int d = 0; d < kDL; ++d) acc[d] = 0.f;
  for (int x0 = 0; x0 < mine; x0 += 32) {
    float wt = 0.f;
    if (x0 + lane < mine) {
      const float4 v = __ldcg(ml + at(part + (x0 + lane) * kWarps));
      wt = ex2((v.x - R) + v.y - U);
      L = fmaf(v.z, ex2(v.x - R), L);
    }
    for (int x1 = x0; x1 < min(mine, x0 + 32); x1 += kMergeRows) {
      if (x1 > 0) fetch(x1);
#pragma unroll
      for (int x = 0; x < kMergeRows; ++x) {
        const float wx = __shfl_sync(0xffffffffu, wt, (x1 + x) & 31);
        if (x1 + x < mine)
#pragma unroll
          for (int d = 0; d < kDL; ++d) acc[d] = fmaf(wx, f[x][d], acc[d]);
      }
    }
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
  if constexpr (kWarps > 1) {
    if (lane == 0) s_l[warp] = L;
#pragma unroll
    for (int d = 0; d < kDL; ++d) s_acc[warp][lane * kDL + d] = acc[d];
    __syncthreads();
    if (part > 0) return;
#pragma unroll
    for (int x = 1; x < kWarps; ++x) {
      L += s_l[warp + x];
#pragma unroll
      for (int d = 0; d < kDL; ++d) acc[d] += s_acc[warp + x][lane * kDL + d];
    }
  }
  if (!live) return;
  const float inv = L == 0.f ? 0.f : 1.f / L;  // 0: no key at all
  const float up = ex2(0.5f * U);  // root of what the weights of acc carry of the value scales (up to 2^129)
#pragma unroll
  for (int d = 0; d < kDL; d += 2)
    *reinterpret_cast<__nv_bfloat162*>(O + row * kD + lane * kDL + d) =
        __floats2bfloat162_rn(acc[d] * inv * up * up, acc[d + 1] * inv * up * up);
  if (lane == 0) LSE[row] = L == 0.f ? -INFINITY : (R + log2f(L)) * kLn2C;
  if (own_only && lane < g.k) sel[row * g.k + lane] = lane == 0 && len > 0 ? own : -1;  // there was no gate
}

// ---------------------------------------------------------------------------------- launch

// A driver entry point, looked up once.
template <typename F>
F driver_entry(const char* name) {
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  const bool ok = cudaGetDriverEntryPoint(name, &p, cudaEnableDefault, &q) == cudaSuccess && q == cudaDriverEntryPointSuccess;
  return ok ? reinterpret_cast<F>(p) : nullptr;
}

// Codes [P * Hkv, ps, D] as dims (d, row, slab); boxes of D x min(ps, tile) x 1, swizzled over the
// whole row (128 or 64 bytes).  The two maps differ in their address alone.
cudaError_t make_codes_maps(CUtensorMap* k, CUtensorMap* v, const void* Kc, const void* Vc, const CacheGeom& g, int tile) {
  static const auto encode = driver_entry<PFN_cuTensorMapEncodeTiled_v12000>("cuTensorMapEncodeTiled");
  static const auto replace = driver_entry<PFN_cuTensorMapReplaceAddress_v12000>("cuTensorMapReplaceAddress");
  if (!encode || !replace) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)g.D, (cuuint64_t)g.ps, (cuuint64_t)g.P * g.Hkv};
  const cuuint64_t strides[2] = {(cuuint64_t)g.D, (cuuint64_t)g.D * g.ps};
  const cuuint32_t box[3] = {(cuuint32_t)g.D, (cuuint32_t)(g.ps < tile ? g.ps : tile), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  if (encode(k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(Kc), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, g.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  *v = *k;
  return replace(v, const_cast<void*>(Vc)) == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int kD, int kH>
cudaError_t launch_gate(const CacheGeom& g, const __nv_bfloat16* Q, const float* Kbar, const int32_t* lens,
                        int32_t* sel, const CacheDecodeWork& w, cudaStream_t st) {
  // CTAs of a cluster share the candidates, 64 blocks each at a time
  int c = 1;
  while (c < 8 && c * kGateWarps * kGateRows < g.MB - 1) c *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)c, (unsigned)g.Hkv, (unsigned)g.B);
  cfg.blockDim = dim3(kGateWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)c;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_gate_kernel<kD, kH>, g, Q, Kbar, lens, sel, w);
}

// Launches a kernel; a dependent one's CTAs may start while the kernel before it runs, and wait for its
// results there.
template <typename... P, typename... A>
cudaError_t launch_kernel(bool dependent, dim3 grid, int threads, size_t smem, cudaStream_t st, void (*kernel)(P...),
                          A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

template <int kD, int kFmt>
cudaError_t launch_decode_t(const CacheGeom& g, const __nv_bfloat16* Q, const uint8_t* Kc, const uint8_t* Vc,
                            const float* Ks, const float* Vs, const float* Kbar, const int32_t* lens,
                            const int32_t* tables, int32_t* sel, const CacheDecodeWork& w, __nv_bfloat16* O,
                            float* LSE, int sms, cudaStream_t st) {
  const bool own_only = g.MB == 1 || g.k == 1;
  cudaError_t e = own_only   ? cudaSuccess
                  : g.G == 1 ? launch_gate<kD, 1>(g, Q, Kbar, lens, sel, w, st)
                  : g.G == 2 ? launch_gate<kD, 2>(g, Q, Kbar, lens, sel, w, st)
                             : launch_gate<kD, 4>(g, Q, Kbar, lens, sel, w, st);
  if (e != cudaSuccess) return e;
  CUtensorMap tk, tv;
  if ((e = make_codes_maps(&tk, &tv, Kc, Vc, g, AttnLayout<kD>::kTile)) != cudaSuccess) return e;
  if ((e = allow_smem<cache_attn_kernel<kD, kFmt>>(AttnLayout<kD>::kAlloc)) != cudaSuccess) return e;
  e = launch_kernel(!own_only, dim3((unsigned)sms), AttnLayout<kD>::kWarps * 32, AttnLayout<kD>::kAlloc, st,
                    cache_attn_kernel<kD, kFmt>, tk, tv, g, Q, Ks, Vs, lens, tables, w, g.B * g.Hkv * ((g.G + 7) / 8),
                    own_only);
  if (e != cudaSuccess) return e;
  // All warps of a CTA on one row while every row's are on the GPU at once, else a warp for each: 512 rows of
  // 8 parts 45.7 us for the step with 8 warps, 47.7 with one; 4096 rows of 9 parts 140 and 127.
  const int64_t rows = (int64_t)g.B * g.Hq;
  if (rows * kMergeWarps <= sms * 64)
    return launch_kernel(true, dim3((unsigned)rows), kMergeWarps * 32, 0, st, cache_merge_kernel<kD, kMergeWarps>, g, lens,
                         w, own_only, sel, O, LSE);
  return launch_kernel(true, dim3((unsigned)((rows + kMergeWarps - 1) / kMergeWarps)), kMergeWarps * 32, 0, st,
                       cache_merge_kernel<kD, 1>, g, lens, w, own_only, sel, O, LSE);
}

}  // namespace

// Keys of a unit, a power of two from 32 (a tile) on: the longest that leaves enough units for each warp,
// as a unit costs a warp about as much as 40 keys.  Units are counted as if half of a group's heads shared
// their choices.  With more blocks than warps, 3 units a warp keep their shares even: 64 caches of 128K
// take 385 us at 1024 keys, 403 at 256 (32/8 heads of 128, top_k 3 of blocks of 2048); 37 ragged ones of
// 64 dimensions 51 us at 256, 58 at 512 (blocks of 512).  With fewer, a bit more than half as many units
// as warps have enough copies on their way to fill the memory: eight caches of 128K take 57 us at 1024
// keys (what the rule takes), 67 at 256; one of 1M 22.5 us at 128 (the rule), 21.6 at 256, 28 at 512.  The
// work space's size follows from this on the host, without a device, so the SMs are those of a B200.
int cache_chunk_keys(const CacheGeom& g) {
  const int64_t entries = (int64_t)g.B * g.Hkv * ((g.G + 7) / 8);
  const int64_t past = (int64_t)(g.k - 1) * (1 + (g.G < 8 ? g.G : 8)) / 2;
  const int64_t blocks = entries * (1 + (past < g.MB - 1 ? past : g.MB - 1));
  const int64_t warps = 148 * (g.D == 64 ? AttnLayout<64>::kWarps : AttnLayout<128>::kWarps);
  const int64_t want = blocks >= warps ? 3 * warps : warps * 3 / 5;
  int ck = 8192;
  while (ck > 32 && (ck / 2 >= g.bs || blocks * ((g.bs + ck - 1) / ck) < want)) ck /= 2;
  return ck;
}

cudaError_t launch_cache_decode(const CacheGeom& g, const __nv_bfloat16* Q, const uint8_t* Kc, const uint8_t* Vc,
                                const float* Ks, const float* Vs, const float* Kbar, const int32_t* lens,
                                const int32_t* tables, int32_t* sel, const CacheDecodeWork& w, __nv_bfloat16* O,
                                float* LSE, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  auto go = [&](auto fn) { return fn(g, Q, Kc, Vc, Ks, Vs, Kbar, lens, tables, sel, w, O, LSE, sms, st); };
  if (g.D == 64)
    return g.fmt == MOBA_CACHE_E4M3 ? go(launch_decode_t<64, MOBA_CACHE_E4M3>) : go(launch_decode_t<64, MOBA_CACHE_INT8>);
  return g.fmt == MOBA_CACHE_E4M3 ? go(launch_decode_t<128, MOBA_CACHE_E4M3>) : go(launch_decode_t<128, MOBA_CACHE_INT8>);
}

}  // namespace moba
