// C ABI of the paged 8-bit KV cache: argument checks, work space and launches.  As in
// moba_api.cu, nothing here allocates or synchronises.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "api_common.cuh"
#include "cache.cuh"

namespace {

using moba::api::cuda_error;

moba_status fail(moba_status st, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return moba::api::fail_with(st, msg);
}

#define MOBA_TRY(x)               \
  do {                            \
    moba_status _s = (x);         \
    if (_s != MOBA_OK) return _s; \
  } while (0)

constexpr int64_t kI32Max = 2147483647LL;

// Distinct blocks that a tile of 8 heads can choose.
int cache_max_segs(const moba::CacheGeom& g) {
  const int past = (g.G < 8 ? g.G : 8) * (g.k - 1);
  return 1 + (past < g.MB - 1 ? past : g.MB - 1);
}

// Validate the parameters and derive the kernels' geometry (host only).
moba_status make_cache_geom(const moba_cache_params* p, moba::CacheGeom* g) {
  if (!p) return fail(MOBA_ERR_INVALID_ARG, "params is NULL");
  if (p->max_seqs < 1) return fail(MOBA_ERR_INVALID_ARG, "max_seqs must be >= 1 (got %d)", p->max_seqs);
  if (p->max_seqs > 65535) return fail(MOBA_ERR_UNSUPPORTED, "max_seqs must be <= 65535 (got %d)", p->max_seqs);
  if (p->max_seqlen < 1) return fail(MOBA_ERR_INVALID_ARG, "max_seqlen must be >= 1 (got %d)", p->max_seqlen);
  if (p->max_seqlen > (1 << 30)) return fail(MOBA_ERR_UNSUPPORTED, "max_seqlen must be <= 2^30 (got %d)", p->max_seqlen);
  if (p->num_pages < 1) return fail(MOBA_ERR_INVALID_ARG, "num_pages must be >= 1 (got %d)", p->num_pages);
  if (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128)
    return fail(MOBA_ERR_UNSUPPORTED, "page_size must be 16, 32, 64 or 128 (got %d)", p->page_size);
  if ((int64_t)p->num_pages * p->page_size > kI32Max)
    return fail(MOBA_ERR_UNSUPPORTED, "num_pages * page_size exceeds 2^31-1");
  if (p->num_q_heads < 1 || p->num_kv_heads < 1 || p->num_q_heads % p->num_kv_heads)
    return fail(MOBA_ERR_INVALID_ARG, "num_q_heads (%d) must be a positive multiple of num_kv_heads (%d)",
                p->num_q_heads, p->num_kv_heads);
  if (p->head_dim != 64 && p->head_dim != 128)
    return fail(MOBA_ERR_UNSUPPORTED, "head_dim must be 64 or 128 (got %d)", p->head_dim);
  if ((int64_t)p->num_kv_heads * p->head_dim > 16384)
    return fail(MOBA_ERR_UNSUPPORTED, "num_kv_heads * head_dim must be <= 16384");
  if (p->num_q_heads > 65535) return fail(MOBA_ERR_UNSUPPORTED, "num_q_heads must be <= 65535 (got %d)", p->num_q_heads);
  if (p->block_size < 128 || p->block_size % 128 || p->block_size > 8192)
    return fail(MOBA_ERR_UNSUPPORTED, "block_size must be a multiple of 128 in [128, 8192] (got %d)", p->block_size);
  if (p->top_k < 1 || p->top_k > moba::kMaxTopK)
    return fail(MOBA_ERR_UNSUPPORTED, "top_k must be in [1, %d] (got %d)", moba::kMaxTopK, p->top_k);
  if (p->format != MOBA_CACHE_E4M3 && p->format != MOBA_CACHE_INT8)
    return fail(MOBA_ERR_UNSUPPORTED, "format must be MOBA_CACHE_E4M3 or MOBA_CACHE_INT8 (got %d)", p->format);
  const int64_t MP = ((int64_t)p->max_seqlen + p->page_size - 1) / p->page_size;
  const int64_t MB = ((int64_t)p->max_seqlen + p->block_size - 1) / p->block_size;
  if (MB > 16384) return fail(MOBA_ERR_UNSUPPORTED, "more than 16384 blocks in one request");
  if ((int64_t)p->num_pages * p->num_kv_heads > kI32Max)
    return fail(MOBA_ERR_UNSUPPORTED, "num_pages * num_kv_heads exceeds 2^31-1");
  if (MP * p->max_seqs > kI32Max) return fail(MOBA_ERR_UNSUPPORTED, "max_seqs * pages of a request exceeds 2^31-1");
  if ((int64_t)p->max_seqs * p->num_q_heads * p->top_k > kI32Max)
    return fail(MOBA_ERR_UNSUPPORTED, "max_seqs * num_q_heads * top_k exceeds 2^31-1");
  g->B = p->max_seqs;
  g->max_len = p->max_seqlen;
  g->MP = (int32_t)MP;
  g->MB = (int32_t)MB;
  g->P = p->num_pages;
  g->ps = p->page_size;
  g->Hq = p->num_q_heads;
  g->Hkv = p->num_kv_heads;
  g->G = p->num_q_heads / p->num_kv_heads;
  g->D = p->head_dim;
  g->bs = p->block_size;
  g->k = p->top_k;
  g->fmt = p->format;
  g->scale = p->softmax_scale > 0.f ? p->softmax_scale : 1.0f / sqrtf((float)p->head_dim);
  g->scale_log2 = g->scale * 1.4426950408889634f;
  g->err = nullptr;
  const int ck = moba::cache_chunk_keys(*g);
  if ((int64_t)cache_max_segs(*g) * ((p->block_size + ck - 1) / ck) * p->max_seqs * p->num_kv_heads * ((g->G + 7) / 8) > kI32Max)
    return fail(MOBA_ERR_UNSUPPORTED, "more than 2^31-1 chunks of chosen blocks");
  return MOBA_OK;
}

moba_status check_ptr(const void* ptr, const char* name, uintptr_t align = 16) {
  if (!ptr) return fail(MOBA_ERR_INVALID_ARG, "%s is NULL", name);
  if ((uintptr_t)ptr & (align - 1)) return fail(MOBA_ERR_ALIGNMENT, "%s is not %d-byte aligned", name, (int)align);
  return MOBA_OK;
}

moba::CacheDecodeWork carve_cache_decode(const moba::CacheGeom& g, char* base) {
  size_t off = 0;
  auto take = [&](size_t bytes) -> char* {
    char* ptr = base ? base + off : nullptr;
    off += (bytes + 255) & ~(size_t)255;
    return ptr;
  };
  moba::CacheDecodeWork w;
  w.CK = moba::cache_chunk_keys(g);
  w.NC = (g.bs + w.CK - 1) / w.CK;
  w.max_segs = cache_max_segs(g);
  const size_t rows = (size_t)g.B * g.Hq, parts = rows * g.k * w.NC;
  const size_t entries = (size_t)g.B * g.Hkv * ((g.G + 7) / 8);
  w.score = (uint64_t*)take(rows * g.MB * sizeof(uint64_t));
  w.segs = (moba::CacheSeg*)take(entries * w.max_segs * sizeof(moba::CacheSeg));
  w.units = (int32_t*)take(entries * sizeof(int32_t));
  w.part_o = (float*)take(parts * g.D * sizeof(float));
  w.part_ml = (float4*)take(parts * sizeof(float4));
  w.sel = (int32_t*)take(rows * g.k * sizeof(int32_t));
  w.bytes = off;
  return w;
}

}  // namespace

extern "C" {

moba_status moba_cache_tables(const moba_cache_params* p, const int32_t* add, const int32_t* lens, int32_t* tables,
                              int32_t* free_pages, const int32_t* free_state, int32_t* lens_out,
                              int32_t* free_state_out, int32_t* cu_new, int32_t* slots, int32_t max_tokens,
                              int32_t* status, void* stream) {
  moba::api::clear_error();
  moba::CacheGeom g;
  MOBA_TRY(make_cache_geom(p, &g));
  if (max_tokens < 0) return fail(MOBA_ERR_INVALID_ARG, "max_tokens must be >= 0 (got %d)", max_tokens);
  MOBA_TRY(check_ptr(add, "add", 4));
  MOBA_TRY(check_ptr(lens, "lens", 4));
  MOBA_TRY(check_ptr(tables, "tables", 4));
  MOBA_TRY(check_ptr(free_pages, "free_pages", 4));
  MOBA_TRY(check_ptr(free_state, "free_state", 4));
  MOBA_TRY(check_ptr(lens_out, "lens_out", 4));
  MOBA_TRY(check_ptr(free_state_out, "free_state_out", 4));
  MOBA_TRY(check_ptr(cu_new, "cu_new", 4));
  if (max_tokens > 0) MOBA_TRY(check_ptr(slots, "slots", 4));
  MOBA_TRY(check_ptr(status, "status", 4));
  MOBA_TRY(moba::api::device_error_word(&g.err));
  const cudaError_t e = moba::launch_cache_tables(g, add, lens, tables, free_pages, free_state, lens_out,
                                                  free_state_out, cu_new, slots, max_tokens, status,
                                                  (cudaStream_t)stream);
  return e == cudaSuccess ? MOBA_OK : cuda_error(e, "cache tables launch");
}

moba_status moba_cache_append(const moba_cache_params* p, const void* K, int64_t k_stride, const void* V,
                              int64_t v_stride, int32_t max_tokens, const int32_t* cu_new, const int32_t* lens,
                              const int32_t* slots, const int32_t* tables, void* Kc, void* Vc, float* Ks, float* Vs,
                              float* Kbar, void* stream) {
  moba::api::clear_error();
  moba::CacheGeom g;
  MOBA_TRY(make_cache_geom(p, &g));
  if (max_tokens < 0) return fail(MOBA_ERR_INVALID_ARG, "max_tokens must be >= 0 (got %d)", max_tokens);
  if (max_tokens == 0) return MOBA_OK;
  const int64_t row = (int64_t)g.Hkv * g.D;
  if (k_stride < row || v_stride < row)
    return fail(MOBA_ERR_INVALID_ARG, "k_stride and v_stride must be >= num_kv_heads * head_dim (%lld)", (long long)row);
  if (k_stride % 8 || v_stride % 8)
    return fail(MOBA_ERR_ALIGNMENT, "k_stride and v_stride must be multiples of 8 elements");
  MOBA_TRY(check_ptr(K, "K"));
  MOBA_TRY(check_ptr(V, "V"));
  MOBA_TRY(check_ptr(cu_new, "cu_new", 4));
  MOBA_TRY(check_ptr(lens, "lens", 4));
  MOBA_TRY(check_ptr(slots, "slots", 4));
  MOBA_TRY(check_ptr(tables, "tables", 4));
  MOBA_TRY(check_ptr(Kc, "Kc"));
  MOBA_TRY(check_ptr(Vc, "Vc"));
  MOBA_TRY(check_ptr(Ks, "Ks"));
  MOBA_TRY(check_ptr(Vs, "Vs"));
  MOBA_TRY(check_ptr(Kbar, "Kbar"));
  MOBA_TRY(moba::api::device_error_word(&g.err));
  const cudaError_t e = moba::launch_cache_append(
      g, (const __nv_bfloat16*)K, k_stride, (const __nv_bfloat16*)V, v_stride, max_tokens, cu_new, lens, slots, tables,
      (uint8_t*)Kc, (uint8_t*)Vc, Ks, Vs, Kbar, (cudaStream_t)stream);
  return e == cudaSuccess ? MOBA_OK : cuda_error(e, "cache append launch");
}

size_t moba_cache_decode_workspace_size(const moba_cache_params* p) {
  moba::CacheGeom g;
  if (make_cache_geom(p, &g) != MOBA_OK) return 0;
  return carve_cache_decode(g, nullptr).bytes;
}

moba_status moba_cache_decode_fwd(const moba_cache_params* p, const void* Q, const void* Kc, const void* Vc,
                                  const float* Ks, const float* Vs, const float* Kbar, const int32_t* lens,
                                  const int32_t* tables, int32_t* sel, void* workspace, size_t workspace_bytes,
                                  void* O, float* LSE, void* stream) {
  moba::api::clear_error();
  moba::CacheGeom g;
  MOBA_TRY(make_cache_geom(p, &g));
  MOBA_TRY(check_ptr(Q, "Q"));
  MOBA_TRY(check_ptr(Kc, "Kc"));
  MOBA_TRY(check_ptr(Vc, "Vc"));
  MOBA_TRY(check_ptr(Ks, "Ks"));
  MOBA_TRY(check_ptr(Vs, "Vs"));
  MOBA_TRY(check_ptr(Kbar, "Kbar"));
  MOBA_TRY(check_ptr(lens, "lens", 4));
  MOBA_TRY(check_ptr(tables, "tables", 4));
  if (sel) MOBA_TRY(check_ptr(sel, "sel", 4));
  MOBA_TRY(check_ptr(O, "O"));
  MOBA_TRY(check_ptr(LSE, "LSE"));
  const size_t need = carve_cache_decode(g, nullptr).bytes;
  if (!workspace) return fail(MOBA_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
  if ((uintptr_t)workspace & 255) return fail(MOBA_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (workspace_bytes < need) return fail(MOBA_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", workspace_bytes, need);
  MOBA_TRY(moba::api::device_error_word(&g.err));
  const moba::CacheDecodeWork w = carve_cache_decode(g, (char*)workspace);
  const cudaError_t e = moba::launch_cache_decode(g, (const __nv_bfloat16*)Q, (const uint8_t*)Kc, (const uint8_t*)Vc,
                                                  Ks, Vs, Kbar, lens, tables, sel ? sel : w.sel, w,
                                                  (__nv_bfloat16*)O, LSE, (cudaStream_t)stream);
  return e == cudaSuccess ? MOBA_OK : cuda_error(e, "cache decode launch");
}

}  // extern "C"
