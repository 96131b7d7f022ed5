// C ABI of the paged cache: argument checks and launches of lh_cache_write,
// lh_cache_read and lh_cache_attn (include/lh.h).
#include <math.h>

#include "lh_cache.cuh"

namespace lh {
namespace {

lh_status fail(lh_status s, const char* call, const char* what) {
  set_error_message("%s: %s", call, what);
  return s;
}
lh_status done(cudaError_t e, const char* call) {
  if (e == cudaSuccess) return LH_OK;
  set_error_message("%s: %s", call, cudaGetErrorString(e));
  return LH_ERR_CUDA;
}
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

lh_status check_cache(const lh_cache* c, const char* call, CacheView* v) {
  if (!c) return fail(LH_ERR_INVALID_ARG, call, "NULL cache");
  if (c->pages < 1 || c->heads < 1) return fail(LH_ERR_INVALID_ARG, call, "sizes must be positive");
  if (c->d != 64 && c->d != 128) return fail(LH_ERR_UNSUPPORTED, call, "d must be 64 or 128");
  if (c->page < 8 || c->page > 4096 || (c->page & (c->page - 1)) != 0)
    return fail(LH_ERR_UNSUPPORTED, call, "page must be a power of two in [8, 4096]");
  if (c->kind < LH_CACHE_BF16 || c->kind > LH_CACHE_INT8) return fail(LH_ERR_INVALID_ARG, call, "bad kind");
  if (c->pages > 0x7fffffffll || c->heads > 65535 || c->pages * c->heads > 0xfffffffell / c->page)
    return fail(LH_ERR_UNSUPPORTED, call, "too many pages or heads");
  if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16))
    return fail(LH_ERR_INVALID_ARG, call, "k, v: NULL or not 16-byte aligned");
  const bool held8 = c->kind == LH_CACHE_E4M3 || c->kind == LH_CACHE_INT8;
  if (held8 && (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)))
    return fail(LH_ERR_INVALID_ARG, call, "k_scale, v_scale: NULL or misaligned");
  int log2 = 0;
  while ((1 << log2) < c->page) ++log2;
  *v = {c->k, c->v, c->k_scale, c->v_scale, c->pages, log2, c->heads, c->d, c->kind};
  return LH_OK;
}

lh_status check_attn(const lh_cache* c, const lh_cache_attn_config* g, const char* call, CacheView* v) {
  const lh_status s = check_cache(c, call, v);
  if (s != LH_OK) return s;
  if (!g) return fail(LH_ERR_INVALID_ARG, call, "NULL cfg");
  if (g->seqs < 0 || g->width < 1 || g->n_tok < 0 || g->max_tokens < 1)
    return fail(LH_ERR_INVALID_ARG, call, "negative size, no page column or no query token");
  if (g->Hq < 1 || g->Hq % c->heads != 0)
    return fail(LH_ERR_INVALID_ARG, call, "Hq must be a multiple of the cache's heads");
  if (g->dtype != LH_BF16 && g->dtype != LH_FP16)
    return g->dtype == LH_FP32 ? fail(LH_ERR_UNSUPPORTED, call, "dtype must be bf16 or fp16")
                               : fail(LH_ERR_INVALID_ARG, call, "bad dtype");
  if ((c->kind == LH_CACHE_BF16 && g->dtype != LH_BF16) || (c->kind == LH_CACHE_FP16 && g->dtype != LH_FP16))
    return fail(LH_ERR_UNSUPPORTED, call, "an unquantised cache takes queries of its own type");
  if (!(g->scale > 0.f) || !isfinite(g->scale)) return fail(LH_ERR_INVALID_ARG, call, "scale must be positive");
  if (!(g->softcap >= 0.f) || !isfinite(g->softcap))
    return fail(LH_ERR_INVALID_ARG, call, "softcap must be 0 or positive");
  if (g->Hq > 65535 || (int64_t)g->max_tokens * (g->Hq / c->heads) > (1 << 20) || g->n_tok > 0x7fffffffll / g->Hq ||
      (int64_t)g->width * c->page > ((int64_t)1 << 30))
    return fail(LH_ERR_UNSUPPORTED, call, "too many query tokens, sequences or positions");
  return LH_OK;
}

// blocks, workspace rows and bytes of a call
size_t attn_ws(const lh_cache* c, const lh_cache_attn_config* g, int64_t* blocks, int64_t* places) {
  *blocks = *places = 0;
  if (g->seqs == 0 || g->n_tok == 0) return 0;
  cache_attn_plan(g->seqs, c->heads, (int64_t)g->max_tokens * (g->Hq / c->heads), (int64_t)g->width * c->page, blocks,
                  places);
  return (size_t)*places * (c->d * sizeof(float) + sizeof(float2));
}

}  // namespace
}  // namespace lh

using namespace lh;

extern "C" {

lh_status lh_cache_write(const lh_cache* cache, int64_t n, int32_t dtype, const void* k, const void* v,
                         const int64_t* k_stride, const int64_t* v_stride, const int64_t* slots, void* err,
                         lh_stream_t stream) {
  const char* kCall = "lh_cache_write";
  CacheIoArgs a{};
  const lh_status s = check_cache(cache, kCall, &a.c);
  if (s != LH_OK) return s;
  if (dtype != LH_BF16 && dtype != LH_FP16 && dtype != LH_FP32) return fail(LH_ERR_INVALID_ARG, kCall, "bad dtype");
  if (n < 0) return fail(LH_ERR_INVALID_ARG, kCall, "negative token count");
  if (n > 0x7fffffffll / cache->heads) return fail(LH_ERR_UNSUPPORTED, kCall, "2^31 rows or more");
  if (n == 0) return LH_OK;
  const uintptr_t elem = dtype == LH_FP32 ? 4 : 2;
  if (!k || !v || !slots || !k_stride || !v_stride || !aligned(k, elem) || !aligned(v, elem) || !aligned(slots, 8) ||
      !aligned(err, 4))
    return fail(LH_ERR_INVALID_ARG, kCall, "NULL or misaligned pointer");
  a.n = n;
  a.k = k;
  a.v = v;
  for (int i = 0; i < 2; ++i) {
    a.k_stride[i] = k_stride[i];
    a.v_stride[i] = v_stride[i];
  }
  a.slots = slots;
  a.errw = static_cast<int*>(err);
  return done(launch_cache_write(a, dtype, (cudaStream_t)stream), kCall);
}

lh_status lh_cache_read(const lh_cache* cache, int32_t seqs, int32_t width, const int32_t* table,
                        const int32_t* starts, int64_t n, int32_t dtype, void* k_out, void* v_out, void* err,
                        lh_stream_t stream) {
  const char* kCall = "lh_cache_read";
  CacheIoArgs a{};
  const lh_status s = check_cache(cache, kCall, &a.c);
  if (s != LH_OK) return s;
  if (dtype != LH_BF16 && dtype != LH_FP16 && dtype != LH_FP32) return fail(LH_ERR_INVALID_ARG, kCall, "bad dtype");
  if (n < 0 || seqs < 0 || width < 1) return fail(LH_ERR_INVALID_ARG, kCall, "negative size or no page column");
  if (n > 0x7fffffffll) return fail(LH_ERR_UNSUPPORTED, kCall, "too many tokens");
  if (n == 0 || seqs == 0) return LH_OK;
  if (!table || !starts || !k_out || !v_out || !aligned(table, 4) || !aligned(starts, 4) || !aligned(k_out, 16) ||
      !aligned(v_out, 16) || !aligned(err, 4))
    return fail(LH_ERR_INVALID_ARG, kCall, "NULL or misaligned pointer");
  a.n = n;
  a.table = table;
  a.starts = starts;
  a.seqs = seqs;
  a.width = width;
  a.k_out = k_out;
  a.v_out = v_out;
  a.errw = static_cast<int*>(err);
  return done(launch_cache_read(a, dtype, (cudaStream_t)stream), kCall);
}

size_t lh_cache_attn_ws_bytes(const lh_cache* cache, const lh_cache_attn_config* cfg) {
  CacheView v;
  if (check_attn(cache, cfg, "lh_cache_attn_ws_bytes", &v) != LH_OK) return 0;
  int64_t blocks, places;
  return attn_ws(cache, cfg, &blocks, &places);
}

lh_status lh_cache_attn(const lh_cache* cache, const lh_cache_attn_config* cfg, const void* q, const int32_t* table,
                        const int32_t* lens, const int32_t* q_start, const uint64_t* tree, const float* slopes,
                        void* o, void* ws, size_t ws_bytes, void* err, lh_stream_t stream) {
  const char* kCall = "lh_cache_attn";
  CacheAttnArgs a{};
  const lh_status s = check_attn(cache, cfg, kCall, &a.c);
  if (s != LH_OK) return s;
  if (tree && slopes) return fail(LH_ERR_UNSUPPORTED, kCall, "a tree and slopes together");
  if (tree && cfg->max_tokens > 64) return fail(LH_ERR_UNSUPPORTED, kCall, "a tree of more than 64 tokens");
  if (!q_start && (cfg->n_tok != cfg->seqs || cfg->max_tokens != 1))
    return fail(LH_ERR_INVALID_ARG, kCall, "without q_start there is one token a sequence");
  if (cfg->seqs == 0 || cfg->n_tok == 0) return LH_OK;
  if (!q || !table || !lens || !o || !aligned(q, 16) || !aligned(o, 16) || !aligned(table, 4) || !aligned(lens, 4) ||
      !aligned(q_start, 4) || !aligned(tree, 8) || !aligned(slopes, 4) || !aligned(err, 4))
    return fail(LH_ERR_INVALID_ARG, kCall, "NULL or misaligned pointer");
  if ((cfg->n_tok > 1 && cfg->q_stride[0] % 8 != 0) || cfg->q_stride[1] % 8 != 0)
    return fail(LH_ERR_INVALID_ARG, kCall, "q_stride: strides must be multiples of 8 elements");
  int64_t blocks, places;
  const size_t need = attn_ws(cache, cfg, &blocks, &places);
  if (need && (!ws || !aligned(ws, 16))) return fail(LH_ERR_INVALID_ARG, kCall, "ws: NULL or not 16-byte aligned");
  if (ws_bytes < need) return fail(LH_ERR_WORKSPACE, kCall, "ws smaller than lh_cache_attn_ws_bytes");
  a.q = q;
  a.q_stride[0] = cfg->q_stride[0];
  a.q_stride[1] = cfg->q_stride[1];
  a.o = o;
  a.n_tok = cfg->n_tok;
  a.table = table;
  a.lens = lens;
  a.q_start = q_start;
  a.tree = tree;
  a.slopes = slopes;
  a.seqs = cfg->seqs;
  a.width = cfg->width;
  a.Hq = cfg->Hq;
  a.max_tokens = cfg->max_tokens;
  a.scale = cfg->scale;
  a.softcap = cfg->softcap;
  a.blocks = (int)blocks;
  if (need) {
    a.part_o = static_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + places * cache->d);
  }
  a.errw = static_cast<int*>(err);
  return done(launch_cache_attn(a, cfg->dtype, (cudaStream_t)stream), kCall);
}

}  // extern "C"
