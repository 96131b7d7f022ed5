// C ABI of the dense attention around the layer: argument checks and launches
// of the rotary, mask and dense attention entry points of include/lh.h.
#include <math.h>

#include "lh_dense.cuh"
#include "lh_rotary.cuh"

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
bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// strides of a TMA tensor or a 16-byte row access: multiples of 8 elements,
// positive wherever there is a second index
bool strides_ok(const int64_t* s, int64_t B, int64_t H, int64_t N) {
  const int64_t n[3] = {B, H, N};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (s[i] <= 0 || s[i] % 8 != 0 || s[i] >= ((int64_t)1 << 38))) return false;
  return true;
}
Strides strides_of(const int64_t* s) { return {s[0], s[1], s[2]}; }

lh_status check_dense(const lh_dense_config* c, const char* call) {
  if (!c) return fail(LH_ERR_INVALID_ARG, call, "NULL cfg");
  if (c->B < 1 || c->N < 1 || c->Hq < 1 || c->Hkv < 1)
    return fail(LH_ERR_INVALID_ARG, call, "sizes must be positive");
  if (c->Hq % c->Hkv != 0) return fail(LH_ERR_INVALID_ARG, call, "Hq must be a multiple of Hkv");
  if (c->d != 64 && c->d != 128) return fail(LH_ERR_UNSUPPORTED, call, "d must be 64 or 128");
  if (c->dtype != LH_BF16 && c->dtype != LH_FP16)
    return c->dtype == LH_FP32 ? fail(LH_ERR_UNSUPPORTED, call, "dtype must be bf16 or fp16")
                               : fail(LH_ERR_INVALID_ARG, call, "bad dtype");
  if (!(c->scale > 0.f) || !isfinite(c->scale)) return fail(LH_ERR_INVALID_ARG, call, "scale must be positive");
  if (!(c->softcap >= 0.f) || !isfinite(c->softcap))
    return fail(LH_ERR_INVALID_ARG, call, "softcap must be 0 or positive");
  if (c->causal != 0 && c->causal != 1) return fail(LH_ERR_INVALID_ARG, call, "causal must be 0 or 1");
  if (c->N > ((int64_t)1 << 30) || c->B > (1 << 20) || c->Hq > 65535 ||
      c->B * c->Hq * ((c->N + 127) / 128) > 0x7fffffffll)
    return fail(LH_ERR_UNSUPPORTED, call, "more than 2^31 - 1 query tiles");
  return LH_OK;
}

DenseArgs dense_args(const lh_dense_config* c, const void* spans, const float* slopes, void* err) {
  DenseArgs a{};
  a.B = (int)c->B;
  a.N = (int)c->N;
  a.Hq = c->Hq;
  a.Hkv = c->Hkv;
  a.n_tiles = (int)((c->N + 127) / 128);
  a.scale = c->scale;
  a.softcap = c->softcap;
  a.slopes = slopes;
  a.mask.causal = c->causal;
  if (spans) {
    const SpanBuffer s = span_buffer(const_cast<void*>(spans), c->B, c->N);
    a.mask.rows = s.rows;
    a.mask.cols = s.cols;
    a.mask.row_tile = reinterpret_cast<const TileSpan*>(s.row_tile);
    a.mask.padded = s.padded;
    a.mask.col_tile = reinterpret_cast<const TileSpan*>(s.col_tile);
  }
  a.errw = static_cast<int*>(err);
  return a;
}

}  // namespace
}  // namespace lh

using namespace lh;

#define CHECK_PTR(p)                                                                                       \
  do {                                                                                                     \
    if (!aligned16(p)) return fail(LH_ERR_INVALID_ARG, kCall, #p ": NULL or not 16-byte aligned");          \
  } while (0)
#define CHECK_STRIDE(s, H)                                                                                 \
  do {                                                                                                     \
    if (!strides_ok(cfg->s, cfg->B, H, cfg->N))                                                            \
      return fail(LH_ERR_INVALID_ARG, kCall, #s ": strides must be positive multiples of 8 elements");     \
  } while (0)

extern "C" {

lh_status lh_rotary(const lh_rotary_config* cfg, const void* q, const void* k, const double* freq,
                    const int32_t* positions, void* q_out, void* k_out, lh_stream_t stream) {
  const char* kCall = "lh_rotary";
  if (!cfg) return fail(LH_ERR_INVALID_ARG, kCall, "NULL cfg");
  if (cfg->B < 0 || cfg->N < 0 || cfg->Hq < 0 || cfg->Hk < 0 || cfg->Hq + (int64_t)cfg->Hk < 1 || cfg->d < 1)
    return fail(LH_ERR_INVALID_ARG, kCall, "negative size, or no heads");
  if (cfg->rot < 0 || cfg->rot > cfg->d || cfg->rot % 2 != 0)
    return fail(LH_ERR_INVALID_ARG, kCall, "rot must be even and in [0, d]");
  if (cfg->layout != LH_ROTARY_HALF && cfg->layout != LH_ROTARY_INTERLEAVED)
    return fail(LH_ERR_INVALID_ARG, kCall, "bad layout");
  if (cfg->dtype != LH_BF16 && cfg->dtype != LH_FP16 && cfg->dtype != LH_FP32)
    return fail(LH_ERR_INVALID_ARG, kCall, "bad dtype");
  if (cfg->inverse != 0 && cfg->inverse != 1) return fail(LH_ERR_INVALID_ARG, kCall, "inverse must be 0 or 1");
  if (cfg->d > 65536 || cfg->Hq > 65535 || cfg->Hk > 65535 || (cfg->N > 0 && cfg->B > ((int64_t)1 << 40) / cfg->N))
    return fail(LH_ERR_UNSUPPORTED, kCall, "too many tokens, heads or channels");
  if (!positions && cfg->N > ((int64_t)1 << 31)) return fail(LH_ERR_UNSUPPORTED, kCall, "positions past 2^31");
  if (cfg->B == 0 || cfg->N == 0) return LH_OK;
  if ((cfg->Hq && (!q || !q_out)) || (cfg->Hk && (!k || !k_out)) || (cfg->rot && !freq))
    return fail(LH_ERR_INVALID_ARG, kCall, "NULL pointer");
  const uintptr_t elem = cfg->dtype == LH_FP32 ? 3 : 1;
  if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)q_out | (uintptr_t)k_out) & elem ||
      ((uintptr_t)freq & 7) || ((uintptr_t)positions & 3))
    return fail(LH_ERR_INVALID_ARG, kCall, "misaligned pointer");
  RotaryArgs a{};
  a.B = cfg->B;
  a.N = cfg->N;
  a.Hq = cfg->Hq;
  a.Hk = cfg->Hk;
  a.d = cfg->d;
  a.rot = cfg->rot;
  a.q = {q, q_out, {}, {}};
  a.k = {k, k_out, {}, {}};
  for (int i = 0; i < 3; ++i) {
    a.q.si[i] = cfg->q_stride[i];
    a.k.si[i] = cfg->k_stride[i];
    a.q.so[i] = cfg->q_out_stride[i];
    a.k.so[i] = cfg->k_out_stride[i];
  }
  a.freq = freq;
  a.pos = positions;
  a.amp = cfg->amplitude;
  a.amp_sin = cfg->inverse ? -cfg->amplitude : cfg->amplitude;
  return done(launch_rotary(a, cfg->dtype, cfg->layout == LH_ROTARY_HALF, (cudaStream_t)stream), kCall);
}

size_t lh_mask_spans_bytes(int64_t B, int64_t N) { return B < 1 || N < 1 ? 0 : span_bytes(B, N); }

lh_status lh_mask_spans(int64_t B, int64_t N, int32_t causal, const int32_t* docs, const uint8_t* prefix, void* spans,
                        lh_stream_t stream) {
  const char* kCall = "lh_mask_spans";
  if (B < 1 || N < 1) return fail(LH_ERR_INVALID_ARG, kCall, "sizes must be positive");
  if (causal != 0 && causal != 1) return fail(LH_ERR_INVALID_ARG, kCall, "causal must be 0 or 1");
  if (N > ((int64_t)1 << 30) || B > (1 << 20)) return fail(LH_ERR_UNSUPPORTED, kCall, "N above 2^30 or B above 2^20");
  CHECK_PTR(spans);
  if ((uintptr_t)docs & 3) return fail(LH_ERR_INVALID_ARG, kCall, "docs: misaligned");
  return done(launch_mask_spans(docs, prefix, B, (int)N, causal, span_buffer(spans, B, N), (cudaStream_t)stream),
              kCall);
}

lh_status lh_dense_fwd(const lh_dense_config* cfg, const void* q, const void* k, const void* v, const void* spans,
                       const float* slopes, void* o, void* o_low, float* lse, void* err, lh_stream_t stream) {
  const char* kCall = "lh_dense_fwd";
  const lh_status s = check_dense(cfg, kCall);
  if (s != LH_OK) return s;
  CHECK_PTR(q); CHECK_PTR(k); CHECK_PTR(v); CHECK_PTR(o); CHECK_PTR(lse);
  if (spans) CHECK_PTR(spans);
  if (o_low) CHECK_PTR(o_low);
  if (((uintptr_t)slopes | (uintptr_t)err) & 3) return fail(LH_ERR_INVALID_ARG, kCall, "slopes or err: misaligned");
  CHECK_STRIDE(q_stride, cfg->Hq); CHECK_STRIDE(k_stride, cfg->Hkv); CHECK_STRIDE(v_stride, cfg->Hkv);
  CHECK_STRIDE(o_stride, cfg->Hq);
  DenseArgs a = dense_args(cfg, spans, slopes, err);
  a.lse = lse;
  CUtensorMap mq, mk, mv;
  if (!make_head_map(&mq, q, cfg->dtype, cfg->B, cfg->Hq, cfg->N, cfg->d, cfg->q_stride) ||
      !make_head_map(&mk, k, cfg->dtype, cfg->B, cfg->Hkv, cfg->N, cfg->d, cfg->k_stride) ||
      !make_head_map(&mv, v, cfg->dtype, cfg->B, cfg->Hkv, cfg->N, cfg->d, cfg->v_stride))
    return fail(LH_ERR_CUDA, kCall, "no tensor map for these strides");
  return done(launch_dense_fwd(a, cfg->d, cfg->dtype == LH_FP16, mq, mk, mv, o, strides_of(cfg->o_stride), o_low,
                               (cudaStream_t)stream),
              kCall);
}

lh_status lh_dense_bwd(const lh_dense_config* cfg, const void* q, const void* k, const void* v, const void* o,
                       const void* o_low, const void* dout, const float* lse, const void* spans, const float* slopes,
                       float* delta, void* dq, void* dk, void* dv, void* err, lh_stream_t stream) {
  const char* kCall = "lh_dense_bwd";
  const lh_status s = check_dense(cfg, kCall);
  if (s != LH_OK) return s;
  CHECK_PTR(q); CHECK_PTR(k); CHECK_PTR(v); CHECK_PTR(o); CHECK_PTR(dout); CHECK_PTR(lse); CHECK_PTR(delta);
  CHECK_PTR(dq); CHECK_PTR(dk); CHECK_PTR(dv);
  if (spans) CHECK_PTR(spans);
  if (o_low) CHECK_PTR(o_low);
  if (((uintptr_t)slopes | (uintptr_t)err) & 3) return fail(LH_ERR_INVALID_ARG, kCall, "slopes or err: misaligned");
  CHECK_STRIDE(q_stride, cfg->Hq); CHECK_STRIDE(k_stride, cfg->Hkv); CHECK_STRIDE(v_stride, cfg->Hkv);
  CHECK_STRIDE(o_stride, cfg->Hq); CHECK_STRIDE(do_stride, cfg->Hq); CHECK_STRIDE(dq_stride, cfg->Hq);
  CHECK_STRIDE(dk_stride, cfg->Hkv); CHECK_STRIDE(dv_stride, cfg->Hkv);
  DenseArgs a = dense_args(cfg, spans, slopes, err);
  a.lse = const_cast<float*>(lse);
  a.delta = delta;
  CUtensorMap mq, mk, mv, mo;
  if (!make_head_map(&mq, q, cfg->dtype, cfg->B, cfg->Hq, cfg->N, cfg->d, cfg->q_stride) ||
      !make_head_map(&mk, k, cfg->dtype, cfg->B, cfg->Hkv, cfg->N, cfg->d, cfg->k_stride) ||
      !make_head_map(&mv, v, cfg->dtype, cfg->B, cfg->Hkv, cfg->N, cfg->d, cfg->v_stride) ||
      !make_head_map(&mo, dout, cfg->dtype, cfg->B, cfg->Hq, cfg->N, cfg->d, cfg->do_stride))
    return fail(LH_ERR_CUDA, kCall, "no tensor map for these strides");
  return done(launch_dense_bwd(a, cfg->d, cfg->dtype == LH_FP16, mq, mk, mv, mo, o, strides_of(cfg->o_stride), o_low,
                               dq, strides_of(cfg->dq_stride), dk, strides_of(cfg->dk_stride), dv,
                               strides_of(cfg->dv_stride), (cudaStream_t)stream),
              kCall);
}

}  // extern "C"
