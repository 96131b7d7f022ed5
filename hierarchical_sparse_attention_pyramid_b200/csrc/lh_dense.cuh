// Masked dense attention over all N tokens (forward and backward): what the
// kernels share.
//
// Every mask here leaves each query i one interval of keys [lo_i, hi_i): its
// document up to itself (causal), extended to the document's leading prefix
// tokens; an empty interval for padding.  Seen from a key j the queries are
// an interval too.  lh_mask_spans writes both, and for each tile of 128 rows
// the least and the greatest bounds, from which a kernel takes the range of
// tiles it visits and which of them need no masking.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "lh_common.cuh"
#include "sm100.cuh"

namespace lh {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994530942f;

// bounds of the non-empty rows of one 128-row tile
struct TileSpan {
  int min_lo, max_hi;  // union of the rows' intervals: [min_lo, max_hi); min_lo >= max_hi: every row is empty
  int max_lo, min_hi;  // what every row sees: [max_lo, min_hi) (empty as soon as one row is)
};

struct MaskView {
  const int2* rows;          // [B][N] keys of a query; NULL: computed from `causal`
  const int2* cols;          // [B][N] queries of a key
  const TileSpan* row_tile;  // [B][n_tiles]
  const TileSpan* col_tile;  // [B][n_tiles]
  const int* padded;         // [B]
  int causal;
};

__device__ __forceinline__ int2 mask_row(const MaskView& m, int b, int i, int N) {
  if (i >= N) return make_int2(0, 0);
  if (m.rows) return __ldg(m.rows + (int64_t)b * N + i);
  return make_int2(0, m.causal ? i + 1 : N);
}
__device__ __forceinline__ int2 mask_col(const MaskView& m, int b, int j, int N) {
  if (j >= N) return make_int2(0, 0);
  if (m.cols) return __ldg(m.cols + (int64_t)b * N + j);
  return make_int2(m.causal ? j : 0, N);
}
__device__ __forceinline__ TileSpan mask_row_tile(const MaskView& m, int b, int t, int N) {
  if (m.rows) {
    const int4 v = __ldg(reinterpret_cast<const int4*>(m.row_tile) + (int64_t)b * ((N + 127) / 128) + t);
    return {v.x, v.y, v.z, v.w};
  }
  if (!m.causal) return {0, N, 0, N};
  return {0, min(N, t * 128 + 128), 0, t * 128 + 1};
}
__device__ __forceinline__ TileSpan mask_col_tile(const MaskView& m, int b, int t, int N) {
  if (m.cols) {
    const int4 v = __ldg(reinterpret_cast<const int4*>(m.col_tile) + (int64_t)b * ((N + 127) / 128) + t);
    return {v.x, v.y, v.z, v.w};
  }
  if (!m.causal) return {0, N, 0, N};
  return {t * 128, N, min(N, t * 128 + 128) - 1, N};
}

// the pieces of a spans buffer (lh_mask_spans_bytes)
struct SpanBuffer {
  int4 *row_tile, *col_tile;  // [B][n_tiles]
  int2 *rows, *cols;          // [B][N]
  int* scratch;               // [B][N]
  int* padded;                // [B] whether a row of the batch has padding
};
inline SpanBuffer span_buffer(void* p, int64_t B, int64_t N) {
  const int64_t tiles = B * ((N + 127) / 128);
  SpanBuffer s;
  s.row_tile = static_cast<int4*>(p);
  s.col_tile = s.row_tile + tiles;
  s.rows = reinterpret_cast<int2*>(s.col_tile + tiles);
  s.cols = s.rows + B * N;
  s.scratch = reinterpret_cast<int*>(s.cols + B * N);
  s.padded = s.scratch + B * N;
  return s;
}
inline size_t span_bytes(int64_t B, int64_t N) {
  return (size_t)(B * ((N + 127) / 128)) * 2 * sizeof(int4) + (size_t)(B * N) * (2 * sizeof(int2) + sizeof(int)) +
         (size_t)B * sizeof(int);
}

// Padding tokens of a tile (nothing sees them, they see nothing): what they
// hold is not to be used, yet a product multiplies it by zero, and zero times a
// NaN is not zero.  So a tile with padding has those rows zeroed in shared
// memory before such a product reads them.  Whether a tile has any its bounds
// say, which the kernels ask only where a row of the batch has padding and a
// tile needs masking.
__device__ __forceinline__ bool has_padding(const MaskView& m, int b) { return m.rows && __ldg(m.padded + b) != 0; }
__device__ __forceinline__ bool empty_keys(const MaskView& m, int b, int t, int N) {
  return mask_col_tile(m, b, t, N).min_hi == 0;
}
__device__ __forceinline__ bool empty_queries(const MaskView& m, int b, int t, int N) {
  return mask_row_tile(m, b, t, N).min_hi == 0;
}
// zero `regions` 128-byte pieces of row r of a tile of 64-channel regions
__device__ __forceinline__ void zero_row(uint8_t* tile, int r, int first, int regions) {
  for (int c = first; c < first + regions; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<uint4*>(tile + c * (128 * 128) + r * 128 + i * 16) = make_uint4(0, 0, 0, 0);
}

// strides of a [B][H][N][d] tensor in elements (d contiguous)
struct Strides {
  int64_t b, h, n;
};

struct DenseArgs {
  int B, N, Hq, Hkv, n_tiles;
  int q_per_cta;    // the forward's query tiles of a CTA, 1 or 2
  float scale;      // of the scores
  float softcap;    // 0: none
  const float* slopes;  // [Hq] or NULL
  MaskView mask;
  float* lse;       // [B][Hq][N]
  float* delta;     // [B][Hq][N]
  int* errw;
};

// ---------------------------------------------------------------------------
// 16-bit element types
// ---------------------------------------------------------------------------
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return F16 ? sm100::pack_f16x2(lo, hi) : sm100::pack_bf16x2(lo, hi);
}
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&u));
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// Outputs of a tile leave a warp as whole lines: its 32 rows of CW bytes lie in
// shared memory, 16-byte chunk c of row r at line_at<CW>(r, c) (8 neighbouring
// rows meet different banks), and go to rows of `dst`, of which `rows` are.
template <int CW>
__device__ __forceinline__ int line_at(int r, int c) {
  return r * CW + ((c ^ (r & (CW / 16 - 1))) << 4);
}
template <int CW>
__device__ __forceinline__ void store_lines(const uint8_t* lines, uint16_t* dst, int64_t stride, int rows, int lane) {
  constexpr int CH = CW / 16;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int r = i * (32 / CH) + lane / CH;
    if (r < rows)
      *reinterpret_cast<uint4*>(dst + r * stride + lane % CH * 8) =
          *reinterpret_cast<const uint4*>(lines + line_at<CW>(r, lane % CH));
  }
}
template <bool F16>
__host__ __device__ constexpr uint32_t idesc16(int M, int N, bool a_mn, bool b_mn) {
  return F16 ? sm100::idesc_f16(M, N, a_mn, b_mn) : sm100::idesc_bf16(M, N, a_mn, b_mn);
}

// tanh, to a relative 1.8e-7: the capped score is softcap * tanh, and a score
// far below the cap keeps its own digits.  For |y| <= 1 the odd polynomial of
// degree 13 that interpolates tanh(y) / y at Chebyshev points of y^2 in
// [0, 1]; beyond, from one exponential and one reciprocal (absolute error 1e-7).
// The polynomial needs neither, whose unit the softmax's own exponentials fill.
__device__ __forceinline__ void tanh_near(float& a, float& b) {
  using namespace sm100;
  constexpr float c[7] = {0.99999994f, -0.33332857f, 0.13325398f, -0.053465176f, 0.02030552f, -0.00621707f,
                          0.0010455536f};
  const uint64_t y = f2_pack(a, b), u = f2_mul(y, y);
  uint64_t p = f2_pack(c[6], c[6]);
#pragma unroll
  for (int k = 5; k >= 0; --k) p = f2_fma(p, u, f2_pack(c[k], c[k]));
  f2_unpack(f2_mul(y, p), a, b);
}
__device__ __forceinline__ float tanh_far(float y) {
  float r;
  const float e = sm100::fast_exp2(y * (2.f * kLog2e));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 1.f));
  return fmaf(-2.f, r, 1.f);
}
__device__ __forceinline__ void tanh_any(float& a, float& b) {
  float na = a, nb = b;
  tanh_near(na, nb);
  a = fabsf(a) <= 1.f ? na : tanh_far(a);
  b = fabsf(b) <= 1.f ? nb : tanh_far(b);
}
__device__ __forceinline__ float tanh_any(float y) {
  float a = y, b = y;
  tanh_any(a, b);
  return a;
}

// tanh of N scores times `pre`, in place; one vote of the warp settles whether
// all of them are below the cap
template <int N>
__device__ __forceinline__ void cap_scores(uint32_t (&r)[N], float pre) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < N; i += 2)
    top = sm100::max3f(top, fabsf(__uint_as_float(r[i])), fabsf(__uint_as_float(r[i + 1])));
  auto each = [&](auto near) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      float a, b;
      sm100::f2_unpack(sm100::f2_mul(sm100::f2_pack(__uint_as_float(r[i]), __uint_as_float(r[i + 1])),
                                     sm100::f2_pack(pre, pre)), a, b);
      if constexpr (decltype(near)::value) tanh_near(a, b);
      else tanh_any(a, b);
      r[i] = __float_as_uint(a);
      r[i + 1] = __float_as_uint(b);
    }
  };
  if (__all_sync(0xffffffffu, top * pre <= 1.f)) each(std::true_type{});
  else each(std::false_type{});
}

// Capped and biased scores: a score s becomes t = tanh(s pre) (capped, by
// cap_scores) or s itself, then the exponent of two t mul - slope2 |i - j|.
struct Mod {
  float pre, mul, slope2;
  bool cap, bias;
};
__device__ __forceinline__ Mod make_mod(const DenseArgs& a, int h) {
  Mod m;
  m.cap = a.softcap > 0.f;
  m.bias = a.slopes != nullptr;
  m.pre = m.cap ? a.scale / a.softcap : 0.f;
  m.mul = (m.cap ? a.softcap : a.scale) * kLog2e;
  m.slope2 = m.bias ? a.slopes[h] * kLog2e : 0.f;
  return m;
}

// 4-D tensor map of a strided 16-bit tensor (with the sequence maps, lh_attn_fwd.cu)
bool make_head_map(CUtensorMap* m, const void* base, int dtype, int64_t B, int64_t H, int64_t N, int D,
                   const int64_t* stride);

cudaError_t launch_mask_spans(const int32_t* docs, const uint8_t* prefix, int64_t B, int N, int causal,
                              const SpanBuffer& s, cudaStream_t st);
cudaError_t launch_dense_fwd(const DenseArgs& a, int d, bool f16, const CUtensorMap& q, const CUtensorMap& k,
                             const CUtensorMap& v, void* o, const Strides& so, void* o_low, cudaStream_t st);
cudaError_t launch_dense_bwd(const DenseArgs& a, int d, bool f16, const CUtensorMap& q, const CUtensorMap& k,
                             const CUtensorMap& v, const CUtensorMap& go, const void* o, const Strides& so,
                             const void* o_low, void* dq, const Strides& sdq, void* dk, const Strides& sdk, void* dv,
                             const Strides& sdv, cudaStream_t st);

}  // namespace lh
