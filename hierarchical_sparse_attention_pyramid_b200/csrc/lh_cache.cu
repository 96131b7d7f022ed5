// Writing tokens into the paged cache, quantised as they are written, and
// reading sequences back.
//
// Both are bound by memory (each element moves once in each direction).  A
// row is one token's head: d/16 lanes of 16 channels each when writing, so
// that the row's largest magnitude is a shuffle reduction, and 16 bytes of held
// values a lane when reading.  A thread carries K and V together, which keeps
// two rows' loads in flight and looks the page up once for both.
#include <cuda_fp8.h>
#include <math.h>

#include <type_traits>

#include "lh_cache.cuh"

namespace lh {
namespace {

constexpr int kThreads = 256;
constexpr int kV = 16;         // channels of a lane when writing (8: 60 us instead of 48 for 87K tokens of 4 heads)
constexpr int kReadHeads = 2;  // heads that a thread reads (1, 4: 52, 55 us instead of 50)

template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

// largest size of three, NaN if one is NaN
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <typename T, int N>
struct alignas(sizeof(T) * N > 16 ? 16 : sizeof(T) * N) Pack {
  T e[N];
};

// x (16 channels of a lane) of a row of LANES lanes into the cache; every lane
// of the warp calls it, the rows that are `live` are stored
template <int KIND, int LANES>
__device__ __forceinline__ void store_row(const float (&x)[kV], void* data, float* scale, int64_t row, int lane_in_row,
                                          bool live) {
  if constexpr (KIND == LH_CACHE_BF16 || KIND == LH_CACHE_FP16) {
    using H = typename std::conditional<KIND == LH_CACHE_BF16, __nv_bfloat16, __half>::type;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      Pack<H, 8> p;
#pragma unroll
      for (int i = 0; i < 8; ++i) p.e[i] = from_f<H>(x[8 * j + i]);
      if (live) reinterpret_cast<Pack<H, 8>*>(data)[(row * LANES + lane_in_row) * 2 + j] = p;
    }
  } else {
    constexpr float top = KIND == LH_CACHE_E4M3 ? 448.f : 127.f;
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kV; i += 2) m = max_abs3(m, x[i], x[i + 1]);
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) m = max_abs3(m, m, __shfl_xor_sync(0xffffffffu, m, d));
    const bool finite = m <= 3.402823466e38f;
    // a row below about 1e-36 would need a multiplier beyond fp32: the largest one is used
    const float inv = m > 0.f ? fminf(__fdiv_rn(top, m), 3.402823466e38f) : 0.f;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t h[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float a = __fmul_rn(x[4 * j + 2 * i], inv), b = __fmul_rn(x[4 * j + 2 * i + 1], inv);
        if constexpr (KIND == LH_CACHE_E4M3) {
          h[i] = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
        } else {
          const int ia = __float2int_rn(fminf(fmaxf(a, -top), top)), ib = __float2int_rn(fminf(fmaxf(b, -top), top));
          h[i] = __byte_perm(ia, ib, 0x0040);
        }
      }
      w[j] = __byte_perm(h[0], h[1], 0x5410);
    }
    // a row with a NaN or an infinity reads back as NaN
    if (live) {
      reinterpret_cast<uint4*>(data)[row * LANES + lane_in_row] = finite ? make_uint4(w[0], w[1], w[2], w[3])
                                                                         : make_uint4(0, 0, 0, 0);
      if (lane_in_row == 0) scale[row] = finite ? __fdiv_rn(m, top) : __int_as_float(0x7fffffff);
    }
  }
}

template <typename T, bool WIDE>
__device__ __forceinline__ void load_row(const T* p, float (&x)[kV]) {
  constexpr int N = 16 / sizeof(T);
#pragma unroll
  for (int j = 0; j < kV / N; ++j) {
    if constexpr (WIDE) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + j);
      const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
      for (int i = 0; i < N; ++i) x[N * j + i] = to_f<T>(e[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x[N * j + i] = to_f<T>(p[N * j + i]);
    }
  }
}

// WIDE: 16-byte loads (pointers and strides allow them)
template <typename T, int KIND, int D, bool WIDE>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheIoArgs a) {
  constexpr int LANES = D / kV;
  const int lane = threadIdx.x % LANES;
  const uint32_t r = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;  // token * heads + head
  const uint32_t tok = r / (uint32_t)a.c.heads;
  const int h = (int)(r % (uint32_t)a.c.heads);
  // every lane reaches the shuffles; rows that are not written compute on
  // zeros.  The rows are loaded beside their slot, not after it.
  float k[kV] = {}, v[kV] = {};
  int64_t slot = -1;
  if (tok < a.n) {
    slot = __ldg(a.slots + tok);
    load_row<T, WIDE>(static_cast<const T*>(a.k) + tok * a.k_stride[0] + h * a.k_stride[1] + lane * kV, k);
    load_row<T, WIDE>(static_cast<const T*>(a.v) + tok * a.v_stride[0] + h * a.v_stride[1] + lane * kV, v);
    if (slot >= a.c.pages << a.c.log2_page) {
      if (lane == 0) report_error(a.errw, ERRW_BOUNDS);
      slot = -1;
    }
  }
  const int64_t page = slot >> a.c.log2_page, at = slot & ((1 << a.c.log2_page) - 1);
  const int64_t row = ((page * a.c.heads + h) << a.c.log2_page) + at;
  store_row<KIND, LANES>(k, a.c.k, a.c.k_scale, row, lane, slot >= 0);
  store_row<KIND, LANES>(v, a.c.v, a.c.v_scale, row, lane, slot >= 0);
}

// the sequence whose rows [starts[s], starts[s+1]) hold row r, -1 for none
__device__ __forceinline__ int find_seq(const int32_t* __restrict__ starts, int seqs, int64_t r) {
  int lo = 0, hi = seqs;  // the last s with starts[s] <= r
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(starts + mid) <= r) lo = mid;
    else hi = mid - 1;
  }
  return lo < seqs && __ldg(starts + lo) <= r && r < __ldg(starts + lo + 1) ? lo : -1;
}

// held: V values of a lane, 8 or 16 bytes of them
template <typename T, int KIND, int V>
__device__ __forceinline__ void widen(const void* src, float scale, T* dst) {
  float x[V];
  if constexpr (KIND == LH_CACHE_BF16 || KIND == LH_CACHE_FP16) {
    using H = typename std::conditional<KIND == LH_CACHE_BF16, __nv_bfloat16, __half>::type;
    const uint4 u = __ldcs(static_cast<const uint4*>(src));
    const H* e = reinterpret_cast<const H*>(&u);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = to_f<H>(e[i]);
  } else {
    uint32_t w[V / 4];
    const uint4 u = __ldcs(static_cast<const uint4*>(src));
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const uint32_t h = w[i / 4] >> (8 * (i % 4));
      float lo, hi;
      if constexpr (KIND == LH_CACHE_E4M3) {
        const __half2_raw f = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(h & 0xffff), __NV_E4M3);
        const float2 f2 = __half22float2(*reinterpret_cast<const __half2*>(&f));
        lo = f2.x, hi = f2.y;
      } else {
        lo = (float)(int8_t)(h & 0xff), hi = (float)(int8_t)((h >> 8) & 0xff);
      }
      x[i] = lo * scale;
      x[i + 1] = hi * scale;
    }
  }
  constexpr int P = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < V; i += P) {
    Pack<T, P> o;
#pragma unroll
    for (int j = 0; j < P; ++j) o.e[j] = from_f<T>(x[i + j]);
    __stcs(reinterpret_cast<uint4*>(dst + i), *reinterpret_cast<const uint4*>(&o));  // read next by another kernel
  }
}

template <typename T, int KIND, int D>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheIoArgs a) {
  constexpr int BYTES = KIND == LH_CACHE_E4M3 || KIND == LH_CACHE_INT8 ? 1 : 2;
  constexpr int V = 16 / BYTES, LANES = D / V;
  const int lane = threadIdx.x % LANES;
  const uint32_t r = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  const int per = (a.c.heads + gridDim.y - 1) / gridDim.y;
  const int h0 = blockIdx.y * per, h1 = min(h0 + per, a.c.heads);
  if (r >= a.n) return;
  const int s = find_seq(a.starts, a.seqs, r);
  if (s < 0) return;  // a row of no sequence is left as it is
  const int64_t pos = r - __ldg(a.starts + s);
  const int64_t col = pos >> a.c.log2_page;
  const int page = col < a.width ? __ldg(a.table + (int64_t)s * a.width + col) : -1;
  if (page < 0 || page >= a.c.pages) {
    if (lane == 0) report_error(a.errw, ERRW_BOUNDS);
    return;
  }
  const int64_t at = pos & ((1 << a.c.log2_page) - 1);
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    const int64_t row = (((int64_t)page * a.c.heads + h) << a.c.log2_page) + at;
    float ks = 1.f, vs = 1.f;
    if constexpr (BYTES == 1) {
      ks = __ldg(a.c.k_scale + row);
      vs = __ldg(a.c.v_scale + row);
    }
    const int64_t src = (row * D + lane * V) * BYTES, dst = ((int64_t)r * a.c.heads + h) * D + lane * V;
    widen<T, KIND, V>(static_cast<const char*>(a.c.k) + src, ks, static_cast<T*>(a.k_out) + dst);
    widen<T, KIND, V>(static_cast<const char*>(a.c.v) + src, vs, static_cast<T*>(a.v_out) + dst);
  }
}

template <typename T, int KIND, int D>
cudaError_t write_d(const CacheIoArgs& a, cudaStream_t st) {
  constexpr int R = kThreads / (D / kV);  // rows of a block
  const int64_t grid = (a.n * a.c.heads + R - 1) / R;
  constexpr int64_t W = 16 / sizeof(T);
  const bool wide = ((reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) & 15) == 0 &&
                    a.k_stride[0] % W == 0 && a.k_stride[1] % W == 0 && a.v_stride[0] % W == 0 &&
                    a.v_stride[1] % W == 0;
  if (wide) cache_write_kernel<T, KIND, D, true><<<dim3((unsigned)grid), kThreads, 0, st>>>(a);
  else cache_write_kernel<T, KIND, D, false><<<dim3((unsigned)grid), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int KIND, int D>
cudaError_t read_d(const CacheIoArgs& a, cudaStream_t st) {
  constexpr int V = KIND == LH_CACHE_E4M3 || KIND == LH_CACHE_INT8 ? 16 : 8;
  constexpr int R = kThreads / (D / V);  // tokens of a block
  const int64_t gx = (a.n + R - 1) / R;
  // a thread walks some heads of its token (one page lookup)
  const int gy = (a.c.heads + kReadHeads - 1) / kReadHeads;
  cache_read_kernel<T, KIND, D><<<dim3((unsigned)gx, (unsigned)gy), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

// one launch of the kernel of a's head size and kind, for elements T
template <typename T, bool WRITE, int KIND>
cudaError_t by_d(const CacheIoArgs& a, cudaStream_t st) {
  if (a.c.d == 128) return WRITE ? write_d<T, KIND, 128>(a, st) : read_d<T, KIND, 128>(a, st);
  return WRITE ? write_d<T, KIND, 64>(a, st) : read_d<T, KIND, 64>(a, st);
}
template <typename T, bool WRITE>
cudaError_t by_kind(const CacheIoArgs& a, cudaStream_t st) {
  switch (a.c.kind) {
    case LH_CACHE_BF16: return by_d<T, WRITE, LH_CACHE_BF16>(a, st);
    case LH_CACHE_FP16: return by_d<T, WRITE, LH_CACHE_FP16>(a, st);
    case LH_CACHE_E4M3: return by_d<T, WRITE, LH_CACHE_E4M3>(a, st);
    default: return by_d<T, WRITE, LH_CACHE_INT8>(a, st);
  }
}
template <bool WRITE>
cudaError_t by_type(const CacheIoArgs& a, int dtype, cudaStream_t st) {
  if (dtype == LH_BF16) return by_kind<__nv_bfloat16, WRITE>(a, st);
  if (dtype == LH_FP16) return by_kind<__half, WRITE>(a, st);
  return by_kind<float, WRITE>(a, st);
}

}  // namespace

cudaError_t launch_cache_write(const CacheIoArgs& a, int dtype, cudaStream_t st) {
  return by_type<true>(a, dtype, st);
}
cudaError_t launch_cache_read(const CacheIoArgs& a, int dtype, cudaStream_t st) {
  return by_type<false>(a, dtype, st);
}

}  // namespace lh
