// Rotary positions: pairs of the first `rot` channels of every head turned by
// angle position * frequency, scaled by an amplitude; the other channels pass
// through.  The inverse turns by the negative angle, which is the adjoint (the
// gradient of the forward).
//
// Bound by memory: each element is read and written once.  A thread owns one
// 16-byte unit of a token (8 or 4 pairs) and walks the heads with it, so that
// the sines and cosines, the only arithmetic of weight, are computed once per
// token and not once per head.  The angle is reduced to a fraction of a turn
// in 64 bits (in 32 a position of 10^6 leaves no digits of the fraction) and
// only the fraction goes to the 32-bit sincospi.  128K tokens of 20 heads of 128
// in bf16, there and back: 446 us, 6.0 TB/s (92% of a copy).
#include <type_traits>

#include "lh_common.cuh"
#include "lh_rotary.cuh"

namespace lh {
namespace {

template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

constexpr int kThreads = 256;

// V: elements of one access (16 bytes' worth, or 1 where rows, strides or the
// rotated part do not allow that).  A unit is V pairs of the half layout (two
// accesses, rot/2 apart), V pairs of the interleaved layout (two neighbouring
// accesses), or V channels of the part that passes through.
template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a) {
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (id >= a.B * a.N * a.units) return;
  const int u = (int)(id % a.units);
  const int64_t tok = id / a.units;
  const int64_t n = tok % a.N, b = tok / a.N;
  const bool turned = u < a.rot_units;
  const int off0 = turned ? (HALF ? u * V : u * 2 * V) : a.rot + (u - a.rot_units) * V;
  const int off1 = HALF ? off0 + a.rot / 2 : off0 + V;
  float s[V], c[V];
  if (turned) {
    const double pos = a.pos ? (double)a.pos[tok] : (double)n;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const double turns = pos * a.freq[u * V + i] * 0.15915494309189533577;  // / (2 pi)
      sincospif((float)(2.0 * (turns - rint(turns))), &s[i], &c[i]);
      s[i] *= a.amp_sin;
      c[i] *= a.amp;
    }
  }
  const int per = (a.Hq + a.Hk + gridDim.y - 1) / gridDim.y;
  const int h0 = blockIdx.y * per, h1 = min(h0 + per, a.Hq + a.Hk);
#pragma unroll 4
  for (int hh = h0; hh < h1; ++hh) {
    const bool isq = hh < a.Hq;
    const int h = isq ? hh : hh - a.Hq;
    const RotaryTensor& x = isq ? a.q : a.k;
    const T* src = static_cast<const T*>(x.in) + b * x.si[0] + h * x.si[1] + n * x.si[2];
    T* dst = static_cast<T*>(x.out) + b * x.so[0] + h * x.so[1] + n * x.so[2];
    using P = Vec<T, V>;
    if (turned) {
      const P p = *reinterpret_cast<const P*>(src + off0), q = *reinterpret_cast<const P*>(src + off1);
      P r, w;
      if constexpr (HALF) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float f = to_f<T>(p.e[i]), g = to_f<T>(q.e[i]);
          r.e[i] = from_f<T>(f * c[i] - g * s[i]);
          w.e[i] = from_f<T>(g * c[i] + f * s[i]);
        }
      } else {
        T in[2 * V], out[2 * V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          in[i] = p.e[i];
          in[V + i] = q.e[i];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float f = to_f<T>(in[2 * i]), g = to_f<T>(in[2 * i + 1]);
          out[2 * i] = from_f<T>(f * c[i] - g * s[i]);
          out[2 * i + 1] = from_f<T>(g * c[i] + f * s[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
          r.e[i] = out[i];
          w.e[i] = out[V + i];
        }
      }
      *reinterpret_cast<P*>(dst + off0) = r;
      *reinterpret_cast<P*>(dst + off1) = w;
    } else {
      *reinterpret_cast<P*>(dst + off0) = *reinterpret_cast<const P*>(src + off0);
    }
  }
}

template <typename T, int V>
cudaError_t launch_v(RotaryArgs a, bool half, cudaStream_t st) {
  a.rot_units = a.rot / 2 / V;
  a.units = a.rot_units + (a.d - a.rot) / V;
  const int64_t gx = (a.B * a.N * a.units + kThreads - 1) / kThreads;
  if (gx > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  // few tokens: the heads are shared out too, until there are two blocks an
  // SM (each recomputes its angles, which no longer cost anything there)
  const int heads = a.Hq + a.Hk;
  int gy = (int)(296 / gx);
  gy = gy < 1 ? 1 : gy > heads ? heads : gy;
  const dim3 grid((unsigned)gx, (unsigned)gy);
  if (half) rotary_kernel<T, V, true><<<grid, kThreads, 0, st>>>(a);
  else rotary_kernel<T, V, false><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

bool aligned(const RotaryTensor& x, int heads, int V) {
  if (!heads) return true;
  if ((reinterpret_cast<uintptr_t>(x.in) | reinterpret_cast<uintptr_t>(x.out)) & 15) return false;
  for (int i = 0; i < 3; ++i)
    if (x.si[i] % V || x.so[i] % V) return false;
  return true;
}

template <typename T>
cudaError_t launch_t(const RotaryArgs& a, bool half, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const bool wide = a.rot % (2 * V) == 0 && a.d % V == 0 && aligned(a.q, a.Hq, V) && aligned(a.k, a.Hk, V);
  return wide ? launch_v<T, V>(a, half, st) : launch_v<T, 1>(a, half, st);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int dtype, bool half, cudaStream_t st) {
  if (dtype == LH_BF16) return launch_t<__nv_bfloat16>(a, half, st);
  if (dtype == LH_FP16) return launch_t<__half>(a, half, st);
  return launch_t<float>(a, half, st);
}

}  // namespace lh
