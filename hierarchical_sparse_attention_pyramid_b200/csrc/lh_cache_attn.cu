// Attention of a few query tokens a sequence (one, or a tree of drafted ones)
// over the paged cache.
//
// Bound by reading the cache once: a key's row meets only the rows of its
// head's group (tokens x Hq / Hkv), a few operations a byte.  So each warp
// takes 16 keys at a time straight from global memory into registers, as the
// operands of 16 x 8 x 16 matrix instructions, and no shared memory stands
// between: K and V of the next 16 keys are asked for as soon as the registers
// of the present ones are free, which keeps 4 to 8 KB a warp in flight.  The
// order of the channels in Q K^T and of the output channels in P V is free, so
// each lane loads 16 contiguous bytes of a row and calls them its fragment.
//
// 8-bit values become 16-bit operands by moving bits: e4m3's exponent and
// fraction are placed in a bf16 (fp16) as they are, which is the value times
// 2^-120 (2^-8), exact also for subnormals, and undone in the score's scale
// and the output's; int8 goes through the exact difference of two small
// numbers.  The scale of a key enters its score, the scale of a value its
// probability.
//
// One block of 4 warps takes one part of one sequence's keys for 16 query
// rows of one head; the warps' running maxima, sums and outputs are joined in
// shared memory in warp order, and the parts of a sequence by a second
// kernel in part order, so that results do not depend on scheduling.
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "lh_cache.cuh"
#include "lh_dense.cuh"

namespace lh {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kKeys = 16;  // keys of a warp's step
// e4m3 as bf16 bits is the value times 2^-120: queries and probabilities are
// raised by 2^60 so that products stay far from the subnormal range
constexpr float kUp = 1152921504606846976.f;  // 2^60

template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// two held values, in bytes 1 and 3 of y (e4m3) or 0 and 2 (int8), as 16-bit
// operands
template <int KIND, bool F16>
__device__ __forceinline__ uint32_t widen2(uint32_t y) {
  if constexpr (KIND == LH_CACHE_E4M3) {
    if constexpr (F16) return (y & 0x80008000u) | ((y >> 1) & 0x3f803f80u);
    return (y & 0x80008000u) | ((y >> 4) & 0x07f007f0u);
  } else if constexpr (F16) {
    // 1024 + (x + 128) as fp16 bits, less 1152
    const uint32_t u = (y & 0x00ff00ffu) ^ 0x64806480u;
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    // (128 + low 7 bits) - (128, or 256 for a negative value) as bf16
    const uint32_t u = (y & 0x007f007fu) | 0x43004300u, w = (y & 0x00800080u) | 0x43004300u;
    const __nv_bfloat162 h = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), *reinterpret_cast<const __nv_bfloat162*>(&w));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
// bytes i and j (0-3: of x, 4-7: of z) where widen2 wants them
template <int KIND>
__device__ __forceinline__ uint32_t place(uint32_t x, uint32_t z, int i, int j) {
  return KIND == LH_CACHE_E4M3 ? __byte_perm(x, z, (uint32_t)(i << 4 | j << 12)) : __byte_perm(x, z, (uint32_t)(i | j << 8));
}

struct Row {     // one of a thread's two query rows
  int limit;     // keys below are seen (the last tokens: by `bits` with a tree)
  uint64_t bits;
  float slope2, at;  // distance bias: slope, position
};

template <typename U>
__device__ __forceinline__ U load_nc(const void* p);
template <>
__device__ __forceinline__ uint4 load_nc<uint4>(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
template <>
__device__ __forceinline__ uint2 load_nc<uint2>(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

template <int D, int KIND, bool F16>
__global__ void __launch_bounds__(kThreads, 3) cache_attn_kernel(const __grid_constant__ CacheAttnArgs a) {
  constexpr bool HELD8 = KIND == LH_CACHE_E4M3 || KIND == LH_CACHE_INT8;
  constexpr int BYTES = HELD8 ? 1 : 2;
  constexpr int E = 16 / BYTES;             // channels of a 16-byte load
  constexpr int KC = D / (4 * E);           // K loads of a lane and key (4 lanes a key)
  constexpr int STEPS = D / 16;             // matrix steps over the channels
  constexpr int VB = D * BYTES / 8 < 16 ? D * BYTES / 8 : 16;  // bytes of a V load (8 lanes a key)
  constexpr int VE = VB / BYTES, VC = D / (8 * VE), VW = VB / 4;
  constexpr bool PF16 = F16 && !HELD8;      // type of P and V: bf16 for 8-bit values, whose scales would push
                                            // probabilities below fp16's range
  constexpr float kDown = KIND == LH_CACHE_E4M3 ? (F16 ? 256.f : kUp) : 1.f;  // what a raw score is short of
  constexpr float kPUp = KIND == LH_CACHE_E4M3 ? kUp : 1.f;
  extern __shared__ __align__(16) uint8_t smem[];
  uint4* sQ = reinterpret_cast<uint4*>(smem);               // [STEPS][32] fragments of the 16 query rows
  float* sO = reinterpret_cast<float*>(smem);               // later [kWarps][16][D]
  float* sML = reinterpret_cast<float*>(smem + kWarps * 16 * D * 4);  // [kWarps][16][2]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int part = blockIdx.x, hk = blockIdx.y;
  const int G = a.Hq / a.c.heads;
  const int row_tiles = (a.max_tokens * G + 15) / 16;
  const int s = blockIdx.z / row_tiles, rt = blockIdx.z % row_tiles;
  int tok0 = s, T = 1;
  if (a.q_start) {
    tok0 = __ldg(a.q_start + s);
    T = __ldg(a.q_start + s + 1) - tok0;
  }
  if (T < 0 || T > a.max_tokens || tok0 < 0 || tok0 + (int64_t)T > a.n_tok) {
    if (threadIdx.x == 0) report_error(a.errw, ERRW_BOUNDS);
    T = max(0, min(T, a.max_tokens));
    if (tok0 < 0 || tok0 + (int64_t)T > a.n_tok) return;
  }
  if (rt * 16 >= T * G) return;
  int len = __ldg(a.lens + s);
  if (len < 0 || (int64_t)len > (int64_t)a.width << a.c.log2_page) {
    if (threadIdx.x == 0) report_error(a.errw, ERRW_BOUNDS);
    len = max(0, min(len, a.width << a.c.log2_page));
  }
  const int64_t k_begin = (int64_t)part * a.chunk;
  const int k0 = (int)(k_begin < len ? k_begin : len), k1 = min(len, k0 + a.chunk);
  if (part > 0 && k0 >= len) return;  // the join knows how many parts a sequence has
  const int ctx = len - T;            // keys before the query tokens' own

  // ------------------------------------------------------------ Q fragments, the thread's rows
  const int n_rows = T * G;
  Row row[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = rt * 16 + g + x * 8;
    const int tk = r < n_rows ? r / G : 0, h = hk * G + (r < n_rows ? r % G : 0);
    row[x].limit = r < n_rows ? (a.tree ? ctx : ctx + tk + 1) : 0;
    row[x].bits = a.tree && r < n_rows ? __ldg(reinterpret_cast<const unsigned long long*>(a.tree) + tok0 + tk) : 0;
    row[x].slope2 = a.slopes ? __ldg(a.slopes + h) * kLog2e : 0.f;
    row[x].at = (float)(ctx + tk);
  }
  for (int i = threadIdx.x; i < STEPS * 32; i += kThreads) {
    const int l = i & 31, st = i >> 5, gg = l >> 2, tt = l & 3;
    const int c = st / (E / 4), j = st % (E / 4);
    const int ch = c * 4 * E + tt * E + 4 * j;  // the lane's four channels of this step
    uint32_t f[4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = rt * 16 + gg + x * 8;
      uint32_t w0 = 0, w1 = 0;
      if (r < n_rows) {
        const uint16_t* p = static_cast<const uint16_t*>(a.q) + (int64_t)(tok0 + r / G) * a.q_stride[0] +
                            (int64_t)(hk * G + r % G) * a.q_stride[1] + ch;
        w0 = p[0] | (uint32_t)p[1] << 16;
        w1 = p[2] | (uint32_t)p[3] << 16;
        if constexpr (KIND == LH_CACHE_E4M3 && !F16) {
          const float2 u = unpack2<false>(w0), v = unpack2<false>(w1);
          w0 = pack2<false>(u.x * kUp, u.y * kUp);
          w1 = pack2<false>(v.x * kUp, v.y * kUp);
        }
      }
      f[x] = w0;
      f[2 + x] = w1;
    }
    sQ[i] = make_uint4(f[0], f[1], f[2], f[3]);
  }
  __syncthreads();

  // ------------------------------------------------------------ keys
  const int page_mask = (1 << a.c.log2_page) - 1;
  // rows of a page are 16 keys or more apart from the next page, or 8: a
  // tile of 8 keys lies in one page
  auto page_of = [&](int key) -> int {  // key a multiple of 8
    if (key >= k1) return -1;
    const int p = __ldg(a.table + (int64_t)s * a.width + (key >> a.c.log2_page));
    if (p < 0 || p >= a.c.pages) {
      if (lane == 0) report_error(a.errw, ERRW_BOUNDS);
      return -1;
    }
    return p;
  };
  // first row of the tile of 8 keys in the cache's rows, -1 without one
  auto row_of = [&](int key, int page) -> int64_t {
    return page < 0 ? -1 : (((int64_t)page * a.c.heads + hk) << a.c.log2_page) + (key & page_mask);
  };
  using KV16 = uint4;
  using VLoad = typename std::conditional<VB == 16, uint4, uint2>::type;
  uint32_t kr[2][KC][4];      // [tile of 8 keys][load]: key g of the tile
  uint32_t vr[2][2][VC][VW];  // [tile][row 2t + x][load]
  float ksc[2][2], vsc[2][2]; // scales of keys 2t, 2t+1 of each tile
  int64_t rows[2];            // of the step whose K is loaded
  auto load_k = [&](int key) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bool live = rows[j] >= 0 && key + 8 * j + g < k1;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        KV16 u = make_uint4(0, 0, 0, 0);
        if (live) u = load_nc<uint4>(static_cast<const char*>(a.c.k) + ((rows[j] + g) * D + c * 4 * E + t * E) * BYTES);
        kr[j][c][0] = u.x, kr[j][c][1] = u.y, kr[j][c][2] = u.z, kr[j][c][3] = u.w;
      }
      if constexpr (HELD8) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const bool lv = rows[j] >= 0 && key + 8 * j + 2 * t + x < k1;
          ksc[j][x] = lv ? __ldg(a.c.k_scale + rows[j] + 2 * t + x) : 0.f;
        }
      }
    }
  };
  auto load_v = [&](int key) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const bool live = rows[j] >= 0 && key + 8 * j + 2 * t + x < k1;
#pragma unroll
        for (int c = 0; c < VC; ++c) {
          VLoad u{};
          if (live)
            u = load_nc<VLoad>(static_cast<const char*>(a.c.v) +
                               ((rows[j] + 2 * t + x) * D + c * 8 * VE + g * VE) * BYTES);
          const uint32_t* w = reinterpret_cast<const uint32_t*>(&u);
#pragma unroll
          for (int i = 0; i < VW; ++i) vr[j][x][c][i] = w[i];
        }
        if constexpr (HELD8) vsc[j][x] = live ? __ldg(a.c.v_scale + rows[j] + 2 * t + x) : 0.f;
      }
  };

  float acc[VC * VE][4];
#pragma unroll
  for (int i = 0; i < VC * VE; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const bool cap = a.softcap > 0.f;
  const float pre = (cap ? a.scale / a.softcap : a.scale * kLog2e) * kDown, cap2 = a.softcap * kLog2e;

  int key = k0 + warp * kKeys;
  int pg[2] = {page_of(key), page_of(key + 8)};
  rows[0] = row_of(key, pg[0]);
  rows[1] = row_of(key + 8, pg[1]);
  load_k(key);
  load_v(key);
  for (; key < k1; key += kWarps * kKeys) {
    const int next = key + kWarps * kKeys;
    const bool bad[2] = {rows[0] < 0, rows[1] < 0};
    rows[0] = row_of(next, page_of(next));
    rows[1] = row_of(next + 8, page_of(next + 8));
    // S of the 16 rows and 16 keys
    float sc[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[j][e] = 0.f;
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
      const uint4 q4 = sQ[st * 32 + lane];
      const uint32_t qa[4] = {q4.x, q4.y, q4.z, q4.w};
      const int c = st / (E / 4), i = st % (E / 4);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t b0, b1;
        if constexpr (HELD8) {
          b0 = widen2<KIND, F16>(place<KIND>(kr[j][c][i], 0, 0, 1));
          b1 = widen2<KIND, F16>(place<KIND>(kr[j][c][i], 0, 2, 3));
        } else {
          b0 = kr[j][c][2 * i];
          b1 = kr[j][c][2 * i + 1];
        }
        mma<F16>(sc[j], qa, b0, b1);
      }
    }
    float kf[2][2];
    if constexpr (HELD8) {
#pragma unroll
      for (int j = 0; j < 2; ++j) kf[j][0] = ksc[j][0] * pre, kf[j][1] = ksc[j][1] * pre;
    } else {
      kf[0][0] = kf[0][1] = kf[1][0] = kf[1][1] = pre;
    }
    load_k(next);
    // exponents of 2, masked
    const bool edge = key + kKeys > (a.tree ? ctx : ctx + 1) || bad[0] || bad[1];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int x = e >> 1, kk = key + 8 * j + 2 * t + (e & 1);
        float y = sc[j][e] * kf[j][e & 1];
        if (cap) y = cap2 * tanh_abs(y);
        if (a.slopes) y = fmaf(-row[x].slope2, fabsf(row[x].at - (float)kk), y);
        if (edge) {
          bool seen = kk < row[x].limit;
          if (a.tree && kk >= ctx) seen = kk < len && ((row[x].bits >> (kk - ctx)) & 1);
          if (!seen || bad[j] || kk >= k1) y = -INFINITY;
        }
        sc[j][e] = y;
      }
    uint32_t pa[4];
    float alpha[2];
    bool move = false;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float mx = fmaxf(fmaxf(sc[0][2 * x], sc[0][2 * x + 1]), fmaxf(sc[1][2 * x], sc[1][2 * x + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // the reference moves only when the maximum exceeds it by more than 8
      const bool mv = mx > m[x] + 8.f;
      const float mn = mv ? mx : m[x];
      alpha[x] = mv ? sm100::fast_exp2(m[x] - mn) : 1.f;
      move |= mv;
      m[x] = mn;
      const float ref = mn == -INFINITY ? 0.f : mn;
      float p[2][2], sum = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          p[j][e] = sm100::fast_exp2(sc[j][2 * x + e] - ref);
          sum += p[j][e];
        }
      l[x] = l[x] * alpha[x] + sum;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if constexpr (HELD8)
          pa[2 * j + x] = pack2<PF16>(p[j][0] * (vsc[j][0] * kPUp), p[j][1] * (vsc[j][1] * kPUp));
        else
          pa[2 * j + x] = pack2<PF16>(p[j][0], p[j][1]);
      }
    }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int i = 0; i < VC * VE; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] *= alpha[e >> 1];
    }
#pragma unroll
    for (int c = 0; c < VC; ++c)
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        uint32_t b[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if constexpr (HELD8)
            b[j] = widen2<KIND, PF16>(place<KIND>(vr[j][0][c][i / 4], vr[j][1][c][i / 4], i % 4, 4 + i % 4));
          else
            b[j] = __byte_perm(vr[j][0][c][i / 2], vr[j][1][c][i / 2], i % 2 ? 0x7632 : 0x5410);
        }
        mma<PF16>(acc[c * VE + i], pa, b[0], b[1]);
      }
    load_v(next);
  }

  // ------------------------------------------------------------ the warps' results
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
  }
  __syncthreads();  // sQ's space is reused
#pragma unroll
  for (int x = 0; x < 2; ++x)
    if (t == 0) {
      sML[(warp * 16 + g + x * 8) * 2] = m[x];
      sML[(warp * 16 + g + x * 8) * 2 + 1] = l[x];
    }
  // accumulator i, element e: row g + 8 (e / 2), column 2t + e % 2 of the
  // step, which is channel c * 8 VE + column * VE + i % VE
#pragma unroll
  for (int i = 0; i < VC * VE; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int ch = (i / VE) * 8 * VE + (2 * t + (e & 1)) * VE + i % VE;
      sO[(warp * 16 + g + (e >> 1) * 8) * D + ch] = acc[i][e];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * D / 2; i += kThreads) {
    const int r = i / (D / 2), ch = i % (D / 2) * 2;
    const int rr = rt * 16 + r;
    if (rr >= n_rows) continue;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sML[(w * 16 + r) * 2]);
    const float ref = mm == -INFINITY ? 0.f : mm;
    float sum = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = sm100::fast_exp2(sML[(w * 16 + r) * 2] - ref);
      const float2 u = *reinterpret_cast<const float2*>(sO + (w * 16 + r) * D + ch);
      sum = fmaf(f, sML[(w * 16 + r) * 2 + 1], sum);
      o0 = fmaf(f, u.x, o0);
      o1 = fmaf(f, u.y, o1);
    }
    constexpr float kBack = KIND == LH_CACHE_E4M3 ? kUp : 1.f;  // the values' other 2^60
    o0 *= kBack;
    o1 *= kBack;
    const int64_t out = (int64_t)(tok0 + rr / G) * a.Hq + hk * G + rr % G;
    if (a.splits == 1) {
      const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
      reinterpret_cast<uint32_t*>(a.o)[(out * D + ch) / 2] = pack2<F16>(o0 * inv, o1 * inv);
    } else {
      *reinterpret_cast<float2*>(a.part_o + (out * a.splits + part) * D + ch) = make_float2(o0, o1);
      if (ch == 0) a.part_ml[out * a.splits + part] = make_float2(mm, sum);
    }
  }
}

// Joins the parts of every query row: a block a row, its warps share the
// parts out and are joined in warp order.
constexpr int kJoinWarps = 4;
template <int D, bool F16>
__global__ void __launch_bounds__(kJoinWarps * 32) cache_attn_join_kernel(const __grid_constant__ CacheAttnArgs a) {
  __shared__ float sO[kJoinWarps][D];
  __shared__ float sL[kJoinWarps];
  __shared__ float sM[kJoinWarps];
  cudaGridDependencySynchronize();
  const int64_t out = blockIdx.x;
  const int tok = (int)(out / a.Hq);
  int s = tok;
  if (a.q_start) {
    int lo = 0, hi = a.seqs;  // the last sequence whose first token is not after this one
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(a.q_start + mid) <= tok) lo = mid;
      else hi = mid - 1;
    }
    s = lo;
    if (s >= a.seqs || __ldg(a.q_start + s) > tok) return;  // a token of no sequence is left as it is
  }
  const int len = max(0, min(__ldg(a.lens + s), a.width << a.c.log2_page));
  const int parts = max(1, min(a.splits, (len + a.chunk - 1) / a.chunk));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float2* ml = a.part_ml + out * a.splits;
  float mm = -INFINITY;
  for (int p = threadIdx.x; p < parts; p += kJoinWarps * 32) mm = fmaxf(mm, ml[p].x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
  if (lane == 0) sM[warp] = mm;
  __syncthreads();
  mm = fmaxf(fmaxf(sM[0], sM[1]), fmaxf(sM[2], sM[3]));
  const float ref = mm == -INFINITY ? 0.f : mm;
  constexpr int C = D / 32;
  float o[C] = {}, sum = 0.f;
#pragma unroll 4
  for (int p = warp; p < parts; p += kJoinWarps) {
    const float2 x = ml[p];
    const float f = sm100::fast_exp2(x.x - ref);
    sum = fmaf(f, x.y, sum);
    const float* po = a.part_o + (out * a.splits + p) * D + lane * C;
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = fmaf(f, po[c], o[c]);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) sO[warp][lane * C + c] = o[c];
  if (lane == 0) sL[warp] = sum;
  __syncthreads();
  const float total = (sL[0] + sL[1]) + (sL[2] + sL[3]);
  const float inv = total > 0.f || total != total ? 1.f / total : 0.f;
  for (int i = threadIdx.x; i < D / 2; i += kJoinWarps * 32) {
    float y[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      y[e] = ((sO[0][2 * i + e] + sO[1][2 * i + e]) + (sO[2][2 * i + e] + sO[3][2 * i + e])) * inv;
    reinterpret_cast<uint32_t*>(a.o)[out * (D / 2) + i] = pack2<F16>(y[0], y[1]);
  }
}

template <int D, int KIND, bool F16>
cudaError_t launch(const CacheAttnArgs& a, cudaStream_t st) {
  constexpr int smem = kWarps * 16 * D * 4 + kWarps * 16 * 2 * 4;
  static_assert(smem <= 48 * 1024, "no opt-in needed");
  const int64_t row_tiles = ((int64_t)a.max_tokens * (a.Hq / a.c.heads) + 15) / 16;
  if (row_tiles * a.seqs > 65535) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)a.splits, (unsigned)a.c.heads, (unsigned)(row_tiles * a.seqs));
  cache_attn_kernel<D, KIND, F16><<<grid, kThreads, smem, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.splits == 1) return e;
  // the join may be brought up while the parts run; it waits for them itself
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.n_tok * a.Hq));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_attn_join_kernel<D, F16>, a);
}

template <int D, bool F16>
cudaError_t by_kind(const CacheAttnArgs& a, cudaStream_t st) {
  switch (a.c.kind) {
    case LH_CACHE_E4M3: return launch<D, LH_CACHE_E4M3, F16>(a, st);
    case LH_CACHE_INT8: return launch<D, LH_CACHE_INT8, F16>(a, st);
    default: return launch<D, F16 ? LH_CACHE_FP16 : LH_CACHE_BF16, F16>(a, st);
  }
}

}  // namespace

// Parts of a sequence's keys.  Enough blocks for three on each of the 148 SMs
// (their registers allow three); several sequences have several lengths, and
// four times as many parts even those out.  A part holds at least 256 keys,
// so that joining it costs less than reading it.
void cache_attn_split(int64_t seqs, int64_t kv_heads, int64_t rows, int64_t longest, int* splits, int* chunk) {
  const int64_t base = seqs * kv_heads * ((rows + 15) / 16);
  const int64_t want = 444 * (seqs > 1 ? 4 : 1);
  int64_t n = want / base;
  const int64_t most = (longest + 255) / 256;
  if (n > most) n = most;
  if (n < 1) n = 1;
  const int64_t unit = kWarps * kKeys;
  int64_t c = ((longest + n - 1) / n + unit - 1) / unit * unit;
  if (c < unit) c = unit;
  *chunk = (int)c;
  *splits = (int)((longest + c - 1) / c < 1 ? 1 : (longest + c - 1) / c);
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, int dtype, cudaStream_t st) {
  if (dtype == LH_FP16) return a.c.d == 128 ? by_kind<128, true>(a, st) : by_kind<64, true>(a, st);
  return a.c.d == 128 ? by_kind<128, false>(a, st) : by_kind<64, false>(a, st);
}

}  // namespace lh
