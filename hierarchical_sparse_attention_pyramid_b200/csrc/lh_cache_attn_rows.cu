// Attention over the paged cache for more than 32 query rows of a key head (a
// tree of drafted tokens, several heads a group): tiles of up to 128 rows on
// the tcgen05 tensor cores.
//
// Each key is read and, where the cache holds 8 bits, turned into a 16-bit
// operand once for all 128 rows.  A unit of 128 keys takes 1024 clocks of matrix
// products at 128 channels but about 5500 in all (3 us; one sequence of 256K
// e4m3 tokens, 4 key heads, 96 rows: 188 us against a floor of 42): by the clock
// the converters spend 3300 on a unit's loads and 1300 on its conversion, and a
// softmax of a thread a row 4600, beside one another but in a chain over two
// stages.  Two groups of softmax warps, of converters, or of both (96 registers a thread),
// and K and V freed apart did not shorten it for 8-bit caches; rows staged by
// asynchronous copies two units ahead, with two softmax groups, took 8% off at
// 16 sequences x 8 heads and nothing at 4, and was not kept.
//   warps 0-3   softmax: thread t owns row t (TMEM lane t) and all 128 keys of
//               a unit; they write the Q tile at the start of a piece and the
//               outputs at its end
//   warps 4-7   converters: the unit's K and V rows, each thread some 16-byte
//               units of them, into a 2-stage ring in the layout that the
//               products read (128-byte swizzle): 8-bit ones through registers
//               (loaded one unit ahead), 16-bit ones by asynchronous copies
//   warp 8      MMA issuer: S = Q K^T one unit ahead into one of two TMEM
//               buffers, then O += P V with P over the S columns it came from
// The work list, the fp16 form of 8-bit values and what their scales multiply
// are as in lh_cache_attn.cu: TMEM columns S [0,128) and [128,256), O
// [256,256+D).
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "lh_cache_attn.cuh"

namespace lh {
namespace {
using namespace sm100;

constexpr int kRows = 128;
constexpr int kConvert = 128, kThreads = 128 + kConvert + 32, kWarps = kThreads / 32, kWarpMma = 8;
constexpr int kRegion = 128 * 128;  // one [128 rows][64 x 16 bit] region

template <int D>
struct Smem {
  static constexpr int kTile = D / 64 * kRegion;
  static constexpr int oQ = 0;
  static constexpr int oK = oQ + kTile;      // 2 stages
  static constexpr int oV = oK + 2 * kTile;  // 2 stages
  static constexpr int oScale = oV + 2 * kTile;  // [2 stages][K, V][128] floats; K: negative for a missing key
  static constexpr int oFlag = oScale + 2048;    // [2] whether a key of the stage is missing
  static constexpr int oBar = oFlag + 16;
  static constexpr int kAlloc = oBar + 256 + 1024;
};

// 16 bytes at (row, 16-byte chunk) of a tile as a 128-byte swizzle lays it out
__device__ __forceinline__ uint4* tile_at(uint8_t* tile, int row, int chunk) {
  return reinterpret_cast<uint4*>(tile + (chunk >> 3) * kRegion + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}
__device__ __forceinline__ uint32_t below(int n) {  // bits 0 .. n - 1
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1;
}
__device__ __forceinline__ bool convert_any(bool x) {  // over the converters, which it also synchronises
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

template <int D, int KIND, bool F16>
__global__ void __launch_bounds__(kThreads, 1) cache_attn_rows_kernel(const __grid_constant__ CacheAttnArgs a) {
  using Lay = Smem<D>;
  constexpr bool HELD8 = KIND == LH_CACHE_E4M3 || KIND == LH_CACHE_INT8, HALF = F16 || HELD8;
  constexpr int ROW = D * (HELD8 ? 1 : 2), U = ROW / 16;           // bytes, 16-byte units of a key's row
  constexpr int STEP = kConvert / U, PASS = kUnit / STEP;          // rows that the converters take at once
  constexpr float kPUp = HELD8 ? 64.f : 1.f;  // raises probabilities (at most 2^8) within fp16's range
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ int64_t scan[kWarps + 1];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::oBar);
  uint64_t* bQ = bars + 0;     // Q of a piece written (128 arrivals)
  uint64_t* bFull = bars + 1;  // [2] K, V and scales of a unit written (128 arrivals)
  uint64_t* bFree = bars + 3;  // [2] its products done: the stage is free, O holds its P V.  One barrier a stage, so
                               // that a softmax warp that is a unit ahead of another cannot take the unit before
                               // for its own: bS of unit i comes after the products of unit i - 2
  uint64_t* bS = bars + 5;     // [2] S of a unit in a TMEM buffer
  uint64_t* bP = bars + 7;     // [2] P of a unit in its TMEM buffer, O rescaled (128 arrivals; a warp may be at the
                               // next unit already when another arrives)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::oBar + 192);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::oBar + 196);
  volatile int* flag = reinterpret_cast<volatile int*>(smem + Lay::oFlag);
  float* scales = reinterpret_cast<float*>(smem + Lay::oScale);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.Hq / a.c.heads;
  Stretch stretch = find_stretch<kWarps>(a, kRows, scan);
  if (stretch.u >= stretch.u_end) return;
  Seq seq = load_seq(a, stretch.s, false);
  Piece piece;
  if (threadIdx.x == 0) {
    mbar_init(bQ, 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bFull[i], kConvert);
      mbar_init(&bFree[i], 1);
      mbar_init(&bS[i], 1);
      mbar_init(&bP[i], 128);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int it = 0;  // units so far, over all pieces: ring stage and S buffer it & 1
  bool ok = true;
  // A sequence of length 0 that has query tokens is a piece without keys (always
  // a whole one: its only unit past kBegin).  No role counts a unit for it; the
  // softmax warps write its zeros.
  auto next_with_keys = [&]() -> bool {
    while (next_piece(a, kRows, stretch, seq, piece))
      if (piece.k0 < piece.k1) return true;
    return false;
  };

  if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idQK = idesc16<HALF>(128, 128, false, false);
    constexpr uint32_t idPV = idesc16<HALF>(128, D, false, true);
    const uint64_t kQ = sdesc_sw128(smem_u32(smem + Lay::oQ), 16, 1024);
    const uint64_t kK = sdesc_sw128(smem_u32(smem + Lay::oK), 16, 1024);
    const uint64_t mV = sdesc_sw128(smem_u32(smem + Lay::oV), kRegion, 1024);
    auto issue_s = [&](int i) -> bool {
      if (!mbar_wait_warp(&bFull[i & 1], (i >> 1) & 1, abort_flag)) return false;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * kRegion + (kk & 3) * 32) >> 4;
        umma_bf16_w(tmem + (i & 1) * 128, kQ + off, kK + (((i & 1) * Lay::kTile) >> 4) + off, idQK, kk > 0 ? 1u : 0u);
      }
      umma_commit_w(&bS[i & 1]);
      return true;
    };
    for (int n = 0; ok && next_with_keys(); ++n) {
      ok = mbar_wait_warp(bQ, n & 1, abort_flag) && issue_s(it);
      for (int key = piece.k0; ok && key < piece.k1; key += kUnit, ++it) {
        if (key + kUnit < piece.k1) ok = issue_s(it + 1);
        ok = ok && mbar_wait_warp(&bP[it & 1], (it >> 1) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const int st = it & 1;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_bf16_tmem_a_w(tmem + 256, tmem + st * 128 + kk * 8,
                             mV + ((st * Lay::kTile + kk * 2048) >> 4), idPV, (key > piece.k0 || kk > 0) ? 1u : 0u);
        umma_commit_w(&bFree[st]);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ converters
    const int ct = threadIdx.x - 128, unit = ct % U, row0 = ct / U;
    uint4 kr[HELD8 ? PASS : 1], vr[HELD8 ? PASS : 1];
    float ks = 0.f, vs = 0.f;
    bool missing = false;
    constexpr uint32_t kNone = 0xffffffffu;
    // lane j < 16 looks up the 8 keys from key + 8 j on, one unit ahead of the
    // loads that need them
    auto look_up = [&](int key) -> uint32_t {
      const int kk = key + 8 * lane;
      return lane < 16 && kk < piece.k1 ? key_rows(a, a.table + (int64_t)stretch.s * a.width, piece.hk, kk) : kNone;
    };
    uint32_t rows = kNone;
    // 8 bits: the rows into registers; 16 bits: copies into the stage.  A row
    // past the piece or of a missing page is zeros.
    auto load = [&](int key, uint8_t* kt, uint8_t* vt) {
      const int n = piece.k1 - key;  // keys from here on
      missing = lane < 16 && 8 * lane < n && rows == kNone;
#pragma unroll
      for (int p = 0; p < PASS; ++p) {
        const int row = row0 + p * STEP;
        const uint32_t r = __shfl_sync(0xffffffffu, rows, row >> 3);
        const bool live = r != kNone && row < n;
        const int64_t at = live ? ((int64_t)r + (row & 7)) * ROW + unit * 16 : 0;
        const char* k = static_cast<const char*>(a.c.k) + at;
        const char* v = static_cast<const char*>(a.c.v) + at;
        if constexpr (HELD8) {
          kr[p] = vr[p] = make_uint4(0, 0, 0, 0);
          if (live) {
            kr[p] = __ldcs(reinterpret_cast<const uint4*>(k));
            vr[p] = __ldcs(reinterpret_cast<const uint4*>(v));
          }
        } else {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(tile_at(kt, row, unit))), "l"(k),
                       "r"(live ? 16 : 0)
                       : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(tile_at(vt, row, unit))), "l"(v),
                       "r"(live ? 16 : 0)
                       : "memory");
        }
      }
      // the scales of key ct
      const uint32_t r = __shfl_sync(0xffffffffu, rows, ct >> 3);
      ks = -1.f, vs = 0.f;
      if (r != kNone && ct < n) {
        ks = HELD8 ? __ldg(a.c.k_scale + (int64_t)r + (ct & 7)) : 1.f;
        vs = HELD8 ? __ldg(a.c.v_scale + (int64_t)r + (ct & 7)) : 1.f;
      }
      rows = look_up(key + kUnit);
    };
    bool have = next_with_keys();
    int key = have ? piece.k0 : 0;
    if (have) rows = look_up(key);
    if (HELD8 && have) load(key, nullptr, nullptr);
    for (; have; ++it) {
      const int st = it & 1;
      uint8_t* kt = smem + Lay::oK + st * Lay::kTile;
      uint8_t* vt = smem + Lay::oV + st * Lay::kTile;
      if (it >= 2) ok = __all_sync(0xffffffffu, ok && mbar_wait(&bFree[st], ((it >> 1) - 1) & 1, abort_flag));
      if (!HELD8 && ok) load(key, kt, vt);
      // every converter comes here, also after a failed wait: all of them stop
      // at the same unit, so that none waits at these barriers alone
      if (convert_any(!ok)) break;
      const bool any = convert_any(missing);
      if constexpr (HELD8) {
#pragma unroll
        for (int p = 0; p < PASS; ++p)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint4 u = x ? vr[p] : kr[p];
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
            uint32_t h[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) widen_row<KIND>(w[i], h[2 * i], h[2 * i + 1]);
            uint8_t* tile = x ? vt : kt;
            const int row = row0 + p * STEP;
            *tile_at(tile, row, 2 * unit) = make_uint4(h[0], h[1], h[2], h[3]);
            *tile_at(tile, row, 2 * unit + 1) = make_uint4(h[4], h[5], h[6], h[7]);
          }
      } else {
        asm volatile("cp.async.wait_all;" ::: "memory");
      }
      scales[st * 256 + ct] = ks;
      scales[st * 256 + 128 + ct] = vs;
      if (ct == 0) flag[st] = any;
      fence_proxy_async_smem();  // the tensor core reads the tiles through the async proxy
      mbar_arrive(&bFull[st]);
      key += kUnit;
      if (key >= piece.k1) {
        have = next_with_keys();
        key = piece.k0;
        if (have) rows = look_up(key);
      }
      if (HELD8 && have) load(key, nullptr, nullptr);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int t = threadIdx.x;  // row of the tile
    const uint32_t tl = tmem + ((uint32_t)(warp * 32) << 16), to = tl + 256;
    const bool cap = a.softcap > 0.f;
    const float pre = cap ? a.scale / a.softcap : a.scale * kLog2e, cap2 = a.softcap * kLog2e;
    auto products_done = [&](int i) { return mbar_wait(&bFree[i & 1], (i >> 1) & 1, abort_flag); };
    while (ok && next_piece(a, kRows, stretch, seq, piece)) {
      const int n_rows = seq.T * G, r = piece.rt * kRows + t, ctx = seq.len - seq.T;
      const bool live = r < n_rows;
      const bool idle = piece.rt * kRows + warp * 32 >= n_rows;  // no row of the warp is one
      const int64_t out = live ? (int64_t)(seq.tok0 + r / G) * a.Hq + piece.hk * G + r % G : 0;
      if (piece.k0 >= piece.k1) {
        for (int i = 0; live && i < D / 8; ++i)
          reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + out * D)[i] = make_uint4(0, 0, 0, 0);
        continue;
      }
      // the row of Q, with 8-bit keys times the power of two that brings its
      // largest value to [2^14, 2^15)
      float up = 1.f;
      {
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + (live ? (int64_t)(seq.tok0 + r / G) * a.q_stride[0] +
                                                                              (int64_t)(piece.hk * G + r % G) * a.q_stride[1]
                                                                        : 0);
        uint4 q[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          q[i] = live ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
        if constexpr (HELD8 && !F16) {
          unsigned top = 0;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, w[e] >> 16 & 0x7fffu));
          }
          top >>= 7;  // biased exponent
          up = __uint_as_float(max(1u, min(254u, 268u - min(268u, top))) << 23);
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          if constexpr (HELD8 && !F16) {
            uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = unpack2<false>(w[e]);
              w[e] = pack2<true>(f.x * up, f.y * up);
            }
            q[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          *tile_at(smem + Lay::oQ, t, i) = q[i];
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(bQ);
      const float qf = pre / up;
      const float slope2 = a.slopes && live ? __ldg(a.slopes + piece.hk * G + r % G) * kLog2e : 0.f;
      const int tk = live ? r / G : 0;
      const int limit = live ? (a.tree ? ctx : ctx + tk + 1) : 0;  // keys below are seen
      const uint64_t bits = a.tree && live ? __ldg(reinterpret_cast<const unsigned long long*>(a.tree) + seq.tok0 + tk) : 0;
      float m_run = -INFINITY, l_run = 0.f;
      float v_ref = kLeastScale;  // 8 bits: power of two at or above the value scales so far
      const int first = it;
      for (int key = piece.k0; key < piece.k1; key += kUnit, ++it) {
        const int st = it & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(&bFull[st], (it >> 1) & 1, abort_flag) &&
                                         mbar_wait(&bS[st], (it >> 1) & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        if (idle) {
          tc_fence_before();
          mbar_arrive(&bP[st]);
          continue;
        }
        const uint32_t ts = tl + st * 128;
        const float* ks = scales + st * 256;
        const float* vs = ks + 128;
        const bool gaps = flag[st];
        const bool edge = key + kUnit > (a.tree ? ctx : ctx + 1) || key + kUnit > piece.k1 || gaps;
        // exponents of two over the scores, half of the keys at a time (a loop,
        // not unrolled: its code is what the warps would wait for)
        uint32_t s[2][32];
        float mx = -INFINITY;
#pragma unroll 1
        for (int hh = 0; hh < 2; ++hh) {
          tmem_ld32(ts + hh * 64, s[0]);
          tmem_ld32(ts + hh * 64 + 32, s[1]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int col = hh * 64 + c * 32;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              float f[4] = {qf, qf, qf, qf};
              if constexpr (HELD8) {
                const float4 k4 = *reinterpret_cast<const float4*>(ks + col + i);
                f[0] *= k4.x, f[1] *= k4.y, f[2] *= k4.z, f[3] *= k4.w;
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) s[c][i + e] = __float_as_uint(__uint_as_float(s[c][i + e]) * f[e]);
            }
            if (cap) {
              cap_scores(s[c], 1.f);
#pragma unroll
              for (int i = 0; i < 32; ++i) s[c][i] = __float_as_uint(__uint_as_float(s[c][i]) * cap2);
            }
            if (a.slopes) {
              const float d0 = (float)(ctx + tk - key - col);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                s[c][i] = __float_as_uint(fmaf(-slope2, fabsf(d0 - (float)i), __uint_as_float(s[c][i])));
            }
            if (edge) {
              // bit i: key + col + i is seen
              uint32_t seen = below(min(limit, piece.k1) - key - col);
              if (a.tree) {
                const int at = ctx - key - col;  // of the first drafted token
                const uint64_t drafted = at >= 0 ? (at < 32 ? bits << at : 0) : (at > -64 ? bits >> -at : 0);
                seen |= (uint32_t)drafted & ~below(at) & below(piece.k1 - key - col);
              }
              if (gaps) seen &= ~__ballot_sync(0xffffffffu, ks[col + lane] < 0.f);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!(seen >> i & 1)) s[c][i] = __float_as_uint(-INFINITY);
            }
#pragma unroll
            for (int i = 0; i < 32; i += 2) mx = max3f(mx, __uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1]));
            tmem_st32(ts + col, s[c]);
          }
        }
        tmem_st_wait();
        // the reference moves only when the maximum exceeds it by more than 8
        const bool move = mx > m_run + 8.f;
        const float m_new = move ? mx : m_run;
        float alpha = move ? fast_exp2(m_run - m_new) : 1.f;
        const float m_ref = m_new == -INFINITY ? 0.f : m_new;
        l_run *= alpha;
        m_run = m_new;
        float vf = 1.f;
        bool lift = false;
        if constexpr (HELD8) {
          const float4 v4 = *reinterpret_cast<const float4*>(vs + lane * 4);
          const unsigned top =
              __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(0.f, fmaxf(fmaxf(v4.x, v4.y), fmaxf(v4.z, v4.w)))));
          lift = __uint_as_float(top) > v_ref;
          if (lift) {
            const float up_v = scale_above(top);
            alpha *= v_ref / up_v;
            v_ref = up_v;
          }
          vf = __uint_as_float(0x7f000000u - __float_as_uint(v_ref)) * kPUp;
        }
        if (it > first && __any_sync(0xffffffffu, move || lift)) {  // O, once the previous P V has added to it
          ok = __all_sync(0xffffffffu, products_done(it - 1));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ++ch) {
            uint32_t o[32];
            tmem_ld32(to + ch * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(to + ch * 32, o);
          }
        }
        float sum[2] = {0.f, 0.f};
        auto p_chunk = [&](uint32_t (&x)[32], int col, uint32_t dst) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = fast_exp2(__uint_as_float(x[i + e]) - m_ref);
            sum[0] += p[0] + p[1];
            sum[1] += p[2] + p[3];
            if constexpr (HELD8) {
              const float4 v4 = *reinterpret_cast<const float4*>(vs + col + i);
              p[0] *= v4.x * vf, p[1] *= v4.y * vf, p[2] *= v4.z * vf, p[3] *= v4.w * vf;
            }
            pk[i / 2] = pack2<HALF>(p[0], p[1]);
            pk[i / 2 + 1] = pack2<HALF>(p[2], p[3]);
          }
          tmem_st16(dst, pk);
        };
        // P over the first half of the S columns
#pragma unroll 1
        for (int hh = 0; hh < 2; ++hh) {
          tmem_ld32(ts + hh * 64, s[0]);
          tmem_ld32(ts + hh * 64 + 32, s[1]);
          tmem_ld_wait();
          p_chunk(s[0], hh * 64, ts + hh * 32);
          p_chunk(s[1], hh * 64 + 32, ts + hh * 32 + 16);
        }
        l_run += sum[0] + sum[1];
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bP[st]);
      }
      if (ok) ok = __all_sync(0xffffffffu, products_done(it - 1));
      if (!ok) break;
      tc_fence_after();
      if (!idle) {
        const float back = HELD8 ? v_ref / kPUp : 1.f;
        const float f = !piece.whole ? back : l_run > 0.f || l_run != l_run ? back / l_run : 0.f;
        const int64_t at = ((int64_t)blockIdx.x * 2 + piece.begun) * kRows + t;
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t o[32];
          tmem_ld32(to + ch * 32, o);
          tmem_ld_wait();
          if (!live) continue;
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = f == 0.f ? 0.f : __uint_as_float(o[i + e]) * f;
            if (piece.whole) {
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + out * D + ch * 32 + i) =
                  make_uint4(pack2<F16>(y[0], y[1]), pack2<F16>(y[2], y[3]), pack2<F16>(y[4], y[5]), pack2<F16>(y[6], y[7]));
            } else {
              float4* dst = reinterpret_cast<float4*>(a.part_o + at * D + ch * 32 + i);
              dst[0] = make_float4(y[0], y[1], y[2], y[3]);
              dst[1] = make_float4(y[4], y[5], y[6], y[7]);
            }
          }
        }
        if (live && !piece.whole) a.part_ml[at] = make_float2(m_run, l_run);
      }
      tc_fence_before();  // the next piece's products overwrite O after its P arrives
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag) report_error(a.errw, ERRW_TIMEOUT);
}

template <int D, int KIND, bool F16>
cudaError_t launch(const CacheAttnArgs& a, cudaStream_t st) {
  auto* fn = cache_attn_rows_kernel<D, KIND, F16>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kAlloc);
  if (e != cudaSuccess) return e;
  fn<<<dim3((unsigned)a.blocks), kThreads, Smem<D>::kAlloc, st>>>(a);
  return cudaGetLastError();
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

cudaError_t launch_cache_attn_rows(const CacheAttnArgs& a, int dtype, cudaStream_t st) {
  if (dtype == LH_FP16) return a.c.d == 128 ? by_kind<128, true>(a, st) : by_kind<64, true>(a, st);
  return a.c.d == 128 ? by_kind<128, false>(a, st) : by_kind<64, false>(a, st);
}

}  // namespace lh
