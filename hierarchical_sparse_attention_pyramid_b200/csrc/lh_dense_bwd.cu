// Masked dense attention, backward.  With P recomputed from LSE,
//   dV = P^T dO,  dP = dO V^T,  dS = P (dP - Delta) (1 - tanh^2),
//   dQ = scale dS K,  dK = scale dS^T Q,  Delta = rowsum(dO * O),
// dK and dV summed over the query heads that share a key head (1 - tanh^2 is
// the derivative of the cap; 1 without one).
//
// Two kernels, each writing its gradients once, so that no sum depends on the
// order in which CTAs finish (a single kernel, 5 instead of 7 matrix products a
// tile, would add dQ up across CTAs, in any order by atomics or in a fixed one
// by waiting for turns; the latter has not been built):
//
// dense_bwd_q_kernel (Delta, dQ) - one CTA per 128-query tile and query head;
//   S = Q K_j^T runs two key tiles ahead into a double-buffered TMEM region
//   and dP = dO V_j^T one tile ahead; dS goes back over the S columns and
//   dQ += dS K_j reads it there.  It computes Delta first and leaves it for
//   the other kernel.
// dense_bwd_kv_kernel (dK, dV) - one CTA per 128-key tile and key head; it
//   steps over the query tiles that see the key tile, for each query head of
//   the group.  S^T = K Q_j^T and dP^T = V dO_j^T; P^T and dS^T go back over
//   the columns they were read from, and dV += P^T dO_j and dK += dS^T Q_j
//   read them there.  Where there are few key tiles, the CTAs of a cluster
//   share the steps of one and add their sums up in rank order.
//
// P and dS enter their products in the inputs' 16-bit type: each rounding is
// half a step relative to its own value and they are averaged over a row's
// keys (a column's queries), so that they stay below the rounding of the
// gradients themselves.  The score scale is left out of dS and applied to the
// fp32 sums: with fp16 that keeps small dS out of the subnormal range.
//
// Bound by the tensor cores: 16K causal tokens, 8 heads of 128: 590 us for dQ's
// three products (1.40 PFLOP/s) and 840 us for the other four (1.31), near the
// 1.37 that a long product of large matrices sustains under the power limit.
#include <type_traits>

#include "lh_dense.cuh"

namespace lh {
namespace {
using namespace sm100;

constexpr int kCompute = 256;    // dQ kernel: two compute warpgroups
constexpr int kThreads = kCompute + 64;
constexpr int kComputeKV = 512;  // dK/dV kernel: four compute warpgroups
constexpr int kThreadsKV = kComputeKV + 64;
constexpr int kRegion = 128 * 128;  // one [128 rows][64 x 16 bit] region

__device__ __forceinline__ void compute_sync_kv() { asm volatile("bar.sync 1, 512;" ::: "memory"); }
// every thread of every CTA of the cluster; shared memory written before is visible after
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// four floats at this CTA's shared address `at` in the CTA of a rank
__device__ __forceinline__ float4 ld_cluster(uint32_t at, int rank) {
  float4 v;
  uint32_t peer;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(peer)
               : "memory");
  return v;
}
__device__ __forceinline__ void compute_sync_q() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// exponents of two of a pair of turned scores, less LSE; d0, d1: distances
__device__ __forceinline__ void exponents(const Mod& m, float t0, float t1, float l0, float l1, float d0, float d1,
                                          float& x0, float& x1) {
  f2_unpack(f2_fma(f2_pack(t0, t1), f2_pack(m.mul, m.mul), f2_pack(-l0, -l1)), x0, x1);
  if (m.bias) {
    x0 = fmaf(-m.slope2, fabsf(d0), x0);
    x1 = fmaf(-m.slope2, fabsf(d1), x1);
  }
}

// ===========================================================================
// dK, dV
// ===========================================================================
// The tiles fill the shared memory of a CTA without slack to align them, so
// the kernel relies on dynamic shared memory starting 1024-byte aligned (it
// has no static shared memory) and checks that it does.
template <int D>
struct KvSmem {
  static constexpr int kTile = D / 64 * kRegion;
  static constexpr int oK = 0;
  static constexpr int oV = oK + kTile;
  static constexpr int oQ = oV + kTile;        // 3 slots of Q_j
  static constexpr int oO = oQ + 3 * kTile;    // 2 slots of dO_j
  static constexpr int oVec = oO + 2 * kTile;  // [2][256] floats: LSE * log2e [128], Delta [128]
  static constexpr int oBar = oVec + 2048;
  static constexpr int kAlloc = oBar + 256;
  static constexpr int kSumRow = D + 4;        // floats of a row of dV or dK laid over the tiles (padded: 16-byte
                                               // stores of neighbouring rows meet different banks)
  static_assert(2 * 128 * kSumRow * 4 <= oVec, "the sums fit over the tiles");
};

template <int D, bool F16, bool MOD>
__global__ void __launch_bounds__(kThreadsKV, 1)
    dense_bwd_kv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                        const __grid_constant__ DenseArgs a, void* __restrict__ dK, const Strides sdk,
                        void* __restrict__ dV, const Strides sdv, const int C) {
  using Lay = KvSmem<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (reinterpret_cast<uintptr_t>(smem_raw) & 1023) {
    if (threadIdx.x == 0) report_error(a.errw, ERRW_BOUNDS);
    return;
  }
  uint8_t* smem = smem_raw;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::oBar);
  uint64_t* bKV = bars + 0;     // K, V landed
  uint64_t* bQload = bars + 1;  // [3] Q_j of a slot landed
  uint64_t* bQfree = bars + 4;  // [3] dK product done with a Q slot
  uint64_t* bOload = bars + 7;  // [2] dO_j of a slot landed
  uint64_t* bOfree = bars + 9;  // [2] dV product done with a dO slot
  uint64_t* bS = bars + 11;     // S^T of the step in TMEM
  uint64_t* bDP = bars + 12;    // dP^T of the step in TMEM
  uint64_t* bP = bars + 13;     // P^T written back (512 arrivals)
  uint64_t* bDS = bars + 14;    // dS^T written back (512 arrivals)
  uint64_t* bDone = bars + 15;  // every product done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::oBar + 192);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::oBar + 196);
  float* sVec = reinterpret_cast<float*>(smem + Lay::oVec);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // key-tile-major grid: with a causal mask the first key tiles are seen by
  // the most queries, and the short ones fill the tail
  const int BH = a.B * a.Hkv, G = a.Hq / a.Hkv;
  const int rank = (int)(blockIdx.x % (unsigned)C), tile = (int)(blockIdx.x / (unsigned)C);
  const int kt = tile / BH;
  const int bh = tile % BH;
  const int b = bh / a.Hkv, hk = bh % a.Hkv;
  const TileSpan span = mask_col_tile(a.mask, b, kt, a.N);
  const int q0 = span.min_lo >> 7;
  const int nq = span.max_hi > span.min_lo ? ((span.max_hi + 127) >> 7) - q0 : 0;
  // step i of the tile: query head hk * G + i / nq, query tile q0 + i % nq;
  // this CTA of the cluster takes the steps [i0, i0 + NJ)
  const int i0 = (int)((int64_t)nq * G * rank / C), NJ = (int)((int64_t)nq * G * (rank + 1) / C) - i0;
  const int h_first = hk * G + (nq ? i0 / nq : 0), qt_first = q0 + (nq ? i0 % nq : 0);

  if (threadIdx.x == 0) {
    mbar_init(bKV, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&bQload[i], 1);
      mbar_init(&bQfree[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bOload[i], 1);
      mbar_init(&bOfree[i], 1);
    }
    mbar_init(bS, 1);
    mbar_init(bDP, 1);
    mbar_init(bP, kComputeKV);
    mbar_init(bDS, kComputeKV);
    mbar_init(bDone, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 17) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  constexpr uint32_t tS = 0, tDP = 128, tDV = 256, tDK = 256 + D;

  if (warp == 16) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0 && NJ > 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmO);
      mbar_expect_tx(bKV, 2 * 128 * D * 2);
      for (int c = 0; c < D / 64; ++c) {
        tma_load_4d(smem + Lay::oK + c * kRegion, &tmK, bKV, c * 64, kt * 128, hk, b);
        tma_load_4d(smem + Lay::oV + c * kRegion, &tmV, bKV, c * 64, kt * 128, hk, b);
      }
      int h = h_first, qt = qt_first;
      for (int j = 0; j < NJ; ++j) {
        const int qs = j % 3, os = j & 1;
        if (j >= 3 && !mbar_wait(&bQfree[qs], ((j / 3) - 1) & 1, abort_flag)) break;
        mbar_expect_tx(&bQload[qs], 128 * D * 2);
        for (int c = 0; c < D / 64; ++c)
          tma_load_4d(smem + Lay::oQ + qs * Lay::kTile + c * kRegion, &tmQ, &bQload[qs], c * 64, qt * 128, h, b);
        if (j >= 2 && !mbar_wait(&bOfree[os], ((j >> 1) - 1) & 1, abort_flag)) break;
        mbar_expect_tx(&bOload[os], 128 * D * 2);
        for (int c = 0; c < D / 64; ++c)
          tma_load_4d(smem + Lay::oO + os * Lay::kTile + c * kRegion, &tmO, &bOload[os], c * 64, qt * 128, h, b);
        if (++qt == q0 + nq) {
          qt = q0;
          ++h;
        }
      }
    }
  } else if (warp == 17) {
    // ------------------------------------------------------------ MMA issuer
    // Order per step j: dV(j) once P^T(j) is back, S^T(j+1) (over the P^T
    // columns dV(j) has read: the tensor core runs in issue order), dK(j) once
    // dS^T(j) is back, dP^T(j+1) (over the dS^T columns dK(j) has read).
    if (NJ > 0) {  // the whole warp; one elected lane issues each instruction
      constexpr uint32_t idF = idesc16<F16>(128, 128, false, false);
      constexpr uint32_t idG = idesc16<F16>(128, D, false, true);
      const uint32_t sQ = smem_u32(smem + Lay::oQ), sO = smem_u32(smem + Lay::oO);
      const uint64_t kK = sdesc_sw128(smem_u32(smem + Lay::oK), 16, 1024);
      const uint64_t kV = sdesc_sw128(smem_u32(smem + Lay::oV), 16, 1024);
      const uint64_t kQ = sdesc_sw128(sQ, 16, 1024), mQ = sdesc_sw128(sQ, kRegion, 1024);
      const uint64_t kO = sdesc_sw128(sO, 16, 1024), mO = sdesc_sw128(sO, kRegion, 1024);
      auto wait_q = [&](int j) -> bool { return mbar_wait_warp(&bQload[j % 3], (j / 3) & 1, abort_flag); };
      auto wait_o = [&](int j) -> bool { return mbar_wait_warp(&bOload[j & 1], (j >> 1) & 1, abort_flag); };
      auto issue_s = [&](int j) {
        const uint32_t qo = ((j % 3) * Lay::kTile) >> 4;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t at = ((kk >> 2) * kRegion + (kk & 3) * 32) >> 4;
          umma_bf16_w(tmem + tS, kK + at, kQ + qo + at, idF, kk > 0 ? 1u : 0u);
        }
        umma_commit_w(bS);
      };
      auto issue_dp = [&](int j) {
        const uint32_t oo = ((j & 1) * Lay::kTile) >> 4;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t at = ((kk >> 2) * kRegion + (kk & 3) * 32) >> 4;
          umma_bf16_w(tmem + tDP, kV + at, kO + oo + at, idF, kk > 0 ? 1u : 0u);
        }
        umma_commit_w(bDP);
      };
      bool ok = mbar_wait_warp(bKV, 0, abort_flag) && wait_q(0);
      if (ok) {
        tc_fence_after();
        issue_s(0);
        ok = wait_o(0);
      }
      if (ok) {
        tc_fence_after();
        issue_dp(0);
      }
      for (int j = 0; ok && j < NJ; ++j) {
        const uint32_t qo = ((j % 3) * Lay::kTile) >> 4, oo = ((j & 1) * Lay::kTile) >> 4;
        if (!mbar_wait_warp(bP, j & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // dV += P^T dO_j
          umma_bf16_tmem_a_w(tmem + tDV, tmem + tS + (kk >> 1) * 32 + (kk & 1) * 8, mO + oo + ((kk * 2048) >> 4), idG,
                             (j > 0 || kk > 0) ? 1u : 0u);
        umma_commit_w(&bOfree[j & 1]);  // dV(j) was the last reader of dO_j
        if (j + 1 < NJ) {
          if (!wait_q(j + 1)) { ok = false; break; }
          tc_fence_after();
          issue_s(j + 1);
        }
        if (!mbar_wait_warp(bDS, j & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // dK += dS^T Q_j
          umma_bf16_tmem_a_w(tmem + tDK, tmem + tDP + (kk >> 1) * 32 + (kk & 1) * 8, mQ + qo + ((kk * 2048) >> 4), idG,
                             (j > 0 || kk > 0) ? 1u : 0u);
        umma_commit_w(&bQfree[j % 3]);  // dK(j) was the last reader of Q_j
        if (j + 1 < NJ) {
          if (!wait_o(j + 1)) { ok = false; break; }
          tc_fence_after();
          issue_dp(j + 1);
        }
      }
      if (ok) umma_commit_w(bDone);
    }
  } else {
    // ------------------------------------------------------------ compute warpgroups
    const int ct = threadIdx.x;            // 0..511
    const int g = warp >> 2;               // query columns [32g, 32g+32) of each step
    const int t = (warp & 3) * 32 + lane;  // key row of the tile (TMEM lane)
    const int kv = kt * 128 + t;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int2 seen = mask_col(a.mask, b, kv, a.N);
    const bool pads = has_padding(a.mask, b);
    const unsigned len = (unsigned)max(0, seen.y - seen.x);
    bool ok = true;
    // LSE (ct < 128) or Delta (128 <= ct < 256) of query row ct & 127 of a
    // step, loaded one step ahead
    auto vec_raw = [&](int h, int qt) -> float {
      const int q = qt * 128 + (ct & 127);
      return q < a.N ? ldg_nc_f32((ct < 128 ? a.lse : a.delta) + ((int64_t)b * a.Hq + h) * a.N + q) : -INFINITY;
    };
    int h = h_first, qt = qt_first;
    float vec_next = ct < 256 && NJ > 0 ? vec_raw(h, qt) : 0.f;
    const float scale_log2 = a.scale * kLog2e;
    const uint64_t c2 = f2_pack(scale_log2, scale_log2);
    Mod mod = MOD ? make_mod(a, h) : Mod{};
    for (int j = 0; j < NJ; ++j) {
      const int buf = j & 1;
      const int qb = qt * 128;
      const bool full = qb >= span.max_lo && qb + 128 <= span.min_hi;
      if (MOD && a.slopes) mod.slope2 = a.slopes[h] * kLog2e;
      if (++qt == q0 + nq) {
        qt = q0;
        ++h;
      }
      const float cur = vec_next;
      if (ct < 256 && j + 1 < NJ) vec_next = vec_raw(h, qt);
      // a query without a key (LSE = -inf) or past N gets P = 2^-inf = 0
      if (ct < 128) sVec[buf * 256 + ct] = cur == -INFINITY ? INFINITY : cur * kLog2e;
      else if (ct < 256) sVec[buf * 256 + ct] = cur == -INFINITY ? 0.f : cur;
      compute_sync_kv();
      const float* lse = sVec + buf * 256;
      const float* del = lse + 128;
      // warp-uniform outcome for the collective TMEM accesses; after a failed
      // wait the loop keeps its compute_sync_kv count and skips the work
      ok = __all_sync(0xffffffffu, ok && mbar_wait(bS, j & 1, abort_flag));
      if (!ok) continue;
      tc_fence_after();
      float p[32];  // P, times the cap's derivative after P^T is stored
      const int lo = seen.x - qb;
      const bool pad = pads && !full && empty_queries(a.mask, b, qb >> 7, a.N);
      if (pad) {
        // padding queries of Q_j (for dK) and dO_j (for dV): warpgroups 0, 1
        // and 2, 3 take a half of the channels each
        ok = __all_sync(0xffffffffu, mbar_wait(&bOload[j & 1], (j >> 1) & 1, abort_flag));
        if (!ok) continue;
        const int2 k = mask_row(a.mask, b, qb + t, a.N);
        if (k.y <= k.x && (g & 1) * 64 < D)
          zero_row(smem + (g < 2 ? Lay::oQ + (j % 3) * Lay::kTile : Lay::oO + (j & 1) * Lay::kTile), t, g & 1, 1);
        fence_proxy_async_smem();
      }
      {
        uint32_t sr[32];
        tmem_ld32(tl + tS + g * 32, sr);
        tmem_ld_wait();
        if (MOD && mod.cap) cap_scores(sr, mod.pre);
        uint32_t ph[16];
        auto p_pass = [&](auto masked) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const int qi = g * 32 + e;
            const float2 l2 = *reinterpret_cast<const float2*>(lse + qi);
            float pa, pb;
            if constexpr (MOD) {
              const float dist = (float)(qb + qi - kv);
              exponents(mod, __uint_as_float(sr[e]), __uint_as_float(sr[e + 1]), l2.x, l2.y, dist, dist + 1.f, pa, pb);
            } else {
              f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), c2, f2_pack(-l2.x, -l2.y)),
                        pa, pb);
            }
            pa = fast_exp2(pa);
            pb = fast_exp2(pb);
            if constexpr (decltype(masked)::value) {
              pa = (unsigned)(qi - lo) < len ? pa : 0.f;
              pb = (unsigned)(qi + 1 - lo) < len ? pb : 0.f;
            }
            ph[e >> 1] = pack2<F16>(pa, pb);
            p[e] = pa;
            p[e + 1] = pb;
          }
        };
        if (full) p_pass(std::false_type{});
        else p_pass(std::true_type{});
        tmem_st16(tl + tS + g * 32, ph);
        if (MOD && mod.cap) {  // times 1 - tanh^2
#pragma unroll
          for (int e = 0; e < 32; ++e) p[e] = fmaf(-p[e] * __uint_as_float(sr[e]), __uint_as_float(sr[e]), p[e]);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bP);
      ok = __all_sync(0xffffffffu, mbar_wait(bDP, j & 1, abort_flag));
      if (!ok) continue;
      tc_fence_after();
      {
        uint32_t dr[32];
        tmem_ld32(tl + tDP + g * 32, dr);
        tmem_ld_wait();
        if (pad) {  // scores and dP of padding queries may be anything
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if ((unsigned)(g * 32 + e - lo) >= len) p[e] = 0.f, dr[e] = 0u;
        }
        uint32_t dh[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 d2 = *reinterpret_cast<const float2*>(del + g * 32 + e);
          const uint64_t diff = f2_sub(f2_pack(__uint_as_float(dr[e]), __uint_as_float(dr[e + 1])), f2_pack(d2.x, d2.y));
          float da, db;
          f2_unpack(f2_mul(f2_pack(p[e], p[e + 1]), diff), da, db);
          dh[e >> 1] = pack2<F16>(da, db);
        }
        tmem_st16(tl + tDP + g * 32, dh);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bDS);
    }
    // dV and dK of this thread's key row, columns [g D/4, (g+1) D/4)
    if (NJ > 0) ok = __all_sync(0xffffffffu, ok && mbar_wait(bDone, 0, abort_flag));
    if (ok) {
      tc_fence_after();
      constexpr int CW = D / 4;
      uint32_t rv[CW], rk[CW];
      if (NJ > 0) {
        if constexpr (CW == 32) {
          tmem_ld32(tl + tDV + g * CW, rv);
          tmem_ld32(tl + tDK + g * CW, rk);
        } else {
          tmem_ld16(tl + tDV + g * CW, rv);
          tmem_ld16(tl + tDK + g * CW, rk);
        }
        tmem_ld_wait();
      }
      if (NJ == 0 || len == 0) {  // a padding key's sums may be anything
#pragma unroll
        for (int e = 0; e < CW; ++e) rv[e] = rk[e] = 0u;
      }
      if (C > 1) {  // over the tiles, which no product or copy uses any more
        float* row = reinterpret_cast<float*>(smem) + t * Lay::kSumRow + g * CW;
#pragma unroll
        for (int e = 0; e < CW; e += 4) {
          *reinterpret_cast<uint4*>(row + e) = make_uint4(rv[e], rv[e + 1], rv[e + 2], rv[e + 3]);
          *reinterpret_cast<uint4*>(row + 128 * Lay::kSumRow + e) = make_uint4(rk[e], rk[e + 1], rk[e + 2], rk[e + 3]);
        }
      } else if (kv < a.N) {
        uint4* dv4 = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(dV) + b * sdv.b + hk * sdv.h +
                                              (int64_t)kv * sdv.n + g * CW);
        uint4* dk4 = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(dK) + b * sdk.b + hk * sdk.h +
                                              (int64_t)kv * sdk.n + g * CW);
#pragma unroll
        for (int q = 0; q < CW / 8; ++q) {
          uint32_t wv[4], wk[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            wv[e] = pack2<F16>(__uint_as_float(rv[8 * q + 2 * e]), __uint_as_float(rv[8 * q + 2 * e + 1]));
            wk[e] = pack2<F16>(__uint_as_float(rk[8 * q + 2 * e]) * a.scale,
                               __uint_as_float(rk[8 * q + 2 * e + 1]) * a.scale);
          }
          dv4[q] = make_uint4(wv[0], wv[1], wv[2], wv[3]);
          dk4[q] = make_uint4(wk[0], wk[1], wk[2], wk[3]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag) report_error(a.errw, ERRW_TIMEOUT);
  if (C > 1) {
    // the cluster's CTAs share out the tile's rows: each sums its rows of dV
    // and dK over the others' shared memory, in rank order
    cluster_sync();
    const int rows = 128 / C;
    constexpr int Q = D / 4;  // float4s of a row
    for (int i = threadIdx.x; i < 2 * rows * Q; i += kThreadsKV) {
      const int which = i / (rows * Q), r = rank * rows + i / Q % rows, c4 = i % Q * 4;
      const uint32_t at = smem_u32(smem) + (uint32_t)((which * 128 + r) * Lay::kSumRow + c4) * 4;
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      for (int p = 0; p < C; ++p) {
        const float4 y = ld_cluster(at, p);
        x[0] += y.x, x[1] += y.y, x[2] += y.z, x[3] += y.w;
      }
      const int kv = kt * 128 + r;
      if (kv < a.N) {
        const Strides& sd = which ? sdk : sdv;
        const float f = which ? a.scale : 1.f;
        uint16_t* dst = reinterpret_cast<uint16_t*>(which ? dK : dV) + b * sd.b + hk * sd.h + (int64_t)kv * sd.n + c4;
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<F16>(x[0] * f, x[1] * f), pack2<F16>(x[2] * f, x[3] * f));
      }
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
  }
}

// ===========================================================================
// Delta, dQ
// ===========================================================================
template <int D>
struct QSmem {
  static constexpr int kTile = D / 64 * kRegion;
  static constexpr int oQ = 0;
  static constexpr int oO = oQ + kTile;      // dO
  static constexpr int oK = oO + kTile;      // 3 stages: K_j is read by S(j) two steps before dQ(j)
  static constexpr int oV = oK + 3 * kTile;  // 2 stages
  static constexpr int oDel = oV + 2 * kTile;  // [2][128] floats
  static constexpr int oBar = oDel + 1024;
  static constexpr int kAlloc = oBar + 256 + 1024;
};

template <int D, bool F16, bool MOD>
__global__ void __launch_bounds__(kThreads, 1)
    dense_bwd_q_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                       const __grid_constant__ DenseArgs a, const void* __restrict__ O, const Strides so,
                       const void* __restrict__ Olow, void* __restrict__ dQ, const Strides sdq) {
  using Lay = QSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::oBar);
  uint64_t* bQO = bars + 0;       // Q, dO landed
  uint64_t* bK = bars + 1;        // [3] K tile of a stage landed
  uint64_t* bV = bars + 4;        // [2] V tile of a stage landed
  uint64_t* bKfree = bars + 6;    // [3] the dQ product is done with a K stage
  uint64_t* bVfree = bars + 9;    // [2] the dP product is done with a V stage
  uint64_t* bS = bars + 11;       // [2] S of a key tile in TMEM buffer
  uint64_t* bDPread = bars + 13;  // dP of the key tile is in registers (256 arrivals)
  uint64_t* bDP = bars + 15;      // dP of the current key tile in TMEM
  uint64_t* bPS = bars + 16;      // dS written over the tile's S columns (256 arrivals)
  uint64_t* bDone = bars + 17;    // every product done
  uint64_t* bDel = bars + 18;     // O and O_low read (256 arrivals)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::oBar + 192);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::oBar + 196);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int BH = a.B * a.Hq;
  const int qt = a.n_tiles - 1 - (int)(blockIdx.x / (unsigned)BH);  // tile-major, last (longest causal) rows first
  const int bh = (int)(blockIdx.x % (unsigned)BH);
  const int b = bh / a.Hq, h = bh % a.Hq, hk = h / (a.Hq / a.Hkv);
  const TileSpan span = mask_row_tile(a.mask, b, qt, a.N);
  const int k0 = span.min_lo >> 7;
  const int NJ = span.max_hi > span.min_lo ? ((span.max_hi + 127) >> 7) - k0 : 0;

  if (threadIdx.x == 0) {
    mbar_init(bQO, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&bK[i], 1);
      mbar_init(&bKfree[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bV[i], 1);
      mbar_init(&bVfree[i], 1);
      mbar_init(&bS[i], 1);
    }
    mbar_init(bDPread, kCompute);
    mbar_init(bDP, 1);
    mbar_init(bPS, kCompute);
    mbar_init(bDone, 1);
    mbar_init(bDel, kCompute);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  constexpr uint32_t tS = 0, tDP = 256, tDQ = 384;  // S, then dS: [2] x 128 columns; dP: 128

  if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0 && NJ > 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      mbar_expect_tx(bQO, 2 * 128 * D * 2);
      for (int c = 0; c < D / 64; ++c) {
        tma_load_4d(smem + Lay::oQ + c * kRegion, &tmQ, bQO, c * 64, qt * 128, h, b);
        tma_load_4d(smem + Lay::oO + c * kRegion, &tmO, bQO, c * 64, qt * 128, h, b);
      }
      for (int j = 0; j < NJ; ++j) {
        const int sk = j % 3, sv = j & 1;
        if (j >= 3 && !mbar_wait(&bKfree[sk], ((j / 3) - 1) & 1, abort_flag)) break;
        mbar_expect_tx(&bK[sk], 128 * D * 2);
        for (int c = 0; c < D / 64; ++c)
          tma_load_4d(smem + Lay::oK + sk * Lay::kTile + c * kRegion, &tmK, &bK[sk], c * 64, (k0 + j) * 128, hk, b);
        if (j == 1 && !mbar_wait(bDel, 0, abort_flag)) break;  // O and O_low are out of the last stages
        if (j >= 2 && !mbar_wait(&bVfree[sv], ((j >> 1) - 1) & 1, abort_flag)) break;
        mbar_expect_tx(&bV[sv], 128 * D * 2);
        for (int c = 0; c < D / 64; ++c)
          tma_load_4d(smem + Lay::oV + sv * Lay::kTile + c * kRegion, &tmV, &bV[sv], c * 64, (k0 + j) * 128, hk, b);
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    // Per key tile j: dP(j+1) as soon as the compute warps hold dP(j) in
    // registers, then dQ += dS(j) K_j once dS(j) is written over tile j's S
    // columns, then S(j+2) into that S buffer (after dQ(j) has read it: the
    // tensor core runs in issue order).
    if (NJ > 0) {  // the whole warp; one elected lane issues each instruction
      constexpr uint32_t idF = idesc16<F16>(128, 128, false, false);
      constexpr uint32_t idG = idesc16<F16>(128, D, false, true);
      const uint64_t kQ = sdesc_sw128(smem_u32(smem + Lay::oQ), 16, 1024);
      const uint64_t kO = sdesc_sw128(smem_u32(smem + Lay::oO), 16, 1024);
      const uint64_t kK = sdesc_sw128(smem_u32(smem + Lay::oK), 16, 1024);
      const uint64_t kV = sdesc_sw128(smem_u32(smem + Lay::oV), 16, 1024);
      const uint64_t mK = sdesc_sw128(smem_u32(smem + Lay::oK), kRegion, 1024);
      auto issue_s = [&](int j) {
        const uint32_t ko = ((j % 3) * Lay::kTile) >> 4;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kRegion + (kk & 3) * 32) >> 4;
          umma_bf16_w(tmem + tS + (j & 1) * 128, kQ + off, kK + ko + off, idF, kk > 0 ? 1u : 0u);
        }
        umma_commit_w(&bS[j & 1]);
      };
      auto issue_dp = [&](int j) {
        const uint32_t vo = ((j & 1) * Lay::kTile) >> 4;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kRegion + (kk & 3) * 32) >> 4;
          umma_bf16_w(tmem + tDP, kO + off, kV + vo + off, idF, kk > 0 ? 1u : 0u);
        }
        umma_commit_w(bDP);
        umma_commit_w(&bVfree[j & 1]);
      };
      bool ok = mbar_wait_warp(bQO, 0, abort_flag) && mbar_wait_warp(&bK[0], 0, abort_flag);
      if (ok) {
        tc_fence_after();
        issue_s(0);
        ok = mbar_wait_warp(&bV[0], 0, abort_flag);
      }
      if (ok) {
        tc_fence_after();
        issue_dp(0);
        if (NJ > 1 && (ok = mbar_wait_warp(&bK[1], 0, abort_flag))) {
          tc_fence_after();
          issue_s(1);
        }
      }
      for (int j = 0; ok && j < NJ; ++j) {
        if (j + 1 < NJ) {
          if (!mbar_wait_warp(&bV[(j + 1) & 1], ((j + 1) >> 1) & 1, abort_flag)) { ok = false; break; }
          if (!mbar_wait_warp(bDPread, j & 1, abort_flag)) { ok = false; break; }
          tc_fence_after();
          issue_dp(j + 1);
        }
        if (!mbar_wait_warp(bPS, j & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint64_t mk = mK + (((j % 3) * Lay::kTile) >> 4);
        const uint32_t sb = tmem + tS + (j & 1) * 128;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // dQ += dS K_j, 16 keys an instruction
          umma_bf16_tmem_a_w(tmem + tDQ, sb + (kk >> 1) * 32 + (kk & 1) * 8, mk + ((kk * 2048) >> 4), idG,
                             (j > 0 || kk > 0) ? 1u : 0u);
        umma_commit_w(&bKfree[j % 3]);
        if (j + 2 < NJ) {
          if (!mbar_wait_warp(&bK[(j + 2) % 3], ((j + 2) / 3) & 1, abort_flag)) { ok = false; break; }
          tc_fence_after();
          issue_s(j + 2);
        }
      }
      if (ok) umma_commit_w(bDone);
    }
  } else {
    // ------------------------------------------------------------ compute warpgroups
    const int g = warp >> 2;               // keys [64g, 64g+64) of every key tile
    const int t = (warp & 3) * 32 + lane;  // query row of the tile (TMEM lane)
    const int q = qt * 128 + t;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    // Delta of the tile's rows.  O and O_low come by asynchronous copies into the
    // last K and V stages, which the producer fills after bDel (loads through the
    // 28 KB that the kernel leaves the L1 cache took 12000 clocks a tile), dO
    // is in shared memory for the product; each warpgroup sums half of the channels.
    float* sDel = reinterpret_cast<float*>(smem + Lay::oDel);
    bool ok = true;
    if (NJ > 1) {
      constexpr int CH = D / 8;  // 16-byte chunks of a row
      uint8_t* tO = smem + Lay::oK + 2 * Lay::kTile;
      uint8_t* tL = smem + Lay::oV + Lay::kTile;
#pragma unroll 4
      for (int i = threadIdx.x; i < 128 * CH; i += kCompute) {
        const int r = i / CH, c = i % CH, n = qt * 128 + r;
        const int live = n < a.N ? 16 : 0;
        const uint16_t* po = reinterpret_cast<const uint16_t*>(O) + b * so.b + h * so.h + (live ? (int64_t)n * so.n + c * 8 : 0);
        const uint32_t at = r * (D * 2) + ((c ^ (r & 7)) << 4);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(tO + at)), "l"(po), "r"(live) : "memory");
        if (Olow) {
          const uint16_t* pl = reinterpret_cast<const uint16_t*>(Olow) + (live ? ((int64_t)bh * a.N + n) * D + c * 8 : 0);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(tL + at)), "l"(pl), "r"(live)
                       : "memory");
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      ok = __all_sync(0xffffffffu, mbar_wait(bQO, 0, abort_flag));
      compute_sync_q();
      float sum = 0.f;
#pragma unroll 4
      for (int i = 0; i < CH / 2; ++i) {
        const int c = g * (CH / 2) + i;
        const int at = t * (D * 2) + ((c ^ (t & 7)) << 4);
        const uint4 u = *reinterpret_cast<const uint4*>(tO + at);
        const uint4 v = Olow ? *reinterpret_cast<const uint4*>(tL + at) : make_uint4(0, 0, 0, 0);
        const uint4 w = *reinterpret_cast<const uint4*>(smem + Lay::oO + (c >> 3) * kRegion + t * 128 +
                                                        (((c & 7) ^ (t & 7)) << 4));
        const uint32_t ua[4] = {u.x, u.y, u.z, u.w}, wa[4] = {w.x, w.y, w.z, w.w}, va[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = unpack2<F16>(ua[e]), y = unpack2<F16>(wa[e]), z = unpack2<F16>(va[e]);
          sum = fmaf(x.x + z.x, y.x, fmaf(x.y + z.y, y.y, sum));
        }
      }
      fence_proxy_async_smem();  // before the copies of the producer over what was read
      mbar_arrive(bDel);
      sDel[g * 128 + t] = sum;
      compute_sync_q();
    }
    float del = NJ > 1 ? sDel[t] + sDel[128 + t] : 0.f;
    const float lse_raw = q < a.N ? a.lse[(int64_t)bh * a.N + q] : -INFINITY;
    const float lse = lse_raw == -INFINITY ? INFINITY : lse_raw * kLog2e;  // no key: P = 2^-inf = 0
    const float scale_log2 = a.scale * kLog2e;
    const uint64_t c2 = f2_pack(scale_log2, scale_log2);
    const uint64_t nl2 = f2_pack(-lse, -lse);
    const int2 keys = mask_row(a.mask, b, q, a.N);
    const bool pads = has_padding(a.mask, b);
    const unsigned len = (unsigned)max(0, keys.y - keys.x);
    if (len == 0) del = 0.f;  // the padding's dO may be anything
    if (NJ != 1 && g == 0 && q < a.N) a.delta[(int64_t)bh * a.N + q] = del;
    uint64_t d2 = f2_pack(del, del);
    const Mod mod = MOD ? make_mod(a, h) : Mod{};
    for (int j = 0; j < NJ; ++j) {
      const int buf = j & 1;
      const int kb = (k0 + j) * 128;
      const bool full = kb >= span.max_lo && kb + 128 <= span.min_hi;
      ok = __all_sync(0xffffffffu, mbar_wait(&bS[buf], (j >> 1) & 1, abort_flag));
      if (!ok) {
        if (NJ == 1) {  // the other warps may be at the two barriers below
          compute_sync_q();
          compute_sync_q();
        }
        break;
      }
      tc_fence_after();
      uint32_t r[2][32];
      tmem_ld32(tl + tS + buf * 128 + g * 64, r[0]);
      tmem_ld32(tl + tS + buf * 128 + g * 64 + 32, r[1]);
      tmem_ld_wait();
      if (MOD && mod.cap) {
        cap_scores(r[0], mod.pre);
        cap_scores(r[1], mod.pre);
      }
      float p[2][32];  // P times the cap's derivative
      auto p_pass = [&](auto masked) {
        const int lo = keys.x - kb - g * 64;
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float pa, pb;
            if constexpr (MOD) {
              const float dist = (float)(q - kb - g * 64 - ch * 32 - e);
              exponents(mod, __uint_as_float(r[ch][e]), __uint_as_float(r[ch][e + 1]), lse, lse, dist, dist - 1.f, pa,
                        pb);
            } else {
              f2_unpack(f2_fma(f2_pack(__uint_as_float(r[ch][e]), __uint_as_float(r[ch][e + 1])), c2, nl2), pa, pb);
            }
            pa = fast_exp2(pa);
            pb = fast_exp2(pb);
            if constexpr (decltype(masked)::value) {
              pa = (unsigned)(ch * 32 + e - lo) < len ? pa : 0.f;
              pb = (unsigned)(ch * 32 + e + 1 - lo) < len ? pb : 0.f;
            }
            p[ch][e] = pa;
            p[ch][e + 1] = pb;
          }
      };
      if (full) p_pass(std::false_type{});
      else p_pass(std::true_type{});
      if (MOD && mod.cap) {  // times 1 - tanh^2
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            p[ch][e] = fmaf(-p[ch][e] * __uint_as_float(r[ch][e]), __uint_as_float(r[ch][e]), p[ch][e]);
      }
      ok = __all_sync(0xffffffffu, mbar_wait(bDP, j & 1, abort_flag));
      if (NJ == 1) {
        // The row's keys all lie in this tile: Delta = sum_j P dP in fp32.
        // With two or three keys, one of them nearly all of the weight,
        // dP - Delta is a small difference, which the roundings of P in O,
        // averaged over more keys, would still show in.
        float sum = 0.f;
        if (ok) {
          tc_fence_after();
          const int lo = keys.x - kb - g * 64;
#pragma unroll 1
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t sv[16], dv[16];
            tmem_ld16(tl + tS + buf * 128 + g * 64 + ch * 16, sv);
            tmem_ld16(tl + tDP + g * 64 + ch * 16, dv);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float x = __uint_as_float(sv[e]) * (MOD ? mod.mul : scale_log2);
              if constexpr (MOD) {
                if (mod.cap) x = tanh_any(__uint_as_float(sv[e]) * mod.pre) * mod.mul;
                if (mod.bias) x = fmaf(-mod.slope2, fabsf((float)(q - kb - g * 64 - ch * 16 - e)), x);
              }
              if ((unsigned)(ch * 16 + e - lo) < len) sum = fmaf(fast_exp2(x - lse), __uint_as_float(dv[e]), sum);
            }
          }
        }
        compute_sync_q();  // both halves have read the sums from O
        sDel[g * 128 + t] = sum;
        compute_sync_q();
        del = sDel[t] + sDel[128 + t];
        d2 = f2_pack(del, del);
        if (g == 0 && q < a.N) a.delta[(int64_t)bh * a.N + q] = del;
      }
      if (!ok) break;
      tc_fence_after();
      const bool pad = pads && !full && empty_keys(a.mask, b, k0 + j, a.N);
      if (pad) {
        // padding keys of K_j (for dQ): each warpgroup takes half of the row
        const int2 s = mask_col(a.mask, b, kb + t, a.N);
        if (s.y <= s.x && g * 64 < D) zero_row(smem + Lay::oK + (j % 3) * Lay::kTile, t, g, 1);
        fence_proxy_async_smem();
      }
      // dP is released as soon as it is in registers, so that the next
      // tile's dP can be computed meanwhile
      uint32_t dr[2][32];
      tmem_ld32(tl + tDP + g * 64, dr[0]);
      tmem_ld32(tl + tDP + g * 64 + 32, dr[1]);
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(bDPread);
      if (pad) {  // scores and dP of padding keys may be anything
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if ((unsigned)(kb + g * 64 + ch * 32 + e - keys.x) >= len) p[ch][e] = 0.f, dr[ch][e] = 0u;
      }
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        uint32_t dh[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const uint64_t diff = f2_sub(f2_pack(__uint_as_float(dr[ch][e]), __uint_as_float(dr[ch][e + 1])), d2);
          float da, db;
          f2_unpack(f2_mul(f2_pack(p[ch][e], p[ch][e + 1]), diff), da, db);
          dh[e >> 1] = pack2<F16>(da, db);
        }
        tmem_st16(tl + tS + buf * 128 + g * 64 + ch * 32, dh);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bPS);
    }
    if (NJ > 0) ok = __all_sync(0xffffffffu, ok && mbar_wait(bDone, 0, abort_flag));
    if (ok) {  // out through the first K stage, which no product or copy uses any more
      tc_fence_after();
      constexpr int CW = D;  // bytes of the warpgroup's half of a row
      uint8_t* lines = smem + Lay::oK + warp * (32 * CW);
      uint32_t rv[D / 64][32];
      if (NJ > 0) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) tmem_ld32(tl + tDQ + g * (D / 2) + c * 32, rv[c]);
        tmem_ld_wait();
      }
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t (&r)[32] = rv[c];
        if (NJ == 0 || len == 0) {
#pragma unroll
          for (int e = 0; e < 32; ++e) r[e] = 0u;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = pack2<F16>(__uint_as_float(r[8 * i + 2 * e]) * a.scale, __uint_as_float(r[8 * i + 2 * e + 1]) * a.scale);
          *reinterpret_cast<uint4*>(lines + line_at<CW>(lane, c * 4 + i)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      __syncwarp();
      const int q0 = q - lane;
      store_lines<CW>(lines, reinterpret_cast<uint16_t*>(dQ) + b * sdq.b + h * sdq.h + (int64_t)q0 * sdq.n + g * (D / 2),
                      sdq.n, a.N - q0, lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag) report_error(a.errw, ERRW_TIMEOUT);
}

template <int D, bool F16, bool MOD>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& go,
                   const DenseArgs& a, const void* o, const Strides& so, const void* o_low, void* dq,
                   const Strides& sdq, void* dk, const Strides& sdk, void* dv, const Strides& sdv, cudaStream_t st) {
  const int64_t gq = (int64_t)a.n_tiles * a.B * a.Hq, gk = (int64_t)a.n_tiles * a.B * a.Hkv;
  if (gq > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  auto* fq = dense_bwd_q_kernel<D, F16, MOD>;
  auto* fk = dense_bwd_kv_kernel<D, F16, MOD>;
  cudaError_t e = cudaFuncSetAttribute(fq, cudaFuncAttributeMaxDynamicSharedMemorySize, QSmem<D>::kAlloc);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(fk, cudaFuncAttributeMaxDynamicSharedMemorySize, KvSmem<D>::kAlloc);
  if (e != cudaSuccess) return e;
  fq<<<dim3((unsigned)gq), kThreads, QSmem<D>::kAlloc, st>>>(q, k, v, go, a, o, so, o_low, dq, sdq);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // Few key tiles leave SMs idle: then a cluster of 2, 4 or 8 CTAs shares the
  // query steps of one, as long as a wave of 148 holds them (257 tokens, 2 key
  // heads of 4 query heads each: 47 us without, 14 with).  Up to two waves of
  // tiles of unequal length pair up (8K tokens in documents, 256 tiles: 149 us
  // without, 133 with clusters of 2, 178 of 4).
  int C = 1;
  while (C < 8 && gk * C * 2 <= 148 && (int64_t)a.n_tiles * (a.Hq / a.Hkv) >= 2 * C) C *= 2;
  if (C == 1 && gk <= 296 && (int64_t)a.n_tiles * (a.Hq / a.Hkv) >= 2) C = 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(gk * C));
  cfg.blockDim = dim3(kThreadsKV);
  cfg.dynamicSmemBytes = KvSmem<D>::kAlloc;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {(unsigned)C, 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fk, q, k, v, go, a, dk, sdk, dv, sdv, C);
}

}  // namespace

cudaError_t launch_dense_bwd(const DenseArgs& a, int d, bool f16, const CUtensorMap& q, const CUtensorMap& k,
                             const CUtensorMap& v, const CUtensorMap& go, const void* o, const Strides& so,
                             const void* o_low, void* dq, const Strides& sdq, void* dk, const Strides& sdk, void* dv,
                             const Strides& sdv, cudaStream_t st) {
  const bool mod = a.softcap > 0.f || a.slopes;
  auto pick = [&](auto D, auto F, auto M) {
    return launch<decltype(D)::value, decltype(F)::value, decltype(M)::value>(q, k, v, go, a, o, so, o_low, dq, sdq, dk,
                                                                              sdk, dv, sdv, st);
  };
  using T = std::true_type;
  using N = std::false_type;
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (d == 128) {
    if (f16) return mod ? pick(D128{}, T{}, T{}) : pick(D128{}, T{}, N{});
    return mod ? pick(D128{}, N{}, T{}) : pick(D128{}, N{}, N{});
  }
  if (f16) return mod ? pick(D64{}, T{}, T{}) : pick(D64{}, T{}, N{});
  return mod ? pick(D64{}, N{}, T{}) : pick(D64{}, N{}, N{});
}

}  // namespace lh
