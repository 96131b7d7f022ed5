// Masked dense attention, forward: O = softmax(cap(scale Q K^T) + bias) V over
// the keys that the mask leaves each query, grouped heads (query head h reads
// key head h / (Hq / Hkv)).
//
// One pass over the keys with a running maximum and sum per query row.  One
// CTA owns two 128-query tiles (A, B; small calls: A alone) of one head and
// streams the key tiles of both through a 2-stage ring; while one tile's softmax
// runs, the tensor core works on the other's products.  Bound by those two
// together: 16K causal tokens, 8 heads of 128: 477 us (1.15 PFLOP/s; the tensor
// cores busy for 59% of the time), with a cap or a distance bias by the softmax.
//   warps 0-3, 4-7  softmax of tile A, B: thread t owns query row t (TMEM
//                   lane t) and all 128 keys of a key tile
//   warp 8          TMA producer
//   warp 9          MMA issuer: per key tile P_A V, the next S_A = Q_A K^T,
//                   P_B V, the next S_B
// TMEM columns: S_A/P_A [0,128), S_B/P_B [128,256), O_A [256,256+D),
// O_B [256+D,256+2D).  P goes back over the first half of the 64 S columns it
// came from, in the inputs' 16-bit type: its rounding (half a step, 2^-8 in bf16)
// is averaged over the row's keys and stays below the rounding of O itself.
// The sums, the maximum, O and LSE are fp32; what O's rounding takes off can be
// written too (O_low): the backward's Delta = rowsum(dO * O) cancels against dP,
// and from the rounded O alone the error of dQ and dK was 1.7 times that of
// rounding the exact gradients, with it 1.4 times.  (O over the sum of the
// rounded P, so that its weights add up to one, left as much and took 502 us
// in place of 477 at 16K causal tokens, 8 heads.)
#include <type_traits>

#include "lh_dense.cuh"

namespace lh {
namespace {
using namespace sm100;

constexpr int kSoftmax = 256;
constexpr int kThreads = kSoftmax + 64;
constexpr int kWarpTma = 8, kWarpMma = 9;
// every kPolyOf-th pair of exponentials of an unmasked tile goes to the FMA
// pipes: the exponential unit makes 16 a clock and SM, 2048 clocks for the two
// query tiles' 2 x 128 x 128, as long as their matrix products take
constexpr int kPolyOf = 4;
constexpr int kRegion = 128 * 128;  // one [128 rows][64 x 16 bit] region

template <int D>
struct Smem {
  static constexpr int kTile = D / 64 * kRegion;
  static constexpr int oQ = 0;               // Q_A, Q_B
  static constexpr int oK = oQ + 2 * kTile;  // 2 stages
  static constexpr int oV = oK + 2 * kTile;  // 2 stages
  static constexpr int oBar = oV + 2 * kTile;
  static constexpr int kAlloc = oBar + 256 + 1024;
};

// MOD: scores are capped or biased (they are turned once and written back to
// TMEM, the masked ones as -inf)
template <int D, bool F16, bool MOD>
__global__ void __launch_bounds__(kThreads, 1)
    dense_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ DenseArgs a, void* __restrict__ O,
                     const Strides so, void* __restrict__ Olow) {
  using Lay = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::oBar);
  uint64_t* bQ = bars + 0;
  uint64_t* bK = bars + 1;       // [2] stages
  uint64_t* bV = bars + 3;       // [2]
  uint64_t* bKVfree = bars + 5;  // [2]
  uint64_t* bS = bars + 7;       // [2] tiles: S in TMEM (and the tile's previous P V done)
  uint64_t* bP = bars + 9;       // [2] tiles x [2] halves of the keys: P in TMEM (128 arrivals); O rescaled
  uint64_t* bO = bars + 13;      // [2] tiles: a P V product done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::oBar + 192);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::oBar + 196);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // pair-major grid, last pairs first: causal rows are longest there, and the
  // short ones fill the tail
  const int n_ctas = (a.n_tiles + a.q_per_cta - 1) / a.q_per_cta;  // of a head
  const int BH = a.B * a.Hq;
  const int qt = (n_ctas - 1 - (int)(blockIdx.x / (unsigned)BH)) * a.q_per_cta;  // first query tile
  const int bh = (int)(blockIdx.x % (unsigned)BH);
  const int b = bh / a.Hq, h = bh % a.Hq, hk = h / (a.Hq / a.Hkv);
  const bool hasB = a.q_per_cta == 2 && qt + 1 < a.n_tiles;
  // key tiles [first, end) of each query tile, and of both
  TileSpan span[2];
  int first[2], end[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    span[x] = {0, 0, 0, 0};
    if (x == 0 || hasB) span[x] = mask_row_tile(a.mask, b, qt + x, a.N);
    first[x] = span[x].min_lo >> 7;
    end[x] = span[x].max_hi > span[x].min_lo ? (span[x].max_hi + 127) >> 7 : first[x];
  }
  const bool liveA = end[0] > first[0], liveB = end[1] > first[1];
  const int j0 = liveA ? (liveB ? min(first[0], first[1]) : first[0]) : first[1];
  const int j1 = liveA ? (liveB ? max(end[0], end[1]) : end[0]) : end[1];

  if (threadIdx.x == 0) {
    mbar_init(bQ, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bK[s], 1);
      mbar_init(&bV[s], 1);
      mbar_init(&bKVfree[s], 1);
      mbar_init(&bS[s], 1);
      mbar_init(&bP[2 * s], 128);
      mbar_init(&bP[2 * s + 1], 128);
      mbar_init(&bO[s], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == kWarpTma) {
    if (lane == 0 && j1 > j0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      mbar_expect_tx(bQ, (hasB ? 2 : 1) * 128 * D * 2);
      for (int x = 0; x < (hasB ? 2 : 1); ++x)
        for (int ch = 0; ch < D / 64; ++ch)
          tma_load_4d(smem + Lay::oQ + x * Lay::kTile + ch * kRegion, &tmQ, bQ, ch * 64, (qt + x) * 128, h, b);
      for (int j = j0; j < j1; ++j) {
        const int i = j - j0, st = i & 1, use = i >> 1;
        if (i >= 2 && !mbar_wait(&bKVfree[st], (use - 1) & 1, abort_flag)) break;
        mbar_expect_tx(&bK[st], 128 * D * 2);
        for (int ch = 0; ch < D / 64; ++ch)
          tma_load_4d(smem + Lay::oK + st * Lay::kTile + ch * kRegion, &tmK, &bK[st], ch * 64, j * 128, hk, b);
        mbar_expect_tx(&bV[st], 128 * D * 2);
        for (int ch = 0; ch < D / 64; ++ch)
          tma_load_4d(smem + Lay::oV + st * Lay::kTile + ch * kRegion, &tmV, &bV[st], ch * 64, j * 128, hk, b);
      }
    }
  } else if (warp == kWarpMma) {
    if (j1 > j0) {  // the whole warp; one elected lane issues each instruction
      constexpr uint32_t idQK = idesc16<F16>(128, 128, false, false);
      constexpr uint32_t idPV = idesc16<F16>(128, D, false, true);
      const uint64_t kQ = sdesc_sw128(smem_u32(smem + Lay::oQ), 16, 1024);
      const uint64_t kK = sdesc_sw128(smem_u32(smem + Lay::oK), 16, 1024);
      const uint64_t mV = sdesc_sw128(smem_u32(smem + Lay::oV), kRegion, 1024);
      auto issue_s = [&](int x, int j) {
        const uint64_t qb = kQ + ((x * Lay::kTile) >> 4), kb = kK + ((((j - j0) & 1) * Lay::kTile) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kRegion + (kk & 3) * 32) >> 4;
          umma_bf16_w(tmem + x * 128, qb + off, kb + off, idQK, kk > 0 ? 1u : 0u);
        }
        umma_commit_w(&bS[x]);
      };
      bool ok = mbar_wait_warp(bQ, 0, abort_flag) && mbar_wait_warp(&bK[0], 0, abort_flag);
      if (ok) {
        tc_fence_after();
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (first[x] == j0 && end[x] > j0) issue_s(x, j0);
      }
      for (int j = j0; ok && j < j1; ++j) {
        const int i = j - j0, st = i & 1;
        // every tile's arrival is waited for, also where neither query tile
        // reads it, so that a stage is never refilled under a copy
        ok = mbar_wait_warp(&bV[st], (i >> 1) & 1, abort_flag);
        bool k_next = false;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!ok) break;
          if (j >= first[x] && j < end[x]) {
            const uint64_t vb = mV + ((st * Lay::kTile) >> 4);
#pragma unroll
            for (int half = 1; half >= 0; --half) {  // keys 64-127 come first
              if (!mbar_wait_warp(&bP[2 * x + half], (j - first[x]) & 1, abort_flag)) { ok = false; break; }
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_bf16_tmem_a_w(tmem + 256 + x * D, tmem + x * 128 + half * 64 + kk * 8,
                                   vb + (((half * 4 + kk) * 2048) >> 4), idPV,
                                   (j > first[x] || half == 0 || kk > 0) ? 1u : 0u);
            }
            if (!ok) break;
            umma_commit_w(&bO[x]);
          }
          if (j + 1 < j1 && !k_next) {
            if (!mbar_wait_warp(&bK[(i + 1) & 1], ((i + 1) >> 1) & 1, abort_flag)) { ok = false; break; }
            k_next = true;
            tc_fence_after();
          }
          if (j + 1 >= first[x] && j + 1 < end[x]) issue_s(x, j + 1);
        }
        if (ok) umma_commit_w(&bKVfree[st]);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int x = warp >> 2;
    const int j_first = x ? first[1] : first[0], j_end = x ? end[1] : end[0];
    const TileSpan sp = x ? span[1] : span[0];
    const int row = (qt + x) * 128 + (warp & 3) * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = tl + x * 128, to = tl + 256 + x * D;
    const int2 keys = mask_row(a.mask, b, row, a.N);
    const bool pads = has_padding(a.mask, b);
    const Mod mod = MOD ? make_mod(a, h) : Mod{};
    const float scale_log2 = !MOD ? a.scale * kLog2e : mod.bias ? 1.f : mod.mul;
    float m_run = -INFINITY, l_run = 0.f;
    float s_ref = 0.f;  // the score that m_run is the exponent of
    bool ok = true;
    for (int j = j_first; j < j_end; ++j) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bS[x], (j - j_first) & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const bool full = j * 128 >= sp.max_lo && j * 128 + 128 <= sp.min_hi;
      const int lo = keys.x - j * 128;
      const unsigned len = (unsigned)max(0, keys.y - keys.x);
      // row maximum over two 64-key halves, in eight independent chains
      uint32_t r[2][32];
      float mc[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) mc[q] = -INFINITY;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        tmem_ld32(ts + hh * 64, r[0]);
        tmem_ld32(ts + hh * 64 + 32, r[1]);
        tmem_ld_wait();
        if constexpr (MOD) {
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            if (mod.cap) cap_scores(r[ch], mod.pre);
            if (mod.bias) {
              const float d0 = (float)(row - j * 128 - hh * 64 - ch * 32);  // distance to key 0 of the chunk
#pragma unroll
              for (int i = 0; i < 32; ++i)
                r[ch][i] = __float_as_uint(
                    fmaf(-mod.slope2, fabsf(d0 - (float)i), __uint_as_float(r[ch][i]) * mod.mul));
            }
            if (!full) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if ((unsigned)(hh * 64 + ch * 32 + i - lo) >= len) r[ch][i] = __float_as_uint(-INFINITY);
            }
            tmem_st32(ts + hh * 64 + ch * 32, r[ch]);
          }
        }
        if (!MOD && !full) {
#pragma unroll
          for (int ch = 0; ch < 2; ++ch)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((unsigned)(hh * 64 + ch * 32 + i - lo) < len)
                mc[ch * 4 + (i >> 3)] = fmaxf(mc[ch * 4 + (i >> 3)], __uint_as_float(r[ch][i]));
        } else {
#pragma unroll
          for (int ch = 0; ch < 2; ++ch)
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              mc[ch * 4 + (i >> 3)] =
                  max3f_nan(mc[ch * 4 + (i >> 3)], __uint_as_float(r[ch][i]), __uint_as_float(r[ch][i + 1]));
        }
      }
      if constexpr (MOD) tmem_st_wait();
      const float mx = max3f_nan(max3f_nan(mc[0], mc[1], mc[2]), max3f_nan(mc[3], mc[4], mc[5]),
                                 max3f_nan(mc[6], mc[7], -INFINITY));
      // The reference moves only when the maximum exceeds it by more than 8
      // (P stays <= 2^8); O and l share it, so the result is exact either way.
      const float m_tile = mx * scale_log2;
      const bool move = m_tile > m_run + 8.f;
      const float m_new = move ? m_tile : m_run;
      const float alpha = move ? fast_exp2(m_run - m_new) : 1.f;
      const float m_ref = m_new == -INFINITY ? 0.f : m_new;  // no key of the row so far: every P is 0
      if (move) s_ref = mx;
      // rescale the O row (the tile's previous P V completed before this S)
      if (j > j_first && __any_sync(0xffffffffu, move)) {
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
      // P over the S columns that each half of the keys came from; the half
      // that the maximum read last is still in registers and goes first, and
      // its P V starts while the other half's P is made
      const uint64_t c2 = f2_pack(scale_log2, scale_log2), nm2 = f2_pack(-m_ref, -m_ref);
      const uint64_t ns2 = f2_pack(-s_ref, -s_ref);
      uint64_t rs2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
      auto p_chunk = [&](auto careful, uint32_t (&sv)[32], int key, uint32_t dst, uint64_t& sum) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const uint64_t s2 = f2_pack(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
          // The careful form takes the difference of the scores first: in
          // s c - m a large m is off by its rounding, 2^-24 of it.
          const uint64_t x2 = decltype(careful)::value ? f2_mul(f2_add(s2, ns2), c2) : f2_fma(s2, c2, nm2);
          float pa, pb;
          if constexpr (decltype(careful)::value) {
            f2_unpack(x2, pa, pb);
            pa = (unsigned)(key + e - lo) < len ? fast_exp2(pa) : 0.f;
            pb = (unsigned)(key + e + 1 - lo) < len ? fast_exp2(pb) : 0.f;
          } else if (!MOD && (e >> 1) % kPolyOf == kPolyOf - 1) {
            poly_exp2(x2, pa, pb);
          } else {
            f2_unpack(x2, pa, pb);
            pa = fast_exp2(pa);
            pb = fast_exp2(pb);
          }
          sum = f2_add(sum, f2_pack(pa, pb));
          pk[e >> 1] = pack2<F16>(pa, pb);
        }
        tmem_st16(dst, pk);
      };
      auto p_pass = [&](auto careful) {
        p_chunk(careful, r[0], 64, ts + 64, rs2[0]);
        tmem_ld32(ts, r[0]);
        p_chunk(careful, r[1], 96, ts + 80, rs2[1]);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bP[2 * x + 1]);
        tmem_ld_wait32(r[0]);
        tmem_ld32(ts + 32, r[1]);
        p_chunk(careful, r[0], 0, ts, rs2[0]);
        tmem_ld_wait32(r[1]);
        p_chunk(careful, r[1], 32, ts + 16, rs2[1]);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bP[2 * x]);
      };
      if (pads && !full && empty_keys(a.mask, b, j, a.N)) {
        const int i = j - j0, t = (warp & 3) * 32 + lane;
        ok = __all_sync(0xffffffffu, mbar_wait(&bV[i & 1], (i >> 1) & 1, abort_flag));
        if (!ok) break;
        const int2 q = mask_col(a.mask, b, j * 128 + t, a.N);
        if (q.y <= q.x) zero_row(smem + Lay::oV + (i & 1) * Lay::kTile, t, 0, D / 64);
        fence_proxy_async_smem();
      }
      // masked tiles, and rows whose scores are beyond 2^16 in size, have a NaN or
      // are all -inf (the polynomial exponentials would make numbers of those)
      if (!MOD && (!full || __any_sync(0xffffffffu, !(fabsf(m_new) <= 65536.f) || mx != mx))) p_pass(std::true_type{});
      else p_pass(std::false_type{});
      float rsa, rsb;
      f2_unpack(f2_add(rs2[0], rs2[1]), rsa, rsb);
      l_run = l_run * alpha + (rsa + rsb);
      m_run = m_new;
    }
    const bool any = j_end > j_first;
    if (ok && any) ok = __all_sync(0xffffffffu, mbar_wait(&bO[x], (j_end - j_first - 1) & 1, abort_flag));
    if (ok && (x == 0 || hasB)) {
      tc_fence_after();
      const float inv_l = l_run > 0.f || l_run != l_run ? 1.f / l_run : 0.f;
      // A thread a row: through shared memory as whole lines, 16K causal tokens take
      // 2% less and 257 tokens 10% more.
      uint16_t* low = Olow ? reinterpret_cast<uint16_t*>(Olow) + ((int64_t)bh * a.N + row) * D : nullptr;
      uint16_t* dst = reinterpret_cast<uint16_t*>(O) + b * so.b + h * so.h + (int64_t)row * so.n;
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t o[32];
        if (any) {
          tmem_ld32(to + ch * 32, o);
          tmem_ld_wait();
        }
        if (row < a.N) {
          uint4* d4 = reinterpret_cast<uint4*>(dst + ch * 32);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[4], v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = l_run == 0.f ? 0.f : __uint_as_float(o[8 * q + 2 * e]) * inv_l;
              const float y = l_run == 0.f ? 0.f : __uint_as_float(o[8 * q + 2 * e + 1]) * inv_l;
              w[e] = pack2<F16>(x, y);
              if (low) {
                const float2 h = unpack2<F16>(w[e]);
                v[e] = pack2<F16>(x - h.x, y - h.y);
              }
            }
            d4[q] = make_uint4(w[0], w[1], w[2], w[3]);
            if (low) reinterpret_cast<uint4*>(low + ch * 32)[q] = make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
      }
      if (row < a.N) a.lse[(int64_t)bh * a.N + row] = l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * kLn2;
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

template <int D, bool F16, bool MOD>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, DenseArgs a, void* o,
                   const Strides& so, void* o_low, cudaStream_t st) {
  // one query tile a CTA where the GPU takes all of them at once: two share the
  // CTA's issue slots and its ring (1024 tokens, 16 heads of 128: 20 us, 24 in
  // pairs; 4096 tokens, 4 heads: 58, 67)
  a.q_per_cta = (int64_t)a.n_tiles * a.B * a.Hq <= 148 ? 1 : 2;
  const int64_t grid = (int64_t)((a.n_tiles + a.q_per_cta - 1) / a.q_per_cta) * a.B * a.Hq;
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  auto* fn = dense_fwd_kernel<D, F16, MOD>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kAlloc);
  if (e != cudaSuccess) return e;
  fn<<<dim3((unsigned)grid), kThreads, Smem<D>::kAlloc, st>>>(q, k, v, a, o, so, o_low);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dense_fwd(const DenseArgs& a, int d, bool f16, const CUtensorMap& q, const CUtensorMap& k,
                             const CUtensorMap& v, void* o, const Strides& so, void* o_low, cudaStream_t st) {
  const bool mod = a.softcap > 0.f || a.slopes;
  auto pick = [&](auto D, auto F, auto M) {
    return launch<decltype(D)::value, decltype(F)::value, decltype(M)::value>(q, k, v, a, o, so, o_low, st);
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
