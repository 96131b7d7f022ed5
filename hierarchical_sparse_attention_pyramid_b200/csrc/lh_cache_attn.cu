// Attention of a few query tokens a sequence (one, or a tree of drafted ones)
// over the paged cache.
//
// Bound by reading the cache once: a key's row meets only the rows of its
// head's group (tokens x Hq / Hkv), a few operations a byte.  So each warp
// streams its keys through a ring of its own in shared memory (asynchronous
// copies, 8 KB in flight a warp, no barrier between warps) and multiplies
// them with matrix instructions of 16 keys (channels) x 8 query rows:
// S^T = K Q^T and O^T = V^T P^T, so that 8 rows fill the instruction, which
// is a group's size in decoding.  P^T turns from the layout of a result into
// that of an operand by 8 x 8 transposes within the warp.  The order of the
// channels in K Q^T and of the output channels in V^T P^T is free, so each
// lane loads 16 contiguous bytes of a row and calls them its fragment.
//
// 8-bit values become fp16 operands, which hold them exactly: e4m3 by the
// hardware's conversion, int8 as the difference of two fp16 numbers whose low
// bits are the value's.  So that queries and probabilities are fp16 operands
// too without leaving its range, a query row is multiplied by a power of two
// that brings its largest value to 2^14 (exact; what is 2^28 times smaller
// than that loses bits), and the probability times the value's scale is taken
// relative to a power of two above the scales met so far.  The scale of a key
// enters its score.
//
// One sequence of 512K int8 tokens, 4 key heads of 128: 86 us (6.4 TB/s); 64
// sequences of up to 8K e4m3 tokens: 41 us against 35 for a copy of the bytes.
//
// A block of 4 warps takes its stretch of the work list (lh_cache_attn.cuh)
// for 8, 16 or 32 query rows of a head; the warps' running maxima, sums and
// outputs are joined in shared memory in warp order.
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "lh_cache_attn.cuh"

namespace lh {
namespace {

// Query rows (tokens x heads of a group) that a block takes.  Up to 32 the
// kernel of this file, above the tensor core tiles: one sequence of 64K e4m3
// tokens, 4 key heads: 32 rows 39 us here and 57 there, 96 rows (three tiles of
// 32 here) 78 and 61.
int cache_attn_row_tile(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 128; }

constexpr int kWarps = 4, kThreads = kWarps * 32;
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {  // zeros where not live
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <int W>
__device__ __forceinline__ void lds(uint32_t (&x)[W], uint32_t at) {
  if constexpr (W == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at));
  else
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(at));
}

// transpose of an 8 x 8 matrix of 16-bit elements held by a warp
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// shapes of one (D, kind): what a warp's ring holds
template <int D, int KIND, int NB>
struct Shape {
  static constexpr bool kHeld8 = KIND == LH_CACHE_E4M3 || KIND == LH_CACHE_INT8;
  static constexpr int kBytes = kHeld8 ? 1 : 2;
  static constexpr int kRow = D * kBytes;                 // bytes of a key's row
  static constexpr int kKeys = kRow <= 128 ? 32 : 16;     // keys of a warp's step: 4 or 8 KB of K and V
  static constexpr int kTile = kKeys * kRow;              // K or V of a step
  static constexpr int kStage = 2 * kTile + (kHeld8 ? 2 * kKeys * 4 : 0);
  static constexpr int kStages = kTile >= 4096 ? 2 : 4;   // 16 KB a warp
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr bool kQShared = NB > 2;                // query fragments in shared memory instead of registers
  static constexpr int kQ = kQShared ? NB * (D / 16) * 256 : 0;
  static constexpr int kOutRow = D + 4;                   // floats of a row of the warps' results
  static constexpr int kOut = kWarps * NB * 8 * (kOutRow + 2) * 4;  // over the ring
  static constexpr int kSmem = kQ + (kRing > kOut ? kRing : kOut);
};

// NB: tiles of 8 query rows that a block takes (each conversion of a held
// value then serves NB matrix instructions)
template <int D, int KIND, bool F16, int NB>
__global__ void __launch_bounds__(kThreads, NB <= 2 ? 3 : 2)
    cache_attn_kernel(const __grid_constant__ CacheAttnArgs a) {
  using Sh = Shape<D, KIND, NB>;
  constexpr bool HELD8 = Sh::kHeld8, HALF = F16 || HELD8;  // HALF: fp16 matrix operands
  constexpr int BYTES = Sh::kBytes, ROW = Sh::kRow, STAGES = Sh::kStages, KEYS = Sh::kKeys, NT = KEYS / 8;
  constexpr int E = 16 / BYTES;             // channels of a 16-byte unit
  constexpr int STEPS = D / 16;             // matrix steps over the channels
  constexpr int VB = ROW / 8 < 16 ? ROW / 8 : 16;  // bytes of a V load (8 lanes a key)
  constexpr int VE = VB / BYTES, VC = D / (8 * VE), VW = VB / 4;
  constexpr float kPUp = HELD8 ? 64.f : 1.f;  // raises probabilities (at most 2^8) within fp16's range
  extern __shared__ __align__(128) uint8_t smem[];
  uint2* sQ = reinterpret_cast<uint2*>(smem);                           // [NB][STEPS][32] where shared
  float* sO = reinterpret_cast<float*>(smem + Sh::kQ);                  // later [kWarps][NB * 8][kOutRow]
  float* sML = sO + kWarps * NB * 8 * Sh::kOutRow;                      // [kWarps][NB * 8][2]

  __shared__ int64_t scan[kWarps + 1];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int G = a.Hq / a.c.heads;
  Stretch stretch = find_stretch<kWarps>(a, 8 * NB, scan);
  if (stretch.u >= stretch.u_end) return;
  Seq seq = load_seq(a, stretch.s, false);
  Piece piece;

  while (next_piece(a, 8 * NB, stretch, seq, piece)) {
    const int s = stretch.s, hk = piece.hk, tok0 = seq.tok0, len = seq.len, k0 = piece.k0, k1 = piece.k1;
    const int r0 = piece.rt * 8 * NB, n_rows = seq.T * G;  // row r: token r / G, head r % G of the group
    const int ctx = len - seq.T;                           // keys before the query tokens' own

    // ------------------------------------------------------------ the ring of keys
    const int32_t* table = a.table + (int64_t)s * a.width;
    constexpr uint32_t kNone = 0xffffffffu;
    // lane j looks up the 8 keys from key + 8 j on (pages hold 8 tokens or more)
    auto look_up = [&](int key) -> uint32_t {
      const int kk = key + 8 * lane;
      return lane >= NT || kk >= k1 ? kNone : key_rows(a, table, hk, kk);
    };
    const uint32_t ring = sm100::smem_u32(sO) + warp * (STAGES * Sh::kStage);
    // 16-byte units of a row are permuted by the row, so that the lanes of one
    // fragment load meet different banks: 4 lanes x 2 rows of K, 2 units x 4
    // even (odd) rows of V
    auto swz = [](int row, int unit) -> uint32_t {
      constexpr int U = ROW / 16;
      const int f = U >= 8 ? (((row >> 1) & 3) << 1) ^ ((row & 1) << 2) : (row >> 1) & 3;
      return (uint32_t)(row * ROW + ((unit ^ f) << 4));
    };
    constexpr int U = ROW / 16, PER = KEYS * U / 32, RPI = 32 / U;  // copies a lane makes, rows of one round of copies
    const char* k_lane = static_cast<const char*>(a.c.k) + (lane / U % 8) * ROW + (lane % U) * 16;
    const char* v_lane = static_cast<const char*>(a.c.v) + (lane / U % 8) * ROW + (lane % U) * 16;
    auto fetch = [&](int key, uint32_t rows, uint32_t base, auto whole) {
      constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint32_t r = __shfl_sync(0xffffffffu, rows, j);
        const char* kp = k_lane + (uint64_t)(WHOLE || r != kNone ? r : 0u) * ROW;
        const char* vp = v_lane + (uint64_t)(WHOLE || r != kNone ? r : 0u) * ROW;
#pragma unroll
        for (int i = 0; i < PER / NT; ++i) {
          const int row = j * 8 + i * RPI + lane / U;
          const bool live = WHOLE || (r != kNone && key + row < k1);
          const uint32_t dst = base + swz(row, lane % U);
          cp_async16(dst, live ? kp + i * RPI * ROW : kp, live);
          cp_async16(dst + Sh::kTile, live ? vp + i * RPI * ROW : vp, live);
        }
      }
      if constexpr (HELD8) {
        const uint32_t r = __shfl_sync(0xffffffffu, rows, lane >> 3 & (NT - 1));
        const bool live = lane < KEYS && (WHOLE || (r != kNone && key + lane < k1));
        const uint64_t at = live ? (uint64_t)r + (lane & 7) : 0;
        if (lane < KEYS) {
          cp_async4(base + 2 * Sh::kTile + lane * 4, a.c.k_scale + at, live);
          cp_async4(base + 2 * Sh::kTile + KEYS * 4 + lane * 4, a.c.v_scale + at, live);
        }
      }
    };
    constexpr int kStride = kWarps * KEYS;
    int key = k0 + warp * KEYS, ahead = key;
    unsigned bad = 0;  // bit NT * slot + j: 8 keys of a slot whose page is missing
    uint32_t rows = look_up(ahead);
    auto fetch_next = [&](int slot) {
      if (ahead < k1) {
        const uint32_t base = ring + slot * Sh::kStage;
        const unsigned none = __ballot_sync(0xffffffffu, rows == kNone) & ((1u << NT) - 1);
        if (none == 0 && ahead + KEYS <= k1) fetch(ahead, rows, base, std::true_type{});
        else fetch(ahead, rows, base, std::false_type{});
        bad = (bad & ~(((1u << NT) - 1) << (NT * slot))) | none << (NT * slot);
        ahead += kStride;
        rows = look_up(ahead);
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) fetch_next(i);

    // ------------------------------------------------------------ query rows
    // Fragment of tile nb, step st: channels ch .. ch + 3 of row nb * 8 + g,
    // ch = c * 4 E + t * E + 4 i with st = c * (E / 4) + i: of a 16-byte unit's
    // channels (8 or 16) the lane's next four.  up: power of two that brings a
    // bf16 row's largest value to [2^14, 2^15) for 8-bit keys
    auto load_q = [&](int nb, uint2 (&f)[STEPS], float& up) {
      const int r = r0 + nb * 8 + g;
      const uint16_t* p = static_cast<const uint16_t*>(a.q) + (int64_t)(tok0 + r / G) * a.q_stride[0] +
                          (int64_t)(hk * G + r % G) * a.q_stride[1] + t * E;
#pragma unroll
      for (int c = 0; c < D / (4 * E); ++c)
#pragma unroll
        for (int i = 0; i < E / 8; ++i) {
          uint4 u = make_uint4(0, 0, 0, 0);
          if (r < n_rows) u = __ldg(reinterpret_cast<const uint4*>(p + c * 4 * E + i * 8));
          f[c * (E / 4) + 2 * i] = make_uint2(u.x, u.y);
          f[c * (E / 4) + 2 * i + 1] = make_uint2(u.z, u.w);
        }
      up = 1.f;
      if constexpr (HELD8 && !F16) {
        unsigned top = 0;
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
          top = max(max(top, max(f[i].x & 0x7fffu, f[i].x >> 16 & 0x7fffu)), max(f[i].y & 0x7fffu, f[i].y >> 16 & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        top >>= 7;  // biased exponent
        up = __uint_as_float(max(1u, min(254u, 268u - min(268u, top))) << 23);
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          const float2 x = unpack2<false>(f[i].x), y = unpack2<false>(f[i].y);
          f[i] = make_uint2(pack2<true>(x.x * up, x.y * up), pack2<true>(y.x * up, y.y * up));
        }
      }
    };
    const bool cap = a.softcap > 0.f, bias = a.slopes != nullptr;
    const float pre = cap ? a.scale / a.softcap : a.scale * kLog2e, cap2 = a.softcap * kLog2e;
    // this thread's columns of a tile: query rows nb * 8 + 2t, 2t + 1
    float qf[NB][2];  // factor of the row's scores
    uint2 qr[Sh::kQShared ? 1 : NB][STEPS];
    static_assert(NB <= kWarps, "a warp a tile");
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float up;
      if constexpr (Sh::kQShared) {
        uint2 f[STEPS];
        load_q(nb, f, up);  // every warp needs the factors; one of them leaves the fragments
        if (warp == nb) {
#pragma unroll
          for (int i = 0; i < STEPS; ++i) sQ[(nb * STEPS + i) * 32 + lane] = f[i];
        }
      } else {
        load_q(nb, qr[nb], up);
      }
      qf[nb][0] = pre / __shfl_sync(0xffffffffu, up, 8 * t);
      qf[nb][1] = pre / __shfl_sync(0xffffffffu, up, 8 * t + 4);
    }
    if constexpr (Sh::kQShared) __syncthreads();

    constexpr int MI = VC * VE / 2;  // accumulators of a tile: 16 output channels each
    float acc[NB][MI][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nb][i][e] = 0.f;
    float m[NB][2], l[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) m[nb][0] = m[nb][1] = -INFINITY, l[nb][0] = l[nb][1] = 0.f;
    float v_ref = kLeastScale;  // 8 bits: power of two at or above the value scales so far, which acc is relative to
    const uint32_t k_at = swz(g, t), v_at0 = swz(2 * t, g * VB >> 4) + (g * VB & 15),
                   v_at1 = swz(2 * t + 1, g * VB >> 4) + (g * VB & 15);

    for (int slot = 0; key < k1; key += kStride, slot = slot + 1 == STAGES ? 0 : slot + 1) {
      cp_wait<STAGES - 2>();
      __syncwarp();  // every lane's copies of this step have landed, and its reads of the last one are done
      fetch_next(slot == 0 ? STAGES - 1 : slot - 1);
      const uint32_t base = ring + slot * Sh::kStage;
      const unsigned missing = bad >> (NT * slot) & ((1u << NT) - 1);
      // S^T: sc[nb][k2][e]: key 16 k2 + g + 8 (e / 2), row nb * 8 + 2t + e % 2
      float sc[NB][NT / 2][4], s2[NB == 1 ? NT / 2 : 1][4];  // one row tile: even and odd steps apart (two chains)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int k2 = 0; k2 < NT / 2; ++k2)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc[nb][k2][e] = 0.f;
            if constexpr (NB == 1) s2[k2][e] = 0.f;
          }
#pragma unroll
      for (int c = 0; c < D / (4 * E); ++c) {
        uint32_t kr[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) lds<4>(kr[j], base + (k_at ^ (uint32_t)(c << 6)) + j * 8 * ROW);
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
          const int st = c * (E / 4) + i;
#pragma unroll
          for (int k2 = 0; k2 < NT / 2; ++k2) {
            uint32_t ka[4];
            if constexpr (HELD8) {
              widen_row<KIND>(kr[2 * k2][i], ka[0], ka[2]);
              widen_row<KIND>(kr[2 * k2 + 1][i], ka[1], ka[3]);
            } else {
              ka[0] = kr[2 * k2][2 * i];
              ka[2] = kr[2 * k2][2 * i + 1];
              ka[1] = kr[2 * k2 + 1][2 * i];
              ka[3] = kr[2 * k2 + 1][2 * i + 1];
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              const uint2 qb = Sh::kQShared ? sQ[(nb * STEPS + st) * 32 + lane] : qr[Sh::kQShared ? 0 : nb][st];
              mma<HALF>(NB == 1 && (st & 1) ? s2[NB == 1 ? k2 : 0] : sc[nb][k2], ka, qb.x, qb.y);
            }
          }
        }
      }
      if constexpr (NB == 1) {
#pragma unroll
        for (int k2 = 0; k2 < NT / 2; ++k2)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[0][k2][e] += s2[k2][e];
      }
      float kf[NT], vf[NT];  // scales of key 8 j + g
      if constexpr (HELD8) {
        float v_new = 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(kf[j]) : "r"(base + 2 * Sh::kTile + (8 * j + g) * 4));
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vf[j]) : "r"(base + 2 * Sh::kTile + KEYS * 4 + (8 * j + g) * 4));
          v_new = fmaxf(v_new, vf[j]);
        }
        if (__any_sync(0xffffffffu, v_new > v_ref)) {
          const unsigned top = __reduce_max_sync(0xffffffffu, __float_as_uint(v_new));
          const float up = scale_above(top);
          const float f = v_ref / up;
          v_ref = up;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[nb][i][e] *= f;
        }
        const float inv = __uint_as_float(0x7f000000u - __float_as_uint(v_ref)) * kPUp;
#pragma unroll
        for (int j = 0; j < NT; ++j) vf[j] *= inv;
      }
      // exponents of 2, masked; then the probabilities
      const bool edge = key + KEYS > (a.tree ? ctx : ctx + 1) || missing;
      uint32_t pb[NB][NT];  // P^T as operands
      bool move = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int x = 0; x < 2; ++x) sc[nb][j / 2][2 * (j & 1) + x] *= HELD8 ? kf[j] * qf[nb][x] : qf[nb][x];
        if (cap) {
          float top = 0.f;
#pragma unroll
          for (int k2 = 0; k2 < NT / 2; ++k2)
#pragma unroll
            for (int e = 0; e < 4; e += 2) top = sm100::max3f(top, fabsf(sc[nb][k2][e]), fabsf(sc[nb][k2][e + 1]));
          auto each = [&](auto near) {
#pragma unroll
            for (int k2 = 0; k2 < NT / 2; ++k2)
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                float& x = sc[nb][k2][e];
                float& y = sc[nb][k2][e + 1];
                if constexpr (decltype(near)::value) tanh_near(x, y);
                else tanh_any(x, y);
                x *= cap2;
                y *= cap2;
              }
          };
          if (__all_sync(0xffffffffu, top <= 1.f)) each(std::true_type{});  // all below the cap
          else each(std::false_type{});
        }
        if (bias) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int r = min(r0 + nb * 8 + 2 * t + x, n_rows - 1);
            // the distance as a whole number first: positions past 2^24 are none in fp32
            const float slope2 = __ldg(a.slopes + hk * G + r % G) * kLog2e, d0 = (float)(ctx + r / G - key - g);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              float& y = sc[nb][j / 2][2 * (j & 1) + x];
              y = fmaf(-slope2, fabsf(d0 - (float)(8 * j)), y);
            }
          }
        }
        if (edge) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int r = r0 + nb * 8 + 2 * t + x;
            const int limit = r < n_rows ? (a.tree ? ctx : ctx + r / G + 1) : 0;  // keys below are seen
            uint64_t bits = 0;
            if (a.tree && r < n_rows) bits = __ldg(reinterpret_cast<const unsigned long long*>(a.tree) + tok0 + r / G);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              const int kk = key + 8 * j + g;
              bool seen = kk < limit;
              if (a.tree && kk >= ctx) seen = (bits >> (kk - ctx)) & 1;
              if (!seen || kk >= k1 || (missing >> j) & 1) sc[nb][j / 2][2 * (j & 1) + x] = -INFINITY;
            }
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float mx = -INFINITY;
#pragma unroll
          for (int k2 = 0; k2 < NT / 2; ++k2) mx = sm100::max3f(mx, sc[nb][k2][x], sc[nb][k2][2 + x]);
          move |= mx > m[nb][x] + 8.f;
        }
      }
      // The reference of the exponents moves only when some key exceeds it by
      // more than 8 (so P stays <= 2^8), which most steps settle by one vote.
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float alpha[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float mx = m[nb][x];
#pragma unroll
            for (int k2 = 0; k2 < NT / 2; ++k2) mx = sm100::max3f(mx, sc[nb][k2][x], sc[nb][k2][2 + x]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            alpha[x] = mx > m[nb][x] ? sm100::fast_exp2(m[nb][x] - mx) : 1.f;
            m[nb][x] = mx;
            l[nb][x] *= alpha[x];
          }
#pragma unroll
          for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nb][i][e] *= alpha[e & 1];
        }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const float ref0 = m[nb][0] == -INFINITY ? 0.f : m[nb][0], ref1 = m[nb][1] == -INFINITY ? 0.f : m[nb][1];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const float p0 = sm100::fast_exp2(sc[nb][j / 2][2 * (j & 1)] - ref0);
          const float p1 = sm100::fast_exp2(sc[nb][j / 2][2 * (j & 1) + 1] - ref1);
          l[nb][0] += p0;
          l[nb][1] += p1;
          pb[nb][j] = transpose8(HELD8 ? pack2<true>(p0 * vf[j], p1 * vf[j]) : pack2<HALF>(p0, p1));
        }
      }
#pragma unroll
      for (int k2 = 0; k2 < NT / 2; ++k2)  // 16 keys
#pragma unroll
        for (int c = 0; c < VC; ++c) {
          uint32_t vr[2][2][VW];  // [tile of 8 keys][row 2t + x]
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            lds<VW>(vr[j][0], base + Sh::kTile + v_at0 + c * 128 + (2 * k2 + j) * 8 * ROW);
            lds<VW>(vr[j][1], base + Sh::kTile + v_at1 + c * 128 + (2 * k2 + j) * 8 * ROW);
          }
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            constexpr int N = HELD8 ? 4 : 2;  // columns of a word
            uint32_t b[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if constexpr (HELD8) {
                widen_cols<KIND>(vr[j][0][w], vr[j][1][w], b[j]);
              } else {
                b[j][0] = __byte_perm(vr[j][0][w], vr[j][1][w], 0x5410);
                b[j][1] = __byte_perm(vr[j][0][w], vr[j][1][w], 0x7632);
              }
            }
#pragma unroll
            for (int i = 0; i < N; i += 2) {
              const uint32_t va[4] = {b[0][i], b[0][i + 1], b[1][i], b[1][i + 1]};
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma<HALF>(acc[nb][(c * VE + w * N + i) / 2], va, pb[nb][2 * k2], pb[nb][2 * k2 + 1]);
            }
          }
        }
    }

    // ------------------------------------------------------------ the warps' results
    cp_wait<0>();
    __syncthreads();  // the ring's space is reused
    const float back = HELD8 ? v_ref / kPUp : 1.f;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[nb][x] += __shfl_xor_sync(0xffffffffu, l[nb][x], 4);
        l[nb][x] += __shfl_xor_sync(0xffffffffu, l[nb][x], 8);
        l[nb][x] += __shfl_xor_sync(0xffffffffu, l[nb][x], 16);
        const int row = warp * NB * 8 + nb * 8 + 2 * t + x;
        if (g == 0) {
          sML[row * 2] = m[nb][x];
          sML[row * 2 + 1] = l[nb][x];
        }
        // accumulator i, element e: row 2t + e % 2, column i * 2 + e / 2 of the
        // lane's: channel c * 8 VE + g * VE + column % VE
#pragma unroll
        for (int i = 0; i < MI; i += 2) {
          const int col = 2 * i, ch = col / VE * 8 * VE + g * VE + col % VE;
          *reinterpret_cast<float4*>(sO + row * Sh::kOutRow + ch) =
              make_float4(acc[nb][i][x] * back, acc[nb][i][2 + x] * back, acc[nb][i + 1][x] * back,
                          acc[nb][i + 1][2 + x] * back);
        }
      }
    __syncthreads();
    for (int i = threadIdx.x; i < NB * 8 * D / 4; i += kThreads) {
      const int r = i / (D / 4), ch = i % (D / 4) * 4;
      const int rr = r0 + r;
      if (rr >= n_rows) break;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sML[(w * NB * 8 + r) * 2]);
      const float ref = mm == -INFINITY ? 0.f : mm;
      float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = sm100::fast_exp2(sML[(w * NB * 8 + r) * 2] - ref);
        const float4 u = *reinterpret_cast<const float4*>(sO + (w * NB * 8 + r) * Sh::kOutRow + ch);
        sum = fmaf(f, sML[(w * NB * 8 + r) * 2 + 1], sum);
        o[0] = fmaf(f, u.x, o[0]);
        o[1] = fmaf(f, u.y, o[1]);
        o[2] = fmaf(f, u.z, o[2]);
        o[3] = fmaf(f, u.w, o[3]);
      }
      if (piece.whole) {
        const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
        const int64_t out = (int64_t)(tok0 + rr / G) * a.Hq + hk * G + rr % G;
        reinterpret_cast<uint2*>(a.o)[(out * D + ch) / 4] =
            make_uint2(pack2<F16>(o[0] * inv, o[1] * inv), pack2<F16>(o[2] * inv, o[3] * inv));
      } else {
        // place 0: a block's first piece, which another one began; place 1: its last, which it begins
        const int64_t at = ((int64_t)blockIdx.x * 2 + piece.begun) * (8 * NB) + r;
        *reinterpret_cast<float4*>(a.part_o + at * D + ch) = make_float4(o[0], o[1], o[2], o[3]);
        if (ch == 0) a.part_ml[at] = make_float2(mm, sum);
      }
    }
    __syncthreads();  // the next piece's ring and query fragments
  }
}

// the block that has unit u (block c of `blocks` takes [total c / blocks, total (c + 1) / blocks))
__device__ __forceinline__ int block_of(int64_t u, int64_t total, int blocks) {
  return (int)(((u + 1) * blocks + total - 1) / total - 1);
}

// Row r of a tile whose pieces the blocks [c0, c1] have, by L lanes, or by all
// PARTS * L threads of the block, each L of them a share of the pieces: a
// share's outputs (lane's groups of 4 channels) and its sum of exponentials.
template <int D, int L, int PARTS>
__device__ __forceinline__ float join_row(const CacheAttnArgs& a, int rows_per_tile, int c0, int c1, int r, bool live,
                                          float* sM, float4 (&o)[D / L / 4]) {
  const int part = PARTS == 1 ? 0 : threadIdx.x / L, lane = threadIdx.x % L;
  auto place = [&](int c) { return ((int64_t)c * 2 + (c == c0)) * rows_per_tile + r; };
  if (!live) c1 = c0 - 1;
  float mm = -INFINITY;
  for (int c = c0 + part * L + lane; c <= c1; c += PARTS * L) mm = fmaxf(mm, a.part_ml[place(c)].x);
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
  if constexpr (PARTS > 1) {
    if (lane == 0) sM[part] = mm;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < PARTS; ++w) mm = fmaxf(mm, sM[w]);
  }
  const float ref = mm == -INFINITY ? 0.f : mm;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < D / L / 4; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll(PARTS == 1 ? 2 : 8)
  for (int c = c0 + part; c <= c1; c += PARTS) {
    const float2 x = a.part_ml[place(c)];
    const float f = sm100::fast_exp2(x.x - ref);
    sum = fmaf(f, x.y, sum);
    const float4* po = reinterpret_cast<const float4*>(a.part_o + place(c) * D) + lane;
#pragma unroll
    for (int i = 0; i < D / L / 4; ++i) {
      const float4 p = po[i * L];
      o[i] = make_float4(fmaf(f, p.x, o[i].x), fmaf(f, p.y, o[i].y), fmaf(f, p.z, o[i].z), fmaf(f, p.w, o[i].w));
    }
  }
  return sum;
}
template <int D, bool F16, int L>
__device__ __forceinline__ void store_joined(const CacheAttnArgs& a, int64_t out, float sum, const float4 (&o)[D / L / 4]) {
  const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
  uint2* dst = reinterpret_cast<uint2*>(a.o) + out * (D / 4) + threadIdx.x % L;
#pragma unroll
  for (int i = 0; i < D / L / 4; ++i)
    dst[i * L] = make_uint2(pack2<F16>(o[i].x * inv, o[i].y * inv), pack2<F16>(o[i].z * inv, o[i].w * inv));
}

// Joins the pieces of the query rows that lie in several blocks.
//
// Rows in few pieces: blocks (x, ..) take the rows of the one (sequence, head,
// row tile) that block x of the work began and did not finish, if there is one,
// L lanes a row.  The work then goes by the blocks and not by the rows of the
// call, most of which one block has whole: 4096 sequences, 32 query heads:
// 19 us, and 1.3 ms with a warp for every row.
// MANY pieces a row, and few rows: block (i, r) takes row r of the i-th
// (sequence, head, row tile); L threads each take a share of its pieces, and the
// shares are joined in their order.  One sequence of 512K tokens: 7 us, 18 us by
// blocks.
constexpr int kJoinThreads = 256;
template <int D, bool F16, bool MANY, int L>
__global__ void __launch_bounds__(kJoinThreads)
    cache_attn_join_kernel(const __grid_constant__ CacheAttnArgs a, int rows_per_tile) {
  constexpr int PARTS = MANY ? kJoinThreads / L : 1;
  __shared__ float4 sO[PARTS][MANY ? L : 1];
  __shared__ float sL[PARTS], sM[PARTS];
  __shared__ int64_t scan[kJoinThreads / 32 + 1];
  const int lane = threadIdx.x & 31, G = a.Hq / a.c.heads;
  Seq seq{0, 0, 0};
  int hk = 0, rt = 0, c0 = 0, c1 = 0;
  if constexpr (!MANY) {
    const Stretch st = find_stretch<kJoinThreads / 32, true>(a, rows_per_tile, scan);
    if (st.u < st.u_end) {
      seq = load_seq(a, st.s, false);
      const int kt_n = key_units(seq.len), tiles = (seq.T * G + rows_per_tile - 1) / rows_per_tile;
      const int inst = (int)(st.in_seq / kt_n), last = (int)(st.in_seq % kt_n);
      const int64_t first = st.u_end - 1 - last;  // its first unit
      hk = inst / tiles, rt = inst % tiles;
      c0 = c1 = blockIdx.x;
      if (last >= kBegin && first + kBegin >= st.u && last + 1 < kt_n)  // some keys here, the first ones, and not all
        c1 = block_of(first + kt_n - 1, st.total, st.blocks);
    }
  } else {
    const int tiles_most = ((int)(a.max_tokens * (int64_t)G) + rows_per_tile - 1) / rows_per_tile;
    const int s = blockIdx.x / (a.c.heads * tiles_most);
    hk = blockIdx.x / tiles_most % a.c.heads;
    rt = blockIdx.x % tiles_most;
    int64_t before = 0, total = 0;  // units before the sequence, and of all
    for (int i = lane; i < a.seqs; i += 32) {
      const int64_t n = seq_units(a, load_seq(a, i, false), rows_per_tile);
      total += n;
      if (i < s) before += n;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, d);
      before += __shfl_xor_sync(0xffffffffu, before, d);
    }
    seq = load_seq(a, s, false);
    const int kt_n = key_units(seq.len), tiles = (seq.T * G + rows_per_tile - 1) / rows_per_tile;
    if (rt < tiles) {
      const int64_t end = before + (int64_t)(hk * tiles + rt + 1) * kt_n;
      const int blocks = (int)min((int64_t)a.blocks, total);
      c0 = block_of(end - kt_n + kBegin, total, blocks);
      c1 = block_of(end - 1, total, blocks);
    }
  }
  cudaGridDependencySynchronize();  // every block: what follows in the stream waits for this kernel alone
  if (c0 == c1) return;             // written by that block
  const int r = MANY ? blockIdx.y : (blockIdx.y * kJoinThreads + threadIdx.x) / L;
  const int row = rt * rows_per_tile + r;
  const bool live = r < rows_per_tile && row < seq.T * G;
  float4 o[D / L / 4];
  float sum = join_row<D, L, PARTS>(a, rows_per_tile, c0, c1, r, live, sM, o);
  if constexpr (MANY) {
    static_assert(D == 4 * L, "a group of channels a lane");
    const int part = threadIdx.x / L, at = threadIdx.x % L;
    sO[part][at] = o[0];
    if (at == 0) sL[part] = sum;
    __syncthreads();
    if (part > 0) return;
    sum = 0.f;
    o[0] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < PARTS; ++w) {
      const float4 p = sO[w][at];
      sum += sL[w];
      o[0] = make_float4(o[0].x + p.x, o[0].y + p.y, o[0].z + p.z, o[0].w + p.w);
    }
  }
  if (live)
    store_joined<D, F16, L>(a, (int64_t)(seq.tok0 + row / G) * a.Hq + hk * G + row % G, sum, o);
}

template <int D, int KIND, bool F16, int NB>
cudaError_t launch(const CacheAttnArgs& a, cudaStream_t st) {
  constexpr int smem = Shape<D, KIND, NB>::kSmem;
  auto* fn = cache_attn_kernel<D, KIND, F16, NB>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  fn<<<dim3((unsigned)a.blocks), kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

template <int D, int KIND, bool F16>
cudaError_t by_rows(const CacheAttnArgs& a, int tile, cudaStream_t st) {
  switch (tile) {
    case 8: return launch<D, KIND, F16, 1>(a, st);
    case 16: return launch<D, KIND, F16, 2>(a, st);
    default: return launch<D, KIND, F16, 4>(a, st);
  }
}
template <int D, bool F16>
cudaError_t by_kind(const CacheAttnArgs& a, int tile, cudaStream_t st) {
  switch (a.c.kind) {
    case LH_CACHE_E4M3: return by_rows<D, LH_CACHE_E4M3, F16>(a, tile, st);
    case LH_CACHE_INT8: return by_rows<D, LH_CACHE_INT8, F16>(a, tile, st);
    default: return by_rows<D, F16 ? LH_CACHE_FP16 : LH_CACHE_BF16, F16>(a, tile, st);
  }
}

template <int D, bool F16>
cudaError_t join(const CacheAttnArgs& a, int rows_per_tile, cudaStream_t st) {
  const int64_t tiles = (int64_t)a.seqs * a.c.heads *
                        (((int64_t)a.max_tokens * (a.Hq / a.c.heads) + rows_per_tile - 1) / rows_per_tile);
  const bool many = a.blocks >= 8 * tiles;  // pieces of a row
  // it may be brought up while the pieces run; it waits for them itself
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = many ? dim3((unsigned)tiles, (unsigned)rows_per_tile)
                     : dim3((unsigned)a.blocks, (unsigned)((rows_per_tile + 31) / 32));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (many) return cudaLaunchKernelEx(&cfg, cache_attn_join_kernel<D, F16, true, D / 4>, a, rows_per_tile);
  if (rows_per_tile == 8) return cudaLaunchKernelEx(&cfg, cache_attn_join_kernel<D, F16, false, D / 4>, a, rows_per_tile);
  return cudaLaunchKernelEx(&cfg, cache_attn_join_kernel<D, F16, false, 8>, a, rows_per_tile);
}

}  // namespace

// Blocks of a call and the rows of their places in the workspace: as many
// blocks as 148 SMs hold at once (three each, two with tiles of 32 rows, one
// with tiles of 128), and no more than the units that sequences as long as the table would have.  No
// sequence has more than one unit of keys: no places.
void cache_attn_plan(int64_t seqs, int64_t kv_heads, int64_t rows, int64_t longest, int64_t* blocks, int64_t* places) {
  const int64_t tile = cache_attn_row_tile(rows);
  const int64_t keys = (longest + kUnit - 1) / kUnit;
  const int64_t inst = seqs * kv_heads * ((rows + tile - 1) / tile);
  const int64_t fit = 148 * (tile == 128 ? 1 : tile == 32 ? 2 : 3);
  *blocks = inst > fit / keys ? fit : inst * keys;
  *places = keys > 1 ? *blocks * 2 * tile : 0;
}

cudaError_t launch_cache_join(const CacheAttnArgs& a, int dtype, int rows_per_tile, cudaStream_t st) {
  if (dtype == LH_FP16) return a.c.d == 128 ? join<128, true>(a, rows_per_tile, st) : join<64, true>(a, rows_per_tile, st);
  return a.c.d == 128 ? join<128, false>(a, rows_per_tile, st) : join<64, false>(a, rows_per_tile, st);
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, int dtype, cudaStream_t st) {
  const int tile = cache_attn_row_tile((int64_t)a.max_tokens * (a.Hq / a.c.heads));
  cudaError_t e;
  if (tile == 128) e = launch_cache_attn_rows(a, dtype, st);
  else if (dtype == LH_FP16) e = a.c.d == 128 ? by_kind<128, true>(a, tile, st) : by_kind<64, true>(a, tile, st);
  else e = a.c.d == 128 ? by_kind<128, false>(a, tile, st) : by_kind<64, false>(a, tile, st);
  return e == cudaSuccess && a.part_o ? launch_cache_join(a, dtype, tile, st) : e;
}

}  // namespace lh
