// The work list of the cache attention, shared by its kernels.
//
// The work is a list of units of 128 keys: sequence by sequence, for each of
// its heads and tiles of query rows all the keys.  As many blocks as the GPU
// holds at once take equal stretches of that list, whatever the lengths of the
// sequences are; a stretch may end inside one (sequence, head, row tile) and
// begin inside another.  What a block has of an unfinished one goes to one of
// its two places in the workspace; a second kernel joins those in block order,
// so that results do not depend on scheduling.
#pragma once

#include "lh_cache.cuh"
#include "lh_dense.cuh"

namespace lh {

constexpr int kUnit = 128;  // keys of a unit of work
// Units that a (sequence, head, row tile) counts before its keys, for what a
// block spends to begin and end one (measured: about what two units of keys
// cost); they come first and hold no keys.
constexpr int kBegin = 2;

// tokens of a sequence, cut to what the call allows (an error is reported
// once, by `report`)
struct Seq {
  int tok0, T, len;
};
__device__ __forceinline__ Seq load_seq(const CacheAttnArgs& a, int s, bool report) {
  Seq q{s, 1, __ldg(a.lens + s)};
  if (a.q_start) {
    q.tok0 = __ldg(a.q_start + s);
    q.T = __ldg(a.q_start + s + 1) - q.tok0;
  }
  const int most = a.width << a.c.log2_page;
  if (q.T < 0 || q.T > a.max_tokens || q.tok0 < 0 || q.tok0 + (int64_t)q.T > a.n_tok || q.len < 0 || q.len > most) {
    if (report) report_error(a.errw, ERRW_BOUNDS);
    q.T = max(0, min(q.T, a.max_tokens));
    if (q.tok0 < 0 || q.tok0 + (int64_t)q.T > a.n_tok) q.T = 0;
    q.len = max(0, min(q.len, most));
  }
  return q;
}
__device__ __forceinline__ int key_units(int len) { return kBegin + max(1, (len + kUnit - 1) / kUnit); }
// units of a sequence: heads x row tiles x units of each
__device__ __forceinline__ int64_t seq_units(const CacheAttnArgs& a, const Seq& q, int rows_per_tile) {
  const int tiles = (q.T * (a.Hq / a.c.heads) + rows_per_tile - 1) / rows_per_tile;
  return (int64_t)a.c.heads * tiles * key_units(q.len);
}
// A block's place in the work list, by all of its threads (WARPS warps).
struct Stretch {
  int64_t u, u_end;  // its units [u, u_end)
  int64_t in_seq;    // u (or the last of them) within its sequence
  int64_t total;     // units of the call
  int s;             // sequence
  int blocks;        // blocks that have any
};
// scan: WARPS + 1 int64 of shared memory.  A thread sums the units of a run of
// sequences; the one whose run holds the first unit (LAST: the last one) looks for its sequence.
template <int WARPS, bool LAST = false>
__device__ __forceinline__ Stretch find_stretch(const CacheAttnArgs& a, int rows_per_tile, int64_t* scan) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (a.seqs + WARPS * 32 - 1) / (WARPS * 32);
  const int s0 = min(a.seqs, (int)threadIdx.x * per), s1 = min(a.seqs, s0 + per);
  int64_t mine = 0;
  for (int i = s0; i < s1; ++i) mine += seq_units(a, load_seq(a, i, blockIdx.x == 0), rows_per_tile);
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  before += incl - mine;
  Stretch r;
  r.blocks = (int)min((int64_t)gridDim.x, total);  // no block of these has an empty stretch
  r.total = total;
  r.u = r.u_end = r.in_seq = 0;
  r.s = 0;
  if (blockIdx.x >= r.blocks) return r;
  r.u = total * blockIdx.x / r.blocks;
  r.u_end = total * (blockIdx.x + 1) / r.blocks;
  const int64_t wanted = LAST ? r.u_end - 1 : r.u;
  __syncthreads();
  if (wanted >= before && wanted < before + mine) {
    int i = s0;
    int64_t at = wanted - before;
    for (;;) {
      const int64_t n = seq_units(a, load_seq(a, i, false), rows_per_tile);
      if (at < n) break;
      at -= n;
      ++i;
    }
    scan[0] = at;
    scan[1] = i;
  }
  __syncthreads();
  r.in_seq = scan[0];
  r.s = (int)scan[1];
  return r;
}

// One piece of a block's stretch: keys [k0, k1) of one (sequence, head, row
// tile); whole: all of its keys, begun: its first ones.
struct Piece {
  Seq seq;
  int hk, rt, k0, k1;
  bool whole, begun;
};
// the next piece with keys, false at the stretch's end
__device__ __forceinline__ bool next_piece(const CacheAttnArgs& a, int rows_per_tile, Stretch& st, Seq& seq, Piece& p) {
  while (st.u < st.u_end) {
    const int kt_n = key_units(seq.len);
    const int tiles = (seq.T * (a.Hq / a.c.heads) + rows_per_tile - 1) / rows_per_tile;
    if (st.in_seq >= (int64_t)a.c.heads * tiles * kt_n) {  // the next sequence with units
      st.in_seq = 0;
      seq = load_seq(a, ++st.s, false);
      continue;
    }
    const int inst = (int)(st.in_seq / kt_n), from = (int)(st.in_seq % kt_n);
    const int to = (int)min((int64_t)kt_n, from + (st.u_end - st.u));
    st.u += to - from;
    st.in_seq += to - from;
    if (to <= kBegin) continue;  // no keys
    const int kt0 = max(from - kBegin, 0);
    p = {seq, inst / tiles, inst % tiles, kt0 * kUnit, min(seq.len, (to - kBegin) * kUnit), kt0 == 0 && to == kt_n,
         kt0 == 0};
    return true;
  }
  return false;
}

// A key head's rows [row, row + 8) among the cache's rows for the 8 keys from
// `key` (a multiple of 8) on, 0xffffffff where the page is not in the cache
__device__ __forceinline__ uint32_t key_rows(const CacheAttnArgs& a, const int32_t* table, int hk, int key) {
  const int p = __ldg(table + (key >> a.c.log2_page));
  if (p >= 0 && p < a.c.pages)
    return (((uint32_t)p * a.c.heads + hk) << a.c.log2_page) + (key & ((1 << a.c.log2_page) - 1));
  report_error(a.errw, ERRW_BOUNDS);
  return 0xffffffffu;
}

// The power of two that the values' scales are taken relative to: at or above
// the largest one (bits of a scale above kLeastScale), whose reciprocal, raised
// by the 2^6 of the probabilities, is finite.
constexpr float kLeastScale = 3.7615819226313200e-37f;  // 2^-121
__device__ __forceinline__ float scale_above(unsigned bits) {
  return __uint_as_float(min(253u, (bits + 0x7fffffu) >> 23) << 23);
}

// two e4m3 bytes (the low half of y) as fp16
__device__ __forceinline__ uint32_t e4m3_half2(uint32_t y) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(y));
  return r;
}
// bytes i and j of y, int8 values raised by 128, as fp16: the bits of 1024 + u
// less 1152
__device__ __forceinline__ uint32_t u8_half2(uint32_t y, int i, int j) {
  const uint32_t u = __byte_perm(y, 0x64646464u, (uint32_t)(i | 4 << 4 | j << 8 | 4 << 12));
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), off);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// the four values of a word of one row: (0, 1), (2, 3)
template <int KIND>
__device__ __forceinline__ void widen_row(uint32_t w, uint32_t& b0, uint32_t& b1) {
  if constexpr (KIND == LH_CACHE_E4M3) {
    b0 = e4m3_half2(w);
    b1 = e4m3_half2(w >> 16);
  } else {
    w ^= 0x80808080u;
    b0 = u8_half2(w, 0, 1);
    b1 = u8_half2(w, 2, 3);
  }
}
// the four columns of a word of two rows: b[i] = (x_i, z_i)
template <int KIND>
__device__ __forceinline__ void widen_cols(uint32_t x, uint32_t z, uint32_t (&b)[4]) {
  uint32_t lo = __byte_perm(x, z, 0x5140), hi = __byte_perm(x, z, 0x7362);
  if constexpr (KIND == LH_CACHE_E4M3) {
    b[0] = e4m3_half2(lo);
    b[1] = e4m3_half2(lo >> 16);
    b[2] = e4m3_half2(hi);
    b[3] = e4m3_half2(hi >> 16);
  } else {
    lo ^= 0x80808080u;
    hi ^= 0x80808080u;
    b[0] = u8_half2(lo, 0, 1);
    b[1] = u8_half2(lo, 2, 3);
    b[2] = u8_half2(hi, 0, 1);
    b[3] = u8_half2(hi, 2, 3);
  }
}

// launch of the join of the pieces of a call's rows (lh_cache_attn.cu)
cudaError_t launch_cache_join(const CacheAttnArgs& a, int dtype, int rows_per_tile, cudaStream_t st);
// more than 32 query rows of a key head: tiles of 128 on the tensor cores
// (lh_cache_attn_rows.cu)
cudaError_t launch_cache_attn_rows(const CacheAttnArgs& a, int dtype, cudaStream_t st);

}  // namespace lh
