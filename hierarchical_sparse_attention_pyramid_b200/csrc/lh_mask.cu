// Spans of the dense attention's masks (lh_dense.cuh): for every token the
// interval of keys that it sees as a query and the interval of queries that
// see it as a key, and their bounds over tiles of 128 tokens.
//
// One block per row of the batch.  A thread owns a run of consecutive tokens;
// the document starts before it and the ends and plain tokens after it come
// from two block scans, so that a row is read twice however its documents lie.
// 16K tokens take a few microseconds, once per batch (all layers share it).
#include "lh_common.cuh"
#include "lh_dense.cuh"

namespace lh {
namespace {

constexpr int kThreads = 1024;

// exclusive scan over the block's threads with op (identity id); reversed:
// over the threads after this one.  `scratch` holds 32 ints.
template <bool REV, typename Op>
__device__ __forceinline__ int block_scan(int v, int id, int* scratch, Op op) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = REV ? __shfl_down_sync(0xffffffffu, x, d) : __shfl_up_sync(0xffffffffu, x, d);
    if (REV ? lane + d < 32 : lane >= d) x = op(x, y);
  }
  __syncthreads();
  if (lane == (REV ? 0 : 31)) scratch[warp] = x;
  __syncthreads();
  int before = id;
  if (REV) {
    for (int w = warp + 1; w < kThreads / 32; ++w) before = op(before, scratch[w]);
  } else {
    for (int w = 0; w < warp; ++w) before = op(before, scratch[w]);
  }
  int prev = REV ? __shfl_down_sync(0xffffffffu, x, 1) : __shfl_up_sync(0xffffffffu, x, 1);
  if (lane == (REV ? 31 : 0)) prev = id;
  return op(before, prev);
}

__global__ void __launch_bounds__(kThreads)
    mask_spans_kernel(const int32_t* __restrict__ docs, const uint8_t* __restrict__ prefix, int N, int causal,
                      int4* __restrict__ row_tile, int4* __restrict__ col_tile, int2* rows, int2* cols, int* plain_from) {
  __shared__ int scratch[32];
  const int64_t base = (int64_t)blockIdx.x * N;
  const int per = (N + kThreads - 1) / kThreads;
  const int i0 = min(N, (int)threadIdx.x * per), i1 = min(N, i0 + per);
  auto doc = [&](int i) { return docs ? __ldg(docs + base + i) : 0; };
  auto edge = [&](int i) { return i == 0 || (docs && doc(i) != doc(i - 1)); };  // a document starts at i
  auto plain = [&](int i) { return !(prefix && __ldg(prefix + base + i)); };
  int last_edge = -1, first_edge = N, first_plain = N;
  for (int i = i0; i < i1; ++i) {
    if (edge(i)) {
      last_edge = i;
      if (first_edge == N) first_edge = i;
    }
    if (first_plain == N && plain(i)) first_plain = i;
  }
  auto mx = [](int x, int y) { return max(x, y); };
  auto mn = [](int x, int y) { return min(x, y); };
  int start = block_scan<false>(last_edge, -1, scratch, mx);
  int end = block_scan<true>(first_edge, N, scratch, mn);
  int next_plain = block_scan<true>(first_plain, N, scratch, mn);
  // backwards: the first plain token from each token on, and the end of its
  // document
  for (int i = i1 - 1; i >= i0; --i) {
    if (plain(i)) next_plain = i;
    plain_from[base + i] = next_plain;
    cols[base + i].y = end;
    if (edge(i)) end = i;
  }
  __syncthreads();
  // forwards: a document's prefix ends at the first plain token from its start on
  for (int i = i0; i < i1; ++i) {
    if (edge(i)) start = i;
    const int e = cols[base + i].y;
    const int pre = min(plain_from[base + start], e);
    const bool pad = doc(i) < 0;
    rows[base + i] = pad ? make_int2(0, 0) : make_int2(start, causal ? max(i + 1, pre) : e);
    cols[base + i] = pad ? make_int2(0, 0) : make_int2(causal && i >= pre ? i : start, e);
  }
  __syncthreads();
  // bounds over tiles, a warp each; one empty row leaves nothing that all see
  const int lane = threadIdx.x & 31, tiles = (N + 127) / 128;
  for (int w = threadIdx.x >> 5; w < 2 * tiles; w += kThreads / 32) {
    const bool is_row = w < tiles;
    const int t = is_row ? w : w - tiles;
    const int2* v = (is_row ? rows : cols) + base;
    int min_lo = N, max_hi = 0, max_lo = 0, min_hi = N;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = t * 128 + r * 32 + lane;
      if (i >= N) continue;
      const int2 s = v[i];
      if (s.y > s.x) {
        min_lo = min(min_lo, s.x);
        max_hi = max(max_hi, s.y);
        max_lo = max(max_lo, s.x);
        min_hi = min(min_hi, s.y);
      } else {
        min_hi = 0;
      }
    }
    min_lo = __reduce_min_sync(0xffffffffu, min_lo);
    max_hi = __reduce_max_sync(0xffffffffu, max_hi);
    max_lo = __reduce_max_sync(0xffffffffu, max_lo);
    min_hi = __reduce_min_sync(0xffffffffu, min_hi);
    if (lane == 0)
      (is_row ? row_tile : col_tile)[(int64_t)blockIdx.x * tiles + t] =
          max_hi > min_lo ? make_int4(min_lo, max_hi, max_lo, min_hi) : make_int4(0, 0, 0, 0);
  }
}

}  // namespace

cudaError_t launch_mask_spans(const int32_t* docs, const uint8_t* prefix, int64_t B, int N, int causal,
                              const SpanBuffer& s, cudaStream_t st) {
  mask_spans_kernel<<<dim3((unsigned)B), kThreads, 0, st>>>(docs, prefix, N, causal, s.row_tile, s.col_tile, s.rows,
                                                            s.cols, s.plain_from);
  return cudaGetLastError();
}

}  // namespace lh
