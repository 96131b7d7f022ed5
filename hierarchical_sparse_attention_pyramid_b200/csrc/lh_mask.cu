// Spans of the dense attention's masks (lh_dense.cuh): for every token the
// interval of keys that it sees as a query and the interval of queries that
// see it as a key, and their bounds over tiles of 128 tokens.
//
// One block per row of the batch.  A thread owns 32 consecutive tokens as bit
// masks: where documents start, where plain (not prefix) tokens are, where
// padding is.  The masks come from ballots over coalesced loads; what lies
// before and after a thread's tokens comes from three block scans; the spans
// then follow from the masks by bit operations, 32 tokens of one thread at a
// time, again with coalesced stores.  Bound by latency: 8K tokens take
// 13 us, 257 tokens 6, once per batch (every layer and both directions share it).
#include "lh_common.cuh"
#include "lh_dense.cuh"

namespace lh {
namespace {

constexpr int kThreads = 1024, kWarps = 32;

// exclusive scan over the block's threads (REV: over the threads after this
// one) with op and its identity; all: the whole block's value
template <bool REV, typename T, typename Op>
__device__ __forceinline__ T block_scan(T v, T id, T* scratch, Op op, T& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T y = REV ? __shfl_down_sync(0xffffffffu, x, d) : __shfl_up_sync(0xffffffffu, x, d);
    if (REV ? lane + d < 32 : lane >= d) x = op(x, y);
  }
  __syncthreads();
  if (lane == (REV ? 0 : 31)) scratch[warp] = x;
  __syncthreads();
  // every warp scans the 32 warps' values
  const T w = scratch[lane];
  T before = (REV ? lane > warp : lane < warp) ? w : id;
  all = w;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    before = op(before, __shfl_xor_sync(0xffffffffu, before, d));
    all = op(all, __shfl_xor_sync(0xffffffffu, all, d));
  }
  T prev = REV ? __shfl_down_sync(0xffffffffu, x, 1) : __shfl_up_sync(0xffffffffu, x, 1);
  if (lane == (REV ? 31 : 0)) prev = id;
  return op(before, prev);
}

struct Bounds {
  int min_lo, max_hi, max_lo, min_hi;
};
__device__ __forceinline__ void widen(Bounds& b, int2 s, bool in) {
  // rows past N do not count; an empty one leaves nothing that all see
  const bool full = in && s.y > s.x;
  b.min_lo = min(b.min_lo, __reduce_min_sync(0xffffffffu, full ? s.x : 0x7fffffff));
  b.max_hi = max(b.max_hi, __reduce_max_sync(0xffffffffu, full ? s.y : 0));
  b.max_lo = max(b.max_lo, __reduce_max_sync(0xffffffffu, full ? s.x : 0));
  b.min_hi = min(b.min_hi, __reduce_min_sync(0xffffffffu, !in ? 0x7fffffff : full ? s.y : 0));
}
__device__ __forceinline__ int4 bounds_of(const Bounds& b) {
  return b.max_hi > b.min_lo ? make_int4(b.min_lo, b.max_hi, b.max_lo, b.min_hi) : make_int4(0, 0, 0, 0);
}

// K: threads of a warp that own tokens, a multiple of 4, so that a warp holds
// whole tiles (a warp takes 32 K tokens, the block 1024 K at a time)
__global__ void __launch_bounds__(kThreads)
    mask_spans_kernel(const int32_t* __restrict__ docs, const uint8_t* __restrict__ prefix, int N, int causal, int K,
                      int4* __restrict__ row_tile, int4* __restrict__ col_tile, int2* __restrict__ rows,
                      int2* __restrict__ cols, int* scratch, int* __restrict__ padded) {
  __shared__ int sInt[kWarps];
  __shared__ uint64_t sLong[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t base = (int64_t)blockIdx.x * N;
  const int per = kThreads * K, chunks = (N + per - 1) / per, tiles = (N + 127) / 128;
  // a chunk's masks, kept between the two passes where there is more than one
  // (3 words a thread, then what follows the chunk: of the row's N words)
  int* kept = scratch + base;
  auto mx = [](uint64_t x, uint64_t y) { return x > y ? x : y; };
  auto mn = [](int x, int y) { return min(x, y); };

  uint32_t edges = 0, plains = 0, pads = 0;
  auto load_masks = [&](int i0) {  // of the warp's tokens from i0 on
    edges = plains = pads = 0;
#pragma unroll 8
    for (int k = 0; k < K; ++k) {
      const int i = i0 + k * 32 + lane;
      int id = 0, prev = 0;
      bool pre = false;
      if (i < N) {
        if (docs) {
          id = __ldg(docs + base + i);
          prev = i > 0 ? __ldg(docs + base + i - 1) : 0;
        }
        pre = prefix && __ldg(prefix + base + i);
      }
      const uint32_t e = __ballot_sync(0xffffffffu, i < N && (i == 0 || id != prev));
      const uint32_t p = __ballot_sync(0xffffffffu, i < N && !pre);
      const uint32_t n = __ballot_sync(0xffffffffu, id < 0);
      if (lane == k) edges = e, plains = p, pads = n;
    }
  };
  // backwards over the chunks: what follows each
  int any_pad = 0;
  int after_edge = N, after_plain = N;  // first document start, first plain token after the chunk
  for (int c = chunks - 1; c >= 0; --c) {
    const int i0 = c * per + warp * 32 * K, own = i0 + lane * 32;
    load_masks(i0);
    any_pad |= pads != 0;
    if (chunks > 1) {
      int* k = kept + c * (per / 32 * 3 + 2);
      if (lane < K) {
        k[(warp * K + lane) * 3] = (int)edges;
        k[(warp * K + lane) * 3 + 1] = (int)plains;
        k[(warp * K + lane) * 3 + 2] = (int)pads;
      }
      if (threadIdx.x == 0) k[per / 32 * 3] = after_edge, k[per / 32 * 3 + 1] = after_plain;
      if (c > 0) {
        int all_edge, all_plain;
        block_scan<true>(edges ? own + __ffs(edges) - 1 : 0x7fffffff, 0x7fffffff, sInt, mn, all_edge);
        block_scan<true>(plains ? own + __ffs(plains) - 1 : 0x7fffffff, 0x7fffffff, sInt, mn, all_plain);
        after_edge = min(after_edge, all_edge);
        after_plain = min(after_plain, all_plain);
      }
    }
  }
  any_pad = __syncthreads_or(any_pad);
  if (threadIdx.x == 0) padded[blockIdx.x] = any_pad;
  // forwards: the spans.  carry: start of the document that a chunk begins in
  // and the end of its prefix
  uint64_t carry = 0;
  for (int c = 0; c < chunks; ++c) {
    const int i0 = c * per + warp * 32 * K, own = i0 + lane * 32;
    if (chunks > 1) {
      const int* k = kept + c * (per / 32 * 3 + 2);
      edges = plains = pads = 0;
      if (lane < K) {
        edges = (uint32_t)k[(warp * K + lane) * 3];
        plains = (uint32_t)k[(warp * K + lane) * 3 + 1];
        pads = (uint32_t)k[(warp * K + lane) * 3 + 2];
      }
      after_edge = k[per / 32 * 3], after_plain = k[per / 32 * 3 + 1];
    }
    int all;
    const int next_edge =
        min(after_edge, block_scan<true>(edges ? own + __ffs(edges) - 1 : 0x7fffffff, 0x7fffffff, sInt, mn, all));
    const int next_plain =
        min(after_plain, block_scan<true>(plains ? own + __ffs(plains) - 1 : 0x7fffffff, 0x7fffffff, sInt, mn, all));
    // the last document that starts in the thread's tokens, and its prefix's end
    uint64_t last = 0;
    if (edges) {
      const int sb = 31 - __clz(edges);
      const uint32_t p = plains >> sb;
      last = (uint64_t)(own + sb) << 32 | (uint32_t)min(p ? own + sb + __ffs(p) - 1 : next_plain, next_edge);
    }
    uint64_t all_last;
    const uint64_t begun = mx(carry, block_scan<false>(last, (uint64_t)0, sLong, mx, all_last));
    carry = mx(carry, all_last);
    Bounds rb{}, cb{};
    for (int k = 0; k < K; ++k) {  // the 32 tokens of lane k
      const int o = i0 + k * 32, i = o + lane;
      if (o >= N) break;
      const uint32_t e = __shfl_sync(0xffffffffu, edges, k), pl = __shfl_sync(0xffffffffu, plains, k);
      const uint32_t pd = __shfl_sync(0xffffffffu, pads, k);
      const int ne = __shfl_sync(0xffffffffu, next_edge, k), np = __shfl_sync(0xffffffffu, next_plain, k);
      const uint64_t bg = __shfl_sync(0xffffffffu, begun, k);
      const uint32_t upto = 0xffffffffu >> (31 - lane);  // bits 0 .. lane
      const uint32_t behind = e & upto, ahead = e & ~upto;
      const int end = ahead ? o + __ffs(ahead) - 1 : ne;
      int start = (int)(bg >> 32), pre = (int)(uint32_t)bg;
      if (behind) {
        const int sb = 31 - __clz(behind);
        const uint32_t p = pl >> sb;
        start = o + sb;
        pre = min(p ? start + __ffs(p) - 1 : np, end);
      }
      int2 r = make_int2(start, causal ? max(i + 1, pre) : end);
      int2 q = make_int2(causal && i >= pre ? i : start, end);
      if (pd >> lane & 1) r = q = make_int2(0, 0);
      if (i < N) {
        rows[base + i] = r;
        cols[base + i] = q;
      }
      if ((o & 127) == 0) rb = cb = Bounds{0x7fffffff, 0, 0, 0x7fffffff};
      widen(rb, r, i < N);
      widen(cb, q, i < N);
      if (((o & 127) == 96 || o + 32 >= N) && lane == 0) {
        row_tile[(int64_t)blockIdx.x * tiles + (o >> 7)] = bounds_of(rb);
        col_tile[(int64_t)blockIdx.x * tiles + (o >> 7)] = bounds_of(cb);
      }
    }
  }
}

}  // namespace

cudaError_t launch_mask_spans(const int32_t* docs, const uint8_t* prefix, int64_t B, int N, int causal,
                              const SpanBuffer& s, cudaStream_t st) {
  int K = ((N + kThreads - 1) / kThreads + 3) / 4 * 4;
  if (K > 32) K = 32;
  mask_spans_kernel<<<dim3((unsigned)B), kThreads, 0, st>>>(docs, prefix, N, causal, K, s.row_tile, s.col_tile, s.rows,
                                                            s.cols, s.scratch, s.padded);
  return cudaGetLastError();
}

}  // namespace lh
