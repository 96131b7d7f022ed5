// The paged key/value cache: shared types of its write, read and attention
// kernels.  A page holds `page` tokens of every head, [heads][page][d], so a
// head's rows within a page are contiguous; 8-bit kinds keep one fp32 scale
// per token and head.
#pragma once

#include "lh_common.cuh"

namespace lh {

struct CacheView {
  void *k, *v;              // [pages][heads][page][d]
  float *k_scale, *v_scale; // [pages][heads][page], 8-bit kinds
  int64_t pages;
  int log2_page, heads, d, kind;
};

struct CacheIoArgs {
  CacheView c;
  int64_t n;                    // tokens: of the write, of the read's outputs
  const void *k, *v;            // write: [n][heads][d] with {token, head} strides
  int64_t k_stride[2], v_stride[2];
  const int64_t* slots;         // write: page * page_size + row of each token; negative: skipped
  const int32_t* table;         // read: [seqs][width] page of each page-sized run of positions
  const int32_t* starts;        // read: [seqs + 1] first output row of each sequence
  int seqs, width;
  void *k_out, *v_out;          // read: [n][heads][d]
  int* errw;
};

struct CacheAttnArgs {
  CacheView c;
  const void* q;                // [n_tok][Hq][d] with {token, head} strides
  int64_t q_stride[2];
  void* o;                      // [n_tok][Hq][d]
  int64_t n_tok;
  const int32_t *table, *lens, *q_start;  // q_start NULL: one token a sequence
  const uint64_t* tree;         // [n_tok] or NULL
  const float* slopes;          // [Hq] or NULL
  int seqs, width, Hq, max_tokens;
  float scale, softcap;
  int blocks;                   // of the grid, which share the work out (cache_attn_plan)
  float* part_o;                // [blocks][2][row tile][d], NULL where no row can be in several blocks
  float2* part_ml;              // [blocks][2][row tile] running maximum (log2 domain) and sum
  int* errw;
};

cudaError_t launch_cache_write(const CacheIoArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_cache_read(const CacheIoArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_cache_attn(const CacheAttnArgs& a, int dtype, cudaStream_t st);
// blocks of a call, and rows of its workspace (host only)
void cache_attn_plan(int64_t seqs, int64_t kv_heads, int64_t rows, int64_t longest, int64_t* blocks, int64_t* places);

}  // namespace lh
