// Internal launch interface of the drafted-decoding calls (draft_api.cu to the kernels).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/tts_decode.h"
#include "cache_view.cuh"

namespace tts {

// Rows b*T + t of k and v into the cache at start[b] + t (write), or back out (read).
struct KvRowsParams {
  const void* k;         // write: source rows (f32, or bf16 when row_bf16)
  const void* v;
  void* k_out;           // read: destination rows
  void* v_out;
  int64_t row_stride;    // elements
  int row_bf16;
  CacheView cache;
  int kv_dtype, head_dim;
  const int32_t* start;
  const int32_t* n_rows; // may be null
  int T;
  int n_sm;
  int32_t* err;
};

struct CommitParams {
  CacheView cache;
  int row_bytes;
  const int32_t* n_past;
  const int32_t* path;
  int64_t path_stride;
  const int32_t* n_accept;
  int T;
  int32_t* err;
};

struct RopeRowsParams {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
  int in_bf16, out_bf16;
  const float* gamma_q;  // null: no norm
  const float* gamma_k;
  float eps;
  const int32_t* pos;
  int rows, n_q_heads, n_kv_heads, head_dim, rot_dim, interleaved;
  const float2* cs;
  int max_pos;
  int n_sm;
  int32_t* err;
};

struct RopeTableParams {
  float2* cs;
  int max_pos, rot_dim;
  double base;
  tts_rope_scaling s;
};

// Tree attention.  The query rows of a stream and kv head are r = t * G + h (node t, q head h
// of the group), taken in blocks of `rows` rows; an item is (stream, kv head, row block).
struct TreeParams {
  const void* q;
  int64_t q_stride;
  int q_bf16;
  CacheView cache;
  const int32_t* n_past;
  const int32_t* n_nodes;      // may be null
  const uint64_t* mask;        // may be null: the chain
  int T, group, n_q_heads;
  float scale_log2;            // scale * log2(e)
  void* out;
  int n_rb, rows;              // row blocks of a (stream, kv head), rows of a block
  int tile;                    // cache rows of a tile
  int n_cta;                   // CTAs the work is cut over
  int fixed;                   // an item's cost beside its tiles (a tile costs 4)
  int whole;                   // 1: one CTA takes whole items only (no partials)
  float* part;                 // partial rows [n_cta][2][rows][D]
  float2* ml;                  // their (maximum, sum) [n_cta][2][rows]
  int32_t* err;
};

cudaError_t launch_kv_write(const KvRowsParams& p, cudaStream_t s);
cudaError_t launch_kv_read(const KvRowsParams& p, cudaStream_t s);
cudaError_t launch_commit(const CommitParams& p, cudaStream_t s);
cudaError_t launch_rope_rows(const RopeRowsParams& p, cudaStream_t s);
cudaError_t launch_rope_table_scaled(const RopeTableParams& p, cudaStream_t s);
cudaError_t launch_tree_attn(const TreeParams& p, int kv_dtype, int head_dim, cudaStream_t s);
bool tree_attn_tc_supported(const tts_kv_desc* d);
cudaError_t launch_tree_attn_tc(const TreeParams& p, int kv_dtype, int head_dim, cudaStream_t s);
cudaError_t launch_tree_combine(const TreeParams& p, int head_dim, cudaStream_t s);

}  // namespace tts
