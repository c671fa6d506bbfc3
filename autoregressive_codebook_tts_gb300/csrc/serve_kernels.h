// Internal launch interface of the calls that serve many requests at once (serve_api.cu to the
// kernels).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/tts_decode.h"
#include "cache_view.cuh"

namespace tts {

struct AddNormParams {
  const void* x;
  const void* res;      // may be null
  void* sum;            // may be null
  const float* gamma;
  void* out;
  float* out_scale;     // E4M3 only
  int64_t x_stride, res_stride, sum_stride, out_stride;
  float eps;
  int rows, n;
  int x_bf16, res_bf16, out_dtype;
};

struct PagePlanParams {
  int32_t* table;
  int B, capacity, page_shift, n_pages, bt_stride;
  int32_t* free_pages;
  int32_t* n_free;
  const int32_t* n_past;
  const int32_t* n_new;
  int T, max_rows;
  int32_t* n_rows;
  int32_t* row_start;
  int32_t* row_stream;
  int32_t* row_pos;
  int64_t* row_slot;
  int32_t* err;
};

// Rows of k and v into the cache rows `slot` of every kv head.
struct KvSlotsParams {
  const void* k;
  const void* v;
  int64_t row_stride;
  int row_bf16;
  CacheView cache;
  int64_t page_rows, n_slots;   // rows of a page (or of a contiguous stream), slots in all
  int kv_dtype, head_dim;
  const int64_t* slot;
  int rows;
  int32_t* err;
};

struct ProjectParams {
  const void* x;
  int64_t x_stride;
  int x_e4m3;
  const float* x_scale;
  const void* w;
  const float* w_scale;
  int n, k, rows;
  tts_adapters ad;              // n_adapters 0: none
  const int32_t* row_stream;    // may be null
  const int32_t* stream_adapter;
  int n_streams;
  void* out;
  int64_t out_stride;
  int out_bf16;
  // workspace: scale x A^T in f32 [rows][rank_max]; with tc also as three bf16 parts
  // [3][rows][rank_max], and each 16 rows' adapter (-1 none, -2 several)
  float* v;
  __nv_bfloat16* v_parts;
  int32_t* block_ad;
  int tc;                       // the adapters' products on the tensor cores too
  int32_t* err;
};

cudaError_t launch_add_norm(const AddNormParams& p, cudaStream_t s);
cudaError_t launch_page_plan(const PagePlanParams& p, cudaStream_t s);
cudaError_t launch_kv_slots(const KvSlotsParams& p, cudaStream_t s);
bool project_tc(int rows);
size_t project_workspace(int rows, int rank_max);
cudaError_t launch_shrink(const ProjectParams& p, cudaStream_t s);
bool project_is_many(const ProjectParams& p);
cudaError_t launch_project_many(const ProjectParams& p, cudaStream_t s);
cudaError_t launch_project(const ProjectParams& p, void* workspace, cudaStream_t s);

}  // namespace tts
