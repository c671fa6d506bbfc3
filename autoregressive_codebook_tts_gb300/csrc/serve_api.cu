// C ABI of the calls that serve many requests at once: argument checks on the host, then launches
// on the caller's stream.  Contract in include/tts_decode.h.
#include <cstdint>
#include <cuda_runtime.h>

#include "checks.h"
#include "serve_kernels.h"

using namespace tts;

namespace {

bool is_row_dtype(int dt) { return dt == TTS_F32 || dt == TTS_BF16; }
// elements of 16 bytes
int quantum(int dt) { return dt == TTS_F32 ? 4 : dt == TTS_BF16 ? 8 : 16; }
bool stride_ok(int64_t stride, int dt) { return stride % quantum(dt) == 0; }

tts_status check_project(int32_t rows, int32_t n, int32_t k, int32_t x_dtype, const tts_adapters* ad) {
  if (x_dtype != TTS_BF16 && x_dtype != TTS_E4M3) return TTS_ERR_DTYPE;
  if (rows < 1 || rows > (1 << 20) || n < 1 || n > (1 << 20) || k < 1 || k > 65536) return TTS_ERR_SHAPE;
  if (k % quantum(x_dtype) != 0) return TTS_ERR_ALIGN;
  if (ad != nullptr) {
    if (ad->a == nullptr || ad->b == nullptr) return TTS_ERR_NULL;
    if (ad->n_adapters < 1 || ad->rank_max < 8 || ad->rank_max > TTS_MAX_ADAPTER_RANK || ad->rank_max % 8 != 0)
      return TTS_ERR_SHAPE;
    // tile coordinates into the pool are 32 bits
    if (static_cast<int64_t>(ad->n_adapters) * n >= (int64_t{1} << 31) ||
        static_cast<int64_t>(ad->n_adapters) * ad->rank_max >= (int64_t{1} << 31))
      return TTS_ERR_SHAPE;
    if (!aligned16(ad->a) || !aligned16(ad->b) || !aligned16(ad->rank) || !aligned16(ad->scale)) return TTS_ERR_ALIGN;
  }
  return TTS_OK;
}

}  // namespace

namespace {
// Maps and counts may be slices that begin at any entry.
template <typename T>
bool own_size(const T* p) { return reinterpret_cast<uintptr_t>(p) % sizeof(T) == 0; }
}  // namespace

extern "C" {

tts_status tts_add_rms_norm(const void* x, int64_t x_stride, int32_t x_dtype, const void* residual, int64_t res_stride,
                            int32_t res_dtype, void* sum_out, int64_t sum_stride, const float* gamma, float eps,
                            int32_t rows, int32_t n, void* out, int64_t out_stride, int32_t out_dtype, float* out_scale,
                            void* stream) {
  const bool with_res = residual != nullptr, codes = out_dtype == TTS_E4M3;
  if (x == nullptr || gamma == nullptr || out == nullptr || (codes && out_scale == nullptr)) return TTS_ERR_NULL;
  if (!with_res && sum_out != nullptr) return TTS_ERR_NULL;
  if (!is_row_dtype(x_dtype) || (with_res && !is_row_dtype(res_dtype)) || (!is_row_dtype(out_dtype) && !codes))
    return TTS_ERR_DTYPE;
  if (rows < 1 || rows > (1 << 24) || n < 8 || n > TTS_MAX_NORM_WIDTH || n % 8 != 0 || !(eps >= 0.f) || x_stride < n ||
      out_stride < n || (with_res && res_stride < n) || (sum_out != nullptr && sum_stride < n))
    return TTS_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(sum_out) || !aligned16(gamma) ||
      !(codes ? reinterpret_cast<uintptr_t>(out) % 8 == 0 && out_stride % 8 == 0 : aligned16(out) && stride_ok(out_stride, out_dtype)) ||
      !aligned16(out_scale) || !stride_ok(x_stride, x_dtype) ||
      (with_res && !stride_ok(res_stride, res_dtype)) || (sum_out != nullptr && !stride_ok(sum_stride, res_dtype)))
    return TTS_ERR_ALIGN;
  // in place means the same rows: same type and stride
  if ((out == x && (out_dtype != x_dtype || out_stride != x_stride)) ||
      (with_res && sum_out == residual && sum_stride != res_stride) || out == residual || out == sum_out)
    return TTS_ERR_LAYOUT;
  if (sum_out != nullptr && sum_out == x) return TTS_ERR_LAYOUT;
  AddNormParams p = {};
  p.x = x;
  p.res = residual;
  p.sum = sum_out;
  p.gamma = gamma;
  p.out = out;
  p.out_scale = out_scale;
  p.x_stride = x_stride;
  p.res_stride = res_stride;
  p.sum_stride = sum_stride;
  p.out_stride = out_stride;
  p.eps = eps;
  p.rows = rows;
  p.n = n;
  p.x_bf16 = x_dtype == TTS_BF16;
  p.res_bf16 = with_res && res_dtype == TTS_BF16;
  p.out_dtype = out_dtype;
  return from_cuda(launch_add_norm(p, as_stream(stream)));
}

size_t tts_project_workspace_size(int32_t rows, int32_t n, int32_t k, int32_t x_dtype, const tts_adapters* ad) {
  if (check_project(rows, n, k, x_dtype, ad) != TTS_OK || ad == nullptr) return 0;
  return project_workspace(rows, ad->rank_max);
}

tts_status tts_project_rows(const void* x, int64_t x_stride, int32_t x_dtype, const float* x_scale, const void* w,
                            const float* w_scale, int32_t n, int32_t k, const tts_adapters* ad, const int32_t* row_stream,
                            const int32_t* stream_adapter, int32_t n_streams, int32_t rows, void* out, int64_t out_stride,
                            int32_t out_dtype, void* workspace, size_t ws_bytes, int32_t* err_flag, void* stream) {
  const bool e4m3 = x_dtype == TTS_E4M3;
  if (x == nullptr || w == nullptr || out == nullptr || (e4m3 && (x_scale == nullptr || w_scale == nullptr)) ||
      (ad != nullptr && stream_adapter == nullptr))
    return TTS_ERR_NULL;
  const tts_status st = check_project(rows, n, k, x_dtype, ad);
  if (st != TTS_OK) return st;
  if (!is_row_dtype(out_dtype)) return TTS_ERR_DTYPE;
  if (x_stride < k || out_stride < n || (ad != nullptr && n_streams < 1)) return TTS_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(w) || !aligned16(out) || !aligned16(x_scale) || !aligned16(w_scale) ||
      !own_size(row_stream) || !own_size(stream_adapter) || !stride_ok(x_stride, x_dtype))
    return TTS_ERR_ALIGN;
  ProjectParams p = {};
  if (ad != nullptr) {
    if (workspace == nullptr || ws_bytes < tts_project_workspace_size(rows, n, k, x_dtype, ad)) return TTS_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return TTS_ERR_ALIGN;
    p.ad = *ad;
  }
  // an input row is read by many CTAs, some after others have written out
  if (out == x || out == w) return TTS_ERR_LAYOUT;
  p.x = x;
  p.x_stride = x_stride;
  p.x_e4m3 = e4m3;
  p.x_scale = x_scale;
  p.w = w;
  p.w_scale = w_scale;
  p.n = n;
  p.k = k;
  p.rows = rows;
  p.row_stream = row_stream;
  p.stream_adapter = stream_adapter;
  p.n_streams = n_streams;
  p.out = out;
  p.out_stride = out_stride;
  p.out_bf16 = out_dtype == TTS_BF16;
  p.err = err_flag;
  return from_cuda(launch_project(p, workspace, as_stream(stream)));
}

tts_status tts_page_plan(const tts_kv_desc* d, int32_t* block_table, int32_t* free_pages, int32_t* n_free,
                         const int32_t* n_past, const int32_t* n_new, int32_t T, int32_t max_rows, int32_t* n_rows,
                         int32_t* row_start, int32_t* row_stream, int32_t* row_pos, int64_t* row_slot, int32_t* err_flag,
                         void* stream) {
  const tts_status st = check_desc(d, true);
  if (st != TTS_OK) return st;
  if (!d->paged || block_table != d->block_table) return TTS_ERR_LAYOUT;
  if (free_pages == nullptr || n_free == nullptr || n_past == nullptr || n_new == nullptr || n_rows == nullptr ||
      row_start == nullptr || row_stream == nullptr || row_pos == nullptr || row_slot == nullptr)
    return TTS_ERR_NULL;
  // (sums of pages are held in 32 bits)
  if (d->B > TTS_MAX_PLAN_STREAMS || d->n_pages > (1 << 30) || T < 0 || max_rows < 1 || max_rows > (1 << 24) ||
      (T > 0 && static_cast<int64_t>(d->B) * T != max_rows))
    return TTS_ERR_SHAPE;
  if (!own_size(block_table) || !own_size(free_pages) || !own_size(n_free) || !own_size(n_past) || !own_size(n_new) ||
      !own_size(n_rows) || !own_size(row_start) || !own_size(row_stream) || !own_size(row_pos) || !own_size(row_slot))
    return TTS_ERR_ALIGN;
  PagePlanParams p = {};
  p.table = block_table;
  p.B = d->B;
  p.capacity = d->capacity;
  p.page_shift = log2i(d->page_size);
  p.n_pages = d->n_pages;
  p.bt_stride = d->bt_stride;
  p.free_pages = free_pages;
  p.n_free = n_free;
  p.n_past = n_past;
  p.n_new = n_new;
  p.T = T;
  p.max_rows = max_rows;
  p.n_rows = n_rows;
  p.row_start = row_start;
  p.row_stream = row_stream;
  p.row_pos = row_pos;
  p.row_slot = row_slot;
  p.err = err_flag;
  return from_cuda(launch_page_plan(p, as_stream(stream)));
}

tts_status tts_kv_write_slots(const void* k, const void* v, int32_t dtype, int64_t row_stride, const tts_kv_cache* c,
                              const tts_kv_desc* d, const int64_t* row_slot, int32_t rows, int32_t* err_flag,
                              void* stream) {
  const tts_status st = check_desc(d, true);
  if (st != TTS_OK) return st;
  const bool scaled = d->kv_dtype == TTS_I8 || d->kv_dtype == TTS_E4M3;
  if (c == nullptr || c->k == nullptr || c->v == nullptr || (scaled && (c->k_scale == nullptr || c->v_scale == nullptr)) ||
      k == nullptr || v == nullptr || row_slot == nullptr)
    return TTS_ERR_NULL;
  if (!is_row_dtype(dtype)) return TTS_ERR_DTYPE;
  if (rows < 1 || rows > (1 << 24) || d->n_kv_heads > 65535 || static_cast<int64_t>(rows) * d->n_kv_heads >= (int64_t{1} << 31) ||
      row_stride < static_cast<int64_t>(d->n_kv_heads) * d->head_dim)
    return TTS_ERR_SHAPE;
  if (!aligned16(c->k) || !aligned16(c->v) || (scaled && (!aligned16(c->k_scale) || !aligned16(c->v_scale))) ||
      !aligned16(k) || !aligned16(v) || !own_size(row_slot) || !stride_ok(row_stride, dtype))
    return TTS_ERR_ALIGN;
  KvSlotsParams p = {};
  p.k = k;
  p.v = v;
  p.row_stride = row_stride;
  p.row_bf16 = dtype == TTS_BF16;
  p.cache.k = c->k;
  p.cache.v = c->v;
  p.cache.k_scale = scaled ? c->k_scale : nullptr;
  p.cache.v_scale = scaled ? c->v_scale : nullptr;
  p.cache.n_kv_heads = d->n_kv_heads;
  p.cache.paged = d->paged;
  p.cache.page_shift = d->paged ? log2i(d->page_size) : 0;
  p.page_rows = d->paged ? d->page_size : d->capacity;
  p.n_slots = p.page_rows * (d->paged ? d->n_pages : d->B);
  p.kv_dtype = d->kv_dtype;
  p.head_dim = d->head_dim;
  p.slot = row_slot;
  p.rows = rows;
  p.err = err_flag;
  return from_cuda(launch_kv_slots(p, as_stream(stream)));
}

}  // extern "C"
