// C ABI of drafted decoding over a quantised cache: argument checks on the host, then
// launches on the caller's stream.  Contract in include/tts_decode.h.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "checks.h"
#include "draft_kernels.h"

using namespace tts;

namespace {

bool row_dtype_ok(int dt) { return dt == TTS_F32 || dt == TTS_BF16; }
// elements of 16 bytes
int row_quantum(int dt) { return dt == TTS_BF16 ? 8 : 4; }

tts_status check_cache(const tts_kv_cache* c, const tts_kv_desc* d, CacheView& v) {
  const tts_status st = check_desc(d, true);
  if (st != TTS_OK) return st;
  if (c == nullptr || c->k == nullptr || c->v == nullptr) return TTS_ERR_NULL;
  const bool scaled = d->kv_dtype == TTS_I8 || d->kv_dtype == TTS_E4M3;
  if (scaled && (c->k_scale == nullptr || c->v_scale == nullptr)) return TTS_ERR_NULL;
  if (!aligned16(c->k) || !aligned16(c->v) || (scaled && (!aligned16(c->k_scale) || !aligned16(c->v_scale))))
    return TTS_ERR_ALIGN;
  if (d->B > 65535 || d->n_kv_heads > 65535) return TTS_ERR_SHAPE;
  v.k = c->k;
  v.v = c->v;
  v.k_scale = scaled ? c->k_scale : nullptr;
  v.v_scale = scaled ? c->v_scale : nullptr;
  v.B = d->B;
  v.n_kv_heads = d->n_kv_heads;
  v.capacity = d->capacity;
  v.paged = d->paged;
  v.page_shift = d->paged ? log2i(d->page_size) : 0;
  v.n_pages = d->paged ? d->n_pages : 0;
  v.bt_stride = d->paged ? d->bt_stride : 0;
  v.block_table = d->paged ? d->block_table : nullptr;
  return TTS_OK;
}

tts_status check_rows(const tts_kv_desc* d, int32_t dtype, int64_t stride, int32_t T) {
  if (!row_dtype_ok(dtype)) return TTS_ERR_DTYPE;
  if (T < 1 || static_cast<int64_t>(d->B) * T > (int64_t{1} << 24) ||
      static_cast<int64_t>(T) * d->n_kv_heads >= (int64_t{1} << 31) - (1 << 16) ||
      stride < static_cast<int64_t>(d->n_kv_heads) * d->head_dim)
    return TTS_ERR_SHAPE;
  return stride % row_quantum(dtype) == 0 ? TTS_OK : TTS_ERR_ALIGN;
}

// The launch of a tree attention: row blocks, tiles and CTAs from shapes alone.
struct TreePlan {
  bool tc;              // tensor cores
  int rows, n_rb, tile, n_cta, whole, fixed;
  size_t part, total;   // bytes of the partial rows, and of the whole workspace
};
TreePlan tree_plan(const tts_kv_desc* d, int T, int q_dtype) {
  TreePlan t = {};
  const int rows = T * (d->n_q_heads / d->n_kv_heads);
  // f32 operands would lose bits on the tensor cores
  t.tc = q_dtype == TTS_BF16 && tree_attn_tc_supported(d);
  t.rows = t.tc ? (rows <= 32 ? 32 : rows <= 64 ? 64 : 128) : (rows <= 8 ? 8 : rows <= 16 ? 16 : 32);
  t.n_rb = (rows + t.rows - 1) / t.rows;
  t.tile = t.tc ? 128 : 64;
  const int64_t items = static_cast<int64_t>(d->B) * d->n_kv_heads * t.n_rb;
  // Short windows are one CTA's each: the combine launch costs more than cutting them saves.  (Five
  // nodes, one / eight streams, whole against cut.  Tensor cores, bf16: 250 rows 7.1 / 7.6 against
  // 12.2 / 13.5 us, 500 rows 9.2 / 9.8 against 12.4 / 14.9, about 1.1 us a tile more.  CUDA cores,
  // f32: 120 rows 12.9 / 13.0 against 12.4 / 15.6 us, 250 rows 22.8 / 23.0 against 14.5 / 23.3.)
  t.whole = d->capacity <= (t.tc ? 6 : 2) * t.tile;
  // An item's query rows, epilogue and partials in units of a quarter tile: two tiles' time, four
  // with 128 query rows on the tensor cores.  (32 streams, 63 nodes, e4m3: 8 146 us, 14 141 us, 18
  // and 20 138 us; one node, int8: 8 38.3 us, 14 39.8 us, 20 41.0 us; f32, 8 streams of 16 nodes: 8
  // 126 us, 14 137 us; 16 nodes gain 1 % with 14: int8 77.4 against 76.7 us, bf16 pages 32.5 against 32.2.)
  t.fixed = t.tc && t.rows == 128 ? 18 : 8;
  t.n_cta = t.whole ? static_cast<int>(items) : (t.tc ? 1 : 2) * sm_count();
  if (!t.whole) {
    const size_t slots = static_cast<size_t>(t.n_cta) * 2 * t.rows;
    t.part = round256(slots * d->head_dim * sizeof(float));
    t.total = t.part + round256(slots * sizeof(float2));
  }
  return t;
}

bool tree_shape_ok(const tts_kv_desc* d, int32_t T) {
  // (the work's units, at most 8 (12 + capacity / 16) or 2 (22 + capacity / 32) a stream and kv
  // head, are counted in 32 bits)
  return T >= 1 && T <= TTS_MAX_TREE_NODES && d->B <= 65535 && d->n_kv_heads <= 65535 &&
         static_cast<int64_t>(d->B) * d->n_kv_heads * (static_cast<int64_t>(d->capacity) + 192) < (int64_t{1} << 31);
}

}  // namespace

extern "C" {

tts_status tts_rope_table_scaled(float* cs, int32_t max_pos, int32_t rot_dim, double base, const tts_rope_scaling* s,
                                 void* stream) {
  if (cs == nullptr || s == nullptr) return TTS_ERR_NULL;
  if (s->kind < TTS_ROPE_NONE || s->kind > TTS_ROPE_PARTS) return TTS_ERR_DTYPE;
  // (a grid holds 65535 blocks of 1024 positions)
  if (max_pos < 1 || max_pos > 65535 * 1024 || rot_dim < 2 || rot_dim > 128 || rot_dim % 2 != 0 || !(base > 1.0) ||
      !std::isfinite(base) || !(s->attn_scale > 0.0) || !std::isfinite(s->attn_scale))
    return TTS_ERR_SHAPE;
  if (s->kind != TTS_ROPE_NONE && (!(s->factor >= 1.0) || !std::isfinite(s->factor))) return TTS_ERR_SHAPE;
  if (s->kind == TTS_ROPE_BASE && rot_dim < 4) return TTS_ERR_SHAPE;
  if (s->kind == TTS_ROPE_PARTS &&
      (s->original_max_pos < 1 || !(s->low_rotations >= 0.0) || !(s->high_rotations > s->low_rotations) ||
       !std::isfinite(s->high_rotations)))
    return TTS_ERR_SHAPE;
  if (!aligned16(cs)) return TTS_ERR_ALIGN;
  const RopeTableParams p = {reinterpret_cast<float2*>(cs), max_pos, rot_dim, base, *s};
  return from_cuda(launch_rope_table_scaled(p, as_stream(stream)));
}

tts_status tts_rope_rows(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int32_t dtype, void* q_out,
                         int64_t q_out_stride, void* k_out, int64_t k_out_stride, int32_t out_dtype,
                         const float* gamma_q, const float* gamma_k, float eps, const int32_t* pos, int32_t rows,
                         int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, int32_t rot_dim, int32_t interleaved,
                         const float* rope_cs, int32_t rope_max_pos, int32_t* err_flag, void* stream) {
  const bool with_k = n_kv_heads > 0;
  if (q == nullptr || q_out == nullptr || pos == nullptr || rope_cs == nullptr ||
      (with_k && (k == nullptr || k_out == nullptr)) || (gamma_q == nullptr && gamma_k != nullptr) ||
      (with_k && gamma_q != nullptr && gamma_k == nullptr))
    return TTS_ERR_NULL;
  if (!row_dtype_ok(dtype) || !row_dtype_ok(out_dtype)) return TTS_ERR_DTYPE;
  if (rows < 1 || rows > (1 << 24) || !head_dim_ok(head_dim) || n_q_heads < 1 || n_q_heads > 65535 || n_kv_heads < 0 ||
      n_kv_heads > 65535 || rot_dim < 2 || rot_dim > head_dim || rot_dim % 2 != 0 || rope_max_pos < 1 || !(eps >= 0.f) ||
      (interleaved != 0 && interleaved != 1))
    return TTS_ERR_SHAPE;
  const int64_t qd = static_cast<int64_t>(n_q_heads) * head_dim, kd = static_cast<int64_t>(n_kv_heads) * head_dim;
  if (q_stride < qd || q_out_stride < qd || (with_k && (k_stride < kd || k_out_stride < kd))) return TTS_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(q_out) || !aligned16(gamma_q) || !aligned16(gamma_k) || !aligned16(rope_cs) ||
      q_stride % row_quantum(dtype) != 0 || q_out_stride % row_quantum(out_dtype) != 0 ||
      (with_k && (!aligned16(k) || !aligned16(k_out) || k_stride % row_quantum(dtype) != 0 ||
                  k_out_stride % row_quantum(out_dtype) != 0)))
    return TTS_ERR_ALIGN;
  // in place means the same rows: same type and stride
  if ((q == q_out && (dtype != out_dtype || q_stride != q_out_stride)) ||
      (with_k && k == k_out && (dtype != out_dtype || k_stride != k_out_stride)))
    return TTS_ERR_LAYOUT;
  RopeRowsParams p = {};
  p.q = q;
  p.k = k;
  p.q_out = q_out;
  p.k_out = k_out;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.q_out_stride = q_out_stride;
  p.k_out_stride = k_out_stride;
  p.in_bf16 = dtype == TTS_BF16;
  p.out_bf16 = out_dtype == TTS_BF16;
  p.gamma_q = gamma_q;
  p.gamma_k = gamma_k;
  p.eps = eps;
  p.pos = pos;
  p.rows = rows;
  p.n_q_heads = n_q_heads;
  p.n_kv_heads = n_kv_heads;
  p.head_dim = head_dim;
  p.rot_dim = rot_dim;
  p.interleaved = interleaved;
  p.cs = reinterpret_cast<const float2*>(rope_cs);
  p.max_pos = rope_max_pos;
  p.n_sm = sm_count();
  p.err = err_flag;
  return from_cuda(launch_rope_rows(p, as_stream(stream)));
}

tts_status tts_kv_write_rows(const void* k, const void* v, int32_t dtype, int64_t row_stride, const tts_kv_cache* cache,
                             const tts_kv_desc* d, const int32_t* start_pos, const int32_t* n_rows, int32_t T,
                             int32_t* err_flag, void* stream) {
  KvRowsParams p = {};
  tts_status st = check_cache(cache, d, p.cache);
  if (st != TTS_OK) return st;
  if (k == nullptr || v == nullptr || start_pos == nullptr) return TTS_ERR_NULL;
  st = check_rows(d, dtype, row_stride, T);
  if (st != TTS_OK) return st;
  if (!aligned16(k) || !aligned16(v)) return TTS_ERR_ALIGN;
  p.k = k;
  p.v = v;
  p.row_stride = row_stride;
  p.row_bf16 = dtype == TTS_BF16;
  p.kv_dtype = d->kv_dtype;
  p.head_dim = d->head_dim;
  p.start = start_pos;
  p.n_rows = n_rows;
  p.T = T;
  p.n_sm = sm_count();
  p.err = err_flag;
  return from_cuda(launch_kv_write(p, as_stream(stream)));
}

tts_status tts_kv_read_rows(const tts_kv_cache* cache, const tts_kv_desc* d, const int32_t* start_pos,
                            const int32_t* n_rows, int32_t T, void* k_out, void* v_out, int32_t out_dtype,
                            int64_t row_stride, int32_t* err_flag, void* stream) {
  KvRowsParams p = {};
  tts_status st = check_cache(cache, d, p.cache);
  if (st != TTS_OK) return st;
  if (k_out == nullptr || v_out == nullptr || start_pos == nullptr) return TTS_ERR_NULL;
  st = check_rows(d, out_dtype, row_stride, T);
  if (st != TTS_OK) return st;
  if (!aligned16(k_out) || !aligned16(v_out)) return TTS_ERR_ALIGN;
  p.k_out = k_out;
  p.v_out = v_out;
  p.row_stride = row_stride;
  p.row_bf16 = out_dtype == TTS_BF16;
  p.kv_dtype = d->kv_dtype;
  p.head_dim = d->head_dim;
  p.start = start_pos;
  p.n_rows = n_rows;
  p.T = T;
  p.n_sm = sm_count();
  p.err = err_flag;
  return from_cuda(launch_kv_read(p, as_stream(stream)));
}

size_t tts_tree_attn_workspace_size(const tts_kv_desc* d, int32_t T, int32_t q_dtype) {
  if (check_desc(d, true) != TTS_OK || !row_dtype_ok(q_dtype) || !tree_shape_ok(d, T)) return 0;
  return tree_plan(d, T, q_dtype).total;
}

tts_status tts_tree_attn(const void* q, int32_t q_dtype, int64_t q_stride, const tts_kv_cache* cache,
                         const tts_kv_desc* d, const int32_t* n_past, const int32_t* n_nodes, const uint64_t* tree_mask,
                         int32_t T, float scale, void* out, void* workspace, size_t ws_bytes, int32_t* err_flag,
                         void* stream) {
  TreeParams p = {};
  const tts_status st = check_cache(cache, d, p.cache);
  if (st != TTS_OK) return st;
  if (q == nullptr || n_past == nullptr || out == nullptr) return TTS_ERR_NULL;
  if (!row_dtype_ok(q_dtype)) return TTS_ERR_DTYPE;
  if (!tree_shape_ok(d, T) || q_stride < static_cast<int64_t>(d->n_q_heads) * d->head_dim || !std::isfinite(scale * 1.4426950408889634f))
    return TTS_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(out) || !aligned16(tree_mask) || q_stride % row_quantum(q_dtype) != 0)
    return TTS_ERR_ALIGN;
  const TreePlan t = tree_plan(d, T, q_dtype);
  if (t.total > 0) {
    if (workspace == nullptr || ws_bytes < t.total) return TTS_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return TTS_ERR_ALIGN;
    p.part = static_cast<float*>(workspace);
    p.ml = reinterpret_cast<float2*>(static_cast<unsigned char*>(workspace) + t.part);
  }
  // a row of q is read by every CTA of its item, some after another has written out
  if (q == out) return TTS_ERR_LAYOUT;
  p.q = q;
  p.q_stride = q_stride;
  p.q_bf16 = q_dtype == TTS_BF16;
  p.n_past = n_past;
  p.n_nodes = n_nodes;
  p.mask = tree_mask;
  p.T = T;
  p.group = d->n_q_heads / d->n_kv_heads;
  p.n_q_heads = d->n_q_heads;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = out;
  p.n_rb = t.n_rb;
  p.rows = t.rows;
  p.tile = t.tile;
  p.n_cta = t.n_cta;
  p.fixed = t.fixed;
  p.whole = t.whole;
  p.err = err_flag;
  const cudaError_t e = t.tc ? launch_tree_attn_tc(p, d->kv_dtype, d->head_dim, as_stream(stream))
                             : launch_tree_attn(p, d->kv_dtype, d->head_dim, as_stream(stream));
  if (e != cudaSuccess || p.whole) return from_cuda(e);
  return from_cuda(launch_tree_combine(p, d->head_dim, as_stream(stream)));
}

tts_status tts_tree_commit(const tts_kv_cache* cache, const tts_kv_desc* d, const int32_t* n_past, const int32_t* path,
                           int64_t path_stride, const int32_t* n_accept, int32_t T, int32_t* err_flag, void* stream) {
  CommitParams p = {};
  const tts_status st = check_cache(cache, d, p.cache);
  if (st != TTS_OK) return st;
  if (n_past == nullptr || path == nullptr || n_accept == nullptr) return TTS_ERR_NULL;
  if (T < 1 || T > TTS_MAX_TREE_NODES || path_stride < T) return TTS_ERR_SHAPE;
  p.row_bytes = d->head_dim * (d->kv_dtype == TTS_F32 ? 4 : d->kv_dtype == TTS_BF16 ? 2 : 1);
  p.n_past = n_past;
  p.path = path;
  p.path_stride = path_stride;
  p.n_accept = n_accept;
  p.T = T;
  p.err = err_flag;
  return from_cuda(launch_commit(p, as_stream(stream)));
}

}  // extern "C"
