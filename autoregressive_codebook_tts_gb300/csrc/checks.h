// Host-side checks shared by the entry points: alignment, the cache descriptor, the
// device's SM count.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/tts_decode.h"

namespace tts {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool is_pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }
inline int log2i(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}
inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }
inline tts_status from_cuda(cudaError_t e) { return e == cudaSuccess ? TTS_OK : TTS_ERR_CUDA; }

inline bool head_dim_ok(int d) { return d == 64 || d == 128; }
inline bool group_ok(int hq, int hkv) {
  if (hq <= 0 || hkv <= 0 || hq % hkv != 0) return false;
  const int g = hq / hkv;
  return g == 1 || g == 2 || g == 4;
}

inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 152;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();  // clear the sticky-free error this query may leave
    return 152;
  }
  return n;
}

// f32 and bf16 caches; with_8bit admits the quantised dtypes too.
inline tts_status check_desc(const tts_kv_desc* d, bool with_8bit = false) {
  if (d == nullptr) return TTS_ERR_NULL;
  if (d->B < 1 || d->capacity < 1 || !head_dim_ok(d->head_dim) || !group_ok(d->n_q_heads, d->n_kv_heads))
    return TTS_ERR_SHAPE;
  if (d->window_quantum < 1 || d->capacity % d->window_quantum != 0) return TTS_ERR_SHAPE;
  if (d->kv_dtype != TTS_F32 && d->kv_dtype != TTS_BF16 &&
      !(with_8bit && (d->kv_dtype == TTS_I8 || d->kv_dtype == TTS_E4M3)))
    return TTS_ERR_DTYPE;
  if (d->paged != 0 && d->paged != 1) return TTS_ERR_LAYOUT;
  if (d->paged) {
    if (d->block_table == nullptr) return TTS_ERR_NULL;
    if (!is_pow2(d->page_size) || d->page_size > 256 || d->capacity % d->page_size != 0 ||
        d->n_pages < 1 || d->bt_stride < d->capacity / d->page_size)
      return TTS_ERR_LAYOUT;
  }
  return TTS_OK;
}

inline size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace tts
