// The caches of the drafted-decoding calls as the kernels see them: a cache row (position
// and kv head of a stream) is an index into K, V and, for 8-bit caches, the scales.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/tts_decode.h"
#include "common.cuh"

namespace tts {

struct CacheView {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int B, n_kv_heads, capacity;
  int paged, page_shift, n_pages, bt_stride;
  const int32_t* block_table;
};

// The page of position pos of stream b (paged caches); negative when it is out of range.
__device__ __forceinline__ int cache_page(const CacheView& c, int b, int pos) {
  const int page = __ldg(c.block_table + static_cast<int64_t>(b) * c.bt_stride + (pos >> c.page_shift));
  return page >= 0 && page < c.n_pages ? page : -1;
}

// Row index of (b, g, pos); `page` from cache_page (ignored when contiguous).
__device__ __forceinline__ int64_t cache_row(const CacheView& c, int b, int g, int pos, int page) {
  if (!c.paged) return (static_cast<int64_t>(b) * c.n_kv_heads + g) * c.capacity + pos;
  return ((static_cast<int64_t>(page) * c.n_kv_heads + g) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

// Codes of the 8-bit caches: kTop is the largest, code() the code nearest to x / s.
//
// x * (1 / s) is off x / s by at most two units in the last place (one rounding of 1 / s, one
// of the product), so it decides the code unless it lies that close to a border between two
// codes; then (about one value in 10^4) the quotient is taken in double.  There it cannot
// land on a border that the exact quotient misses: x - border * s is a multiple of the
// smaller last place of x and of s / 2, so a nonzero one is at least 2^-33 of x.
struct I8Code {
  static constexpr float kTop = 127.f;
  static __device__ __forceinline__ uint32_t code(float x, float s, float inv) {
    const float t = x * inv;
    float c = rintf(t);
    if (!(fabsf(t - c) < 0.49995f) || !(fabsf(t) < 200.f)) {
      const double e = rint(static_cast<double>(x) / static_cast<double>(s));
      c = static_cast<float>(fmin(fmax(e, -127.0), 127.0));
    }
    return static_cast<uint32_t>(static_cast<int>(c)) & 0xffu;
  }
  static __device__ __forceinline__ float value(uint32_t code) {
    return static_cast<float>(static_cast<int>(static_cast<int8_t>(code & 0xffu)));
  }
};
struct E4m3Code {
  static constexpr float kTop = 448.f;
  static __device__ __forceinline__ uint32_t code(float x, float s, float inv) {
    float t = x * inv;
    // 20 mantissa bits are dropped from a normal code; a border has them at 0x80000
    const uint32_t low = (__float_as_uint(t) & 0xfffffu) - 0x80000u + 8u;
    const float a = fabsf(t);
    // (below 2^-6 the codes are 2^-9 apart, below 2^-10 all is 0)
    if (low <= 16u || (a < 0.015625f && a > 0.0009f) || !(a < 460.f)) {
      // rounded to odd on the way to f32: no border between codes is crossed or reached
      const double e = static_cast<double>(x) / static_cast<double>(s);
      t = __double2float_rz(e);
      if (static_cast<double>(t) != e) t = __uint_as_float(__float_as_uint(t) | 1u);
    }
    return __nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
  }
  static __device__ __forceinline__ float value(uint32_t code) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code & 0xffu), __NV_E4M3);
    return __half2float(__half(h));
  }
};

// Cache element types: bytes, and the values of a 16-byte vector of them (unscaled).
struct CodeI8 { uint8_t x; };
struct CodeE4m3 { uint8_t x; };

template <typename KvT> struct CacheElem;
template <> struct CacheElem<float> {
  static constexpr int kBytes = 4, kVec = 4;
  static constexpr bool kScaled = false;
  static __device__ __forceinline__ void values(const uint4 v, float (&f)[4]) { unpack_f32x4(v, f); }
};
template <> struct CacheElem<__nv_bfloat16> {
  static constexpr int kBytes = 2, kVec = 8;
  static constexpr bool kScaled = false;
  static __device__ __forceinline__ void values(const uint4 v, float (&f)[8]) { unpack_bf16x8(v, f); }
};
template <typename Code> struct CacheElem8 {
  static constexpr int kBytes = 1, kVec = 16;
  static constexpr bool kScaled = true;
  static __device__ __forceinline__ void values(const uint4 v, float (&f)[16]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = Code::value(w[i >> 2] >> (8 * (i & 3)));
  }
};
template <> struct CacheElem<CodeI8> : CacheElem8<I8Code> {};
template <> struct CacheElem<CodeE4m3> : CacheElem8<E4m3Code> {};

}  // namespace tts
