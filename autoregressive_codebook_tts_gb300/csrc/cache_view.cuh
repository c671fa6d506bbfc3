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
  const int page = __ldcg(c.block_table + static_cast<int64_t>(b) * c.bt_stride + (pos >> c.page_shift));
  return page >= 0 && page < c.n_pages ? page : -1;
}

// Row index of (b, g, pos); `page` from cache_page (ignored when contiguous).
__device__ __forceinline__ int64_t cache_row(const CacheView& c, int b, int g, int pos, int page) {
  if (!c.paged) return (static_cast<int64_t>(b) * c.n_kv_heads + g) * c.capacity + pos;
  return ((static_cast<int64_t>(page) * c.n_kv_heads + g) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

// The largest magnitude of three values: a NaN where one is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Puts fix(x[e], e) as entry e's code into w, for each e whose byte in d is not 0.
template <int N, typename Fix>
__device__ __forceinline__ void each_marked(uint32_t (&d)[N / 4], const float (&x)[N], uint32_t (&w)[N / 4], Fix fix) {
#pragma unroll
  for (int e = 0; e < N; e += 4)
    while (d[e / 4] != 0) {
      const int at = (__ffs(d[e / 4]) - 1) & 24;
      const float y = at < 16 ? (at == 0 ? x[e] : x[e + 1]) : (at == 16 ? x[e + 2] : x[e + 3]);
      w[e / 4] = (w[e / 4] & ~(0xffu << at)) | fix(y, e + (at >> 3)) << at;
      d[e / 4] &= ~(0xffu << at);
    }
}

// Codes of the 8-bit caches: kTop is the largest; codes() the codes nearest to the exact
// quotients x / s of N entries, four to a word.
//
// x * (1 / s) is off x / s by at most two units in the last place (one rounding of 1 / s, one
// of the product).  Codes rise with the quotient: where a product with a value just below 1 / s and one
// with a value just above it have the same code, x / s has it too.  (fast_codes() takes those `steps` last
// places of inv away.  A step is at least 2^-24 of inv, and a rounding on the way to the product at
// most that, so steps is one more than the roundings.)  The other entries are decided by the exact
// remainder x - q s, which one fused multiply-add gives with its right sign; one at a time, for half a
// percent of the entries of a bf16 row are on a border or beside it (none of an f32 row's), which leaves
// most warps with a few; but all of a lane's at once where each of its words has one, as in rows whose
// quotients are ties (16 x 1024 rows of 8 heads of them, bf16 to int8: 39 us, one at a time 59).  (No
// entry is that far below s that the remainder could underflow: tiny rows are scaled up first.)
template <typename Code, int N>
__device__ __forceinline__ bool fast_codes(const float (&x)[N], float inv, int steps, uint32_t (&w)[N / 4], uint32_t (&d)[N / 4]) {
  const float below = __uint_as_float(__float_as_uint(inv) - steps), above = __uint_as_float(__float_as_uint(inv) + steps);
  uint32_t any = 0;
#pragma unroll
  for (int e = 0; e < N / 4; ++e) {
    w[e] = Code::four(x + 4 * e, below);
    d[e] = w[e] ^ Code::four(x + 4 * e, above);
    any |= d[e];
  }
  return any != 0;
}
template <typename Code, int N>
__device__ __forceinline__ void codes(const float (&x)[N], float s, uint32_t (&w)[N / 4]) {
  const bool tiny = s < 1e-27f;
  const float inv = 1.0f / s;
  uint32_t d[N / 4];
  if (fast_codes<Code>(x, inv, 3, w, d) || tiny) {
    const float up = tiny ? 1.152921504606846976e18f : 1.0f;   // 2^60
    const float su = s * up, iu = 1.0f / su;
    bool all = true;
#pragma unroll
    for (int e = 0; e < N / 4; ++e) all = all && d[e] != 0;
    all = all || tiny;
    if (all) {
#pragma unroll
      for (int e = 0; e < N / 4; ++e) {
        w[e] = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) w[e] |= Code::nearest(x[4 * e + k] * up, su, iu) << (8 * k);
      }
    } else {
      each_marked(d, x, w, [&](float y, int) { return Code::nearest(y * up, su, iu); });
    }
  }
}

struct I8Code {
  static constexpr float kTop = 127.f;
  static __device__ __forceinline__ uint32_t nearest(float x, float s, float inv) {
    // (1.5 2^23 + an integer has it in its low bits: no conversions, which are slow)
    const float t = x * inv, r = __fadd_rn(t, 12582912.f), c = __fsub_rn(r, 12582912.f);
    // the border beyond c on the quotient's side: is the quotient past it, or on it?
    const float side = copysignf(1.f, t - c), past = side * fmaf(-(c + 0.5f * side), s, x);
    const float to = past > 0.f || (past == 0.f && (__float_as_uint(r) & 1u) != 0) ? side : 0.f;
    return __float_as_uint(fminf(fmaxf(r + to, 12582785.f), 12583039.f)) & 0xffu;
  }
  // t + 1.5 2^23 has the nearest integer in its low bits
  static __device__ __forceinline__ uint32_t four(const float* x, float inv) {
    const float2 i2 = make_float2(inv, inv), magic = make_float2(12582912.f, 12582912.f);
    const float2 a = __ffma2_rn(make_float2(x[0], x[1]), i2, magic), b = __ffma2_rn(make_float2(x[2], x[3]), i2, magic);
    return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                       __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
  }
  // the values of a word's codes: code + 128 in the low bits of 2^23
  static __device__ __forceinline__ void values(uint32_t w, float (&f)[4]) {
    w ^= 0x80808080u;
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 + k)) - 8388736.f;
  }
  static __device__ __forceinline__ float value(uint32_t code) {
    return static_cast<float>(static_cast<int>(static_cast<int8_t>(code & 0xffu)));
  }
};
struct E4m3Code {
  static constexpr float kTop = 448.f;
  static __device__ __forceinline__ uint32_t nearest(float x, float s, float inv) {
    // the quotient to its last place, then rounded to odd: towards zero, the last bit set
    // when anything is left, so that the rounding to the code meets no border by accident
    float q = x * inv;
    q = fmaf(fmaf(-q, s, x), inv, q);
    const float left = fmaf(-q, s, x);
    // (a quotient that underflows is a zero of its sign already: no last place below it)
    if (left != 0.f && q != 0.f) {
      uint32_t u = __float_as_uint(q);
      if ((left < 0.f) != (q < 0.f)) --u;   // |q| is above the quotient
      q = __uint_as_float(u | 1u);
    }
    return __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
  }
  static __device__ __forceinline__ uint32_t four(const float* x, float inv) {
    const float2 i2 = make_float2(inv, inv);
    const float2 a = __fmul2_rn(make_float2(x[0], x[1]), i2), b = __fmul2_rn(make_float2(x[2], x[3]), i2);
    return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3)) |
           static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3)) << 16;
  }
  static __device__ __forceinline__ void values(uint32_t w, float (&f)[4]) {
    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffffu), __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3);
    const float2 x = __half22float2(__half2(a)), y = __half22float2(__half2(b));
    f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
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
    for (int i = 0; i < 4; ++i) {
      float x[4];
      Code::values(w[i], x);
      f[4 * i] = x[0]; f[4 * i + 1] = x[1]; f[4 * i + 2] = x[2]; f[4 * i + 3] = x[3];
    }
  }
};
template <> struct CacheElem<CodeI8> : CacheElem8<I8Code> {};
template <> struct CacheElem<CodeE4m3> : CacheElem8<E4m3Code> {};

}  // namespace tts
