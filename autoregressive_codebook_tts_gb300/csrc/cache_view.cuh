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

// Codes of the 8-bit caches: kTop is the largest; codes() the codes nearest to the exact
// quotients x / s of N entries, four to a word.
//
// x * (1 / s) is off x / s by at most two units in the last place (one rounding of 1 / s, one
// of the product), so it decides the code unless it lies that close to a border between two
// codes.  If any of a lane's entries does (about one in 10^4), all of them are decided by the
// exact remainder x - q s, which one fused multiply-add gives with its right sign.  (No entry
// is that far below s that the remainder could underflow: tiny rows are scaled up first.)
template <typename Code, int N>
__device__ __forceinline__ void codes(const float (&x)[N], float s, uint32_t (&w)[N / 4]) {
  const bool tiny = s < 1e-27f;
  const float inv = 1.0f / s;
  if (Code::fast(x, inv, w) || tiny) {
    const float up = tiny ? 1.152921504606846976e18f : 1.0f;   // 2^60
    const float su = s * up, iu = 1.0f / su;
#pragma unroll
    for (int e = 0; e < N / 4; ++e) {
      w[e] = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) w[e] |= Code::nearest(x[4 * e + k] * up, su, iu) << (8 * k);
    }
  }
}

struct I8Code {
  static constexpr float kTop = 127.f;
  static __device__ __forceinline__ uint32_t nearest(float x, float s, float inv) {
    const float t = x * inv;
    float c = rintf(t);
    // the border beyond c on the quotient's side: is the quotient past it, or on it?
    const float side = copysignf(1.f, t - c), past = side * fmaf(-(c + 0.5f * side), s, x);
    if (past > 0.f || (past == 0.f && (static_cast<int>(c) & 1) != 0)) c += side;
    return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(c, -127.f), 127.f))) & 0xffu;
  }
  // t + 1.5 2^23 has the nearest integer in its low bits; whether one of the quotients is near
  // a border
  template <int N>
  static __device__ __forceinline__ bool fast(const float (&x)[N], float inv, uint32_t (&w)[N / 4]) {
    float off = 0.f;
    const float2 i2 = make_float2(inv, inv), magic = make_float2(12582912.f, 12582912.f),
                 back = make_float2(-12582912.f, -12582912.f), one = make_float2(-1.f, -1.f);
#pragma unroll
    for (int e = 0; e < N; e += 4) {
      uint32_t b[4];
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        const float2 t = __fmul2_rn(make_float2(x[e + k], x[e + k + 1]), i2), r = __fadd2_rn(t, magic);
        const float2 d = __ffma2_rn(__fadd2_rn(r, back), one, t);
        off = fmaxf(off, fmaxf(fabsf(d.x), fabsf(d.y)));
        b[k] = __float_as_uint(r.x);
        b[k + 1] = __float_as_uint(r.y);
      }
      w[e / 4] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    }
    return !(off < 0.49995f);
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
  template <int N>
  static __device__ __forceinline__ bool fast(const float (&x)[N], float inv, uint32_t (&w)[N / 4]) {
    // 20 mantissa bits are dropped from a normal code; a border has them at 0x80000.  Below
    // 2^-6 the codes are 2^-9 apart: taken in double down to where all is 0.
    uint32_t border = ~0u, small = ~0u;
#pragma unroll
    for (int e = 0; e < N; e += 4) {
      float t[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        t[k] = __fmul_rn(x[e + k], inv);
        const uint32_t u = __float_as_uint(t[k]);
        border = min(border, (u & 0xfffffu) - 0x7fff8u);
        small = min(small, (u & 0x7fffffffu) - 0x3a6bedfau);   // 0.0009
      }
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(t[0], t[1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(t[2], t[3]), __NV_SATFINITE, __NV_E4M3);
      w[e / 4] = lo | (hi << 16);
    }
    return border <= 16u || small < 0x3c800000u - 0x3a6bedfau;   // 2^-6
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
