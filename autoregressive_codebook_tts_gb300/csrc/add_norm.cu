// The residual's addition and the RMS norm of the sum, to f32, bf16 or e4m3 rows with a scale.
//
// A row is read once and held in registers (eight entries a vector): the sum is stored, its mean square
// is reduced by shuffles and through shared memory, and y leaves in the output's type.  Sums and
// statistics are in f32.  Nothing is read twice, so the kernel is bound by HBM on many rows and by the
// launch and one round trip to memory on few.  n 2048: 32 rows 2.7 us; 6001 rows, bf16 throughout 18.2
// (5.4 TB/s), f32 in and bf16 out 27.6 (6.2 TB/s, 0.92 of the measured copy rate), e4m3 out 22.9 (3.8 TB/s; two
// more reductions a row and the codes).
//
// e4m3: the root is common to a row's entries and their largest, so the code of entry i is that
// nearest to 448 h_i g_i / max |h g|, with no rounding of y in between.  Quotients of f32 values decide it
// unless a border lies within their error (an entry in some 10^5, more where gamma and the entries have
// few bits); those are decided one at a time by the products in double, which holds them exactly.  (Taken
// from the rounded y, one code in 10^4 is another.)
#include "cache_view.cuh"
#include "serve_kernels.h"

namespace tts {
namespace {

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
  unpack_bf16x8(__ldcs(reinterpret_cast<const uint4*>(p)), f);
}
__device__ __forceinline__ uint32_t pair(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *(reinterpret_cast<float4*>(p) + 1) = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7]));
}
__device__ __forceinline__ void gamma8(const float* p, float (&g)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  g[0] = a.x; g[1] = a.y; g[2] = a.z; g[3] = a.w; g[4] = b.x; g[5] = b.y; g[6] = b.z; g[7] = b.w;
}
// an f32 value rounded to the residual's type
__device__ __forceinline__ float as_stored(float x, const float*) { return x; }
__device__ __forceinline__ float as_stored(float x, const __nv_bfloat16*) { return __bfloat162float(__float2bfloat16_rn(x)); }

// The code of an entry from its exact product, against the largest of the row.
__device__ __noinline__ uint32_t code_exact(float h, float gamma, double most) {
  return __nv_cvt_double_to_fp8(E4m3Code::kTop * (static_cast<double>(h) * static_cast<double>(gamma)) / most, __NV_SATFINITE,
                                __NV_E4M3);
}

// A block a row, V vectors a thread.  (A warp a row with eight vectors a lane has fewer loads in flight
// an SM for its registers: 6001 rows of 2048, bf16 to bf16 25.2 us against 19.2.)
template <typename X, typename R, typename O, int V>
__global__ void __launch_bounds__(V == 1 ? 512 : 1024) add_norm_kernel(const AddNormParams p) {
  constexpr bool kCodes = sizeof(O) == 1;
  __shared__ float s_sum[32];
  __shared__ uint32_t s_top[32];
  __shared__ int s_rest;   // what the largest product is above its rounded value, as an ordered integer
  grid_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = threadIdx.x, nt = blockDim.x;
  const int64_t row = blockIdx.x;
  const X* x = static_cast<const X*>(p.x) + row * p.x_stride;
  const R* res = static_cast<const R*>(p.res) + row * p.res_stride;
  float h[V][8], g[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int at = (j * nt + t) * 8;
    if (at < p.n) {
      load8(x + at, h[j]);
      float q[8];
      if (p.res != nullptr) load8(res + at, q);
      gamma8(p.gamma + at, g[j]);
      if (p.res != nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[j][e] = as_stored(q[e] + h[j][e], static_cast<const R*>(nullptr));
        if (p.sum != nullptr) store8(static_cast<R*>(p.sum) + row * p.sum_stride + at, h[j]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[j][e] = 0.f;
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(h[j][e], h[j][e], ss);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
  if (lane == 0) s_sum[warp] = ss;
  if (kCodes && t == 0) s_rest = static_cast<int>(0x80000000u);
  __syncthreads();
  ss = lane < nt / 32 ? s_sum[lane] : 0.f;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
  const float r = 1.0f / sqrtf(ss / static_cast<float>(p.n) + p.eps);
  if constexpr (!kCodes) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int at = (j * nt + t) * 8;
      if (at < p.n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[j][e] = h[j][e] * r * g[j][e];
        store8(static_cast<O*>(p.out) + row * p.out_stride + at, h[j]);
      }
    }
  } else {
    // by the power of two below the root (exact), so that the products are as large as y
    const float u = __uint_as_float(__float_as_uint(r) & 0x7f800000u);
    // magnitudes order as their bits do; infinities and NaN are the largest
    float most = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if ((j * nt + t) * 8 < p.n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[j][e] *= u;
#pragma unroll
        for (int e = 0; e < 8; e += 2) most = max_abs(most, h[j][e] * g[j][e], h[j][e + 1] * g[j][e + 1]);
      }
    const uint32_t mine = __float_as_uint(most) & 0x7fffffffu;
    uint32_t top = __reduce_max_sync(kFull, mine);
    if (lane == 0) s_top[warp] = top;
    __syncthreads();
    top = __reduce_max_sync(kFull, lane < nt / 32 ? s_top[lane] : 0u);
    const float largest = __uint_as_float(top), inv = E4m3Code::kTop / largest;
    // (u may be half the root: y can be past f32's range where the products are not)
    const float most_y = largest * (r / u);
    const bool bad = top >= 0x7f800000u || (top != 0 && !(most_y < __uint_as_float(0x7f800000u))), plain = bad || top == 0;   // plain: codes 0
    if (t == 0) p.out_scale[row] = bad ? __uint_as_float(0x7fc00000u) : top == 0 ? 0.f : most_y * (1.0f / E4m3Code::kTop);
    uint32_t w[V][2], d[V][2];
    bool near = false;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      w[j][0] = w[j][1] = d[j][0] = d[j][1] = 0;
      if ((j * nt + t) * 8 < p.n && !plain) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = h[j][e] * g[j][e];
        // (roundings: the product, the largest, its quotient, the quotient of the two)
        near = fast_codes<E4m3Code>(y, inv, 5, w[j], d[j]) || near;
        if (mine == top) {
          // one of the products that round to the largest may be it
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if ((__float_as_uint(y[e]) & 0x7fffffffu) == top) {
              const int rest = __float_as_int(copysignf(1.f, y[e]) * fmaf(h[j][e], g[j][e], -y[e]));
              atomicMax(&s_rest, rest ^ ((rest >> 31) & 0x7fffffff));
            }
        }
      }
    }
    if (__syncthreads_or(near) && near) {
      const int rest = s_rest;
      const double exact = static_cast<double>(largest) + static_cast<double>(__int_as_float(rest ^ ((rest >> 31) & 0x7fffffff)));
#pragma unroll
      for (int j = 0; j < V; ++j)
        each_marked(d[j], h[j], w[j], [&](float x, int e) { return code_exact(x, __ldg(p.gamma + (j * nt + t) * 8 + e), exact); });
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int at = (j * nt + t) * 8;
      if (at < p.n) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + row * p.out_stride + at) = make_uint2(w[j][0], w[j][1]);
    }
  }
}

template <typename X, typename R, typename O>
cudaError_t launch(const AddNormParams& p, cudaStream_t s) {
  const int vecs = p.n / 8, v = vecs <= 512 ? 1 : 2;
  const dim3 grid(p.rows), block(((vecs + v - 1) / v + 31) / 32 * 32);
  return v == 1 ? launch_pdl(add_norm_kernel<X, R, O, 1>, grid, block, 0, s, p)
                : launch_pdl(add_norm_kernel<X, R, O, 2>, grid, block, 0, s, p);
}
template <typename X, typename R>
cudaError_t launch_out(const AddNormParams& p, cudaStream_t s) {
  switch (p.out_dtype) {
    case TTS_F32: return launch<X, R, float>(p, s);
    case TTS_BF16: return launch<X, R, __nv_bfloat16>(p, s);
    default: return launch<X, R, uint8_t>(p, s);
  }
}

}  // namespace

cudaError_t launch_add_norm(const AddNormParams& p, cudaStream_t s) {
  if (p.x_bf16) return p.res_bf16 ? launch_out<__nv_bfloat16, __nv_bfloat16>(p, s) : launch_out<__nv_bfloat16, float>(p, s);
  return p.res_bf16 ? launch_out<float, __nv_bfloat16>(p, s) : launch_out<float, float>(p, s);
}

}  // namespace tts
