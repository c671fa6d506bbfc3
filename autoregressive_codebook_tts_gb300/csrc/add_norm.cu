// The residual's addition and the RMS norm of the sum, to f32, bf16 or e4m3 rows with a scale.
//
// A row is read once and held in registers (eight entries a vector): the sum is stored, its mean
// square is reduced by shuffles (and through shared memory where a row has several warps), and y
// leaves in the output's type; for e4m3 the row's largest |y| is reduced in the same way.  Sums and
// statistics are in f32.  Nothing is read twice, so the kernel is bound by HBM on many rows and by
// the launch and one round trip to memory on few.
#include "cache_view.cuh"
#include "serve_kernels.h"

namespace tts {
namespace {

constexpr int kRowsPerBlock = 4;   // where a warp has a row of its own

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
// an f32 value rounded to the residual's type
__device__ __forceinline__ float as_stored(float x, const float*) { return x; }
__device__ __forceinline__ float as_stored(float x, const __nv_bfloat16*) { return __bfloat162float(__float2bfloat16_rn(x)); }

// V vectors a thread.  WARP: a warp has a row of its own, else a block has.
template <typename X, typename R, typename O, int V, bool WARP>
__global__ void __launch_bounds__(WARP ? kRowsPerBlock * 32 : (V == 1 ? 512 : 1024)) add_norm_kernel(const AddNormParams p) {
  constexpr bool kCodes = sizeof(O) == 1;
  __shared__ float s_sum[32];
  __shared__ uint32_t s_top[32];
  grid_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = WARP ? lane : static_cast<int>(threadIdx.x), nt = WARP ? 32 : static_cast<int>(blockDim.x);
  const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + warp : blockIdx.x;
  if (row >= p.rows) return;   // (a whole warp; no block barrier follows for WARP)
  const X* x = static_cast<const X*>(p.x) + row * p.x_stride;
  const R* res = static_cast<const R*>(p.res) + row * p.res_stride;
  float h[V][8];
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int at = (j * nt + t) * 8;
    if (at < p.n) load8(x + at, h[j]);
    else
#pragma unroll
      for (int e = 0; e < 8; ++e) h[j][e] = 0.f;
  }
  if (p.res != nullptr) {
    float q[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int at = (j * nt + t) * 8;
      if (at < p.n) load8(res + at, q[j]);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int at = (j * nt + t) * 8;
      if (at < p.n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[j][e] = as_stored(q[j][e] + h[j][e], static_cast<const R*>(nullptr));
        if (p.sum != nullptr) store8(static_cast<R*>(p.sum) + row * p.sum_stride + at, h[j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(h[j][e], h[j][e], ss);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
  if (!WARP) {
    if (lane == 0) s_sum[warp] = ss;
    __syncthreads();
    ss = lane < nt / 32 ? s_sum[lane] : 0.f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
  }
  const float r = 1.0f / sqrtf(ss / static_cast<float>(p.n) + p.eps);
  // magnitudes order as their bits do; infinities and NaN are the largest
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int at = (j * nt + t) * 8;
    if (at < p.n) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p.gamma + at));
      const float4 b = __ldg(reinterpret_cast<const float4*>(p.gamma + at) + 1);
      const float g[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[j][e] = h[j][e] * r * g[e];
        if (kCodes) top = max(top, __float_as_uint(h[j][e]) & 0x7fffffffu);
      }
      if constexpr (!kCodes) store8(static_cast<O*>(p.out) + row * p.out_stride + at, h[j]);
    }
  }
  if constexpr (kCodes) {
    top = __reduce_max_sync(kFull, top);
    if (!WARP) {
      if (lane == 0) s_top[warp] = top;
      __syncthreads();
      top = __reduce_max_sync(kFull, lane < nt / 32 ? s_top[lane] : 0u);
    }
    const bool bad = top >= 0x7f800000u;
    const float s = bad ? __uint_as_float(0x7fc00000u) : __uint_as_float(top) * (1.0f / E4m3Code::kTop);
    if (t == 0) p.out_scale[row] = s;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int at = (j * nt + t) * 8;
      if (at < p.n) {
        uint32_t w[2] = {};
        if (!bad && s != 0.f) codes<E4m3Code>(h[j], s, w);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + row * p.out_stride + at) = make_uint2(w[0], w[1]);
      }
    }
  }
}

template <typename X, typename R, typename O>
cudaError_t launch(const AddNormParams& p, cudaStream_t s) {
  const int vecs = p.n / 8;
  // A warp a row needs no block barrier, and its lanes have several loads in flight; with few rows
  // a block a row has more of them.
  if (vecs <= 256 && p.rows >= 4 * p.n_sm) {
    const dim3 grid((p.rows + kRowsPerBlock - 1) / kRowsPerBlock), block(kRowsPerBlock * 32);
    if (vecs <= 64) return launch_pdl(add_norm_kernel<X, R, O, 2, true>, grid, block, 0, s, p);
    if (vecs <= 128) return launch_pdl(add_norm_kernel<X, R, O, 4, true>, grid, block, 0, s, p);
    return launch_pdl(add_norm_kernel<X, R, O, 8, true>, grid, block, 0, s, p);
  }
  const int v = vecs <= 512 ? 1 : 2;
  const dim3 grid(p.rows), block(((vecs + v - 1) / v + 31) / 32 * 32);
  return v == 1 ? launch_pdl(add_norm_kernel<X, R, O, 1, false>, grid, block, 0, s, p)
                : launch_pdl(add_norm_kernel<X, R, O, 2, false>, grid, block, 0, s, p);
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
