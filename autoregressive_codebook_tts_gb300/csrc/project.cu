// A shared projection with every request's own low-rank adapter, as first kernels on the CUDA
// cores: the adapters' narrow products x A^T of every row, then 64 x 64 tiles of x W^T with the
// adapters' wide products added in the epilogue.  All in f32.
#include "cache_view.cuh"
#include "serve_kernels.h"

namespace tts {
namespace {

// The adapter of row r: -1 none, -2 the row is of no request.
__device__ __forceinline__ int row_adapter(const ProjectParams& p, int r, int* bad) {
  const int s = p.row_stream == nullptr ? r : __ldcg(p.row_stream + r);
  if (s < 0) return -2;
  if (p.ad.n_adapters == 0) return -1;
  if (s >= p.n_streams) {
    *bad |= TTS_EFLAG_ID_RANGE;
    return -1;
  }
  const int a = __ldcg(p.stream_adapter + s);
  if (a >= p.ad.n_adapters) {
    *bad |= TTS_EFLAG_ID_RANGE;
    return -1;
  }
  return a < 0 ? -1 : a;
}
__device__ __forceinline__ int adapter_rank(const ProjectParams& p, int a, int* bad) {
  const int r = p.ad.rank == nullptr ? p.ad.rank_max : __ldcg(p.ad.rank + a);
  if (r < 0 || r > p.ad.rank_max) *bad |= TTS_EFLAG_NVALID;
  return min(max(r, 0), p.ad.rank_max);
}

template <bool E4M3>
__device__ __forceinline__ float entry(const void* p, int64_t i) {
  if (E4M3) return E4m3Code::value(__ldg(static_cast<const uint8_t*>(p) + i));
  return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(p) + i)) << 16);
}

// v[r][j] = scale_a x_scale[r] sum_k x[r][k] A_a[j][k], a warp a rank of a row.
template <bool E4M3>
__global__ void __launch_bounds__(256) shrink_kernel(const ProjectParams p) {
  grid_wait();
  grid_launch_dependents();
  const int r = blockIdx.x, lane = threadIdx.x & 31;
  int bad = 0;
  const int a = row_adapter(p, r, &bad);
  const int rank = a >= 0 ? adapter_rank(p, a, &bad) : 0;
  if (threadIdx.x == 0 && bad != 0) set_err(p.err, bad);
  if (a < 0) return;
  float s = p.ad.scale == nullptr ? 1.f : __ldcg(p.ad.scale + a);
  if (E4M3) s *= __ldcg(p.x_scale + r);
  for (int j = threadIdx.x >> 5; j < rank; j += 8) {
    const int64_t at = (static_cast<int64_t>(a) * p.ad.rank_max + j) * p.k;
    float acc = 0.f;
    for (int k = lane; k < p.k; k += 32) acc = fmaf(entry<E4M3>(p.x, r * p.x_stride + k), entry<false>(p.ad.a, at + k), acc);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) acc += __shfl_xor_sync(kFull, acc, o);
    if (lane == 0) p.v[static_cast<int64_t>(r) * p.ad.rank_max + j] = acc * s;
  }
}

constexpr int kTile = 64, kStep = 16;

template <bool E4M3>
__global__ void __launch_bounds__(256) project_kernel(const ProjectParams p) {
  __shared__ float sx[kStep][kTile + 1], sw[kStep][kTile + 1];
  grid_wait();
  grid_launch_dependents();
  const int r0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < p.k; k0 += kStep) {
    for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
      const int row = i / kStep, k = i % kStep;
      const bool in = k0 + k < p.k;
      sx[k][row] = in && r0 + row < p.rows ? entry<E4M3>(p.x, (r0 + row) * p.x_stride + k0 + k) : 0.f;
      sw[k][row] = in && n0 + row < p.n ? entry<E4M3>(p.w, static_cast<int64_t>(n0 + row) * p.k + k0 + k) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sx[k][ty * 4 + i], sw[k][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + ty * 4 + i;
    if (r >= p.rows) break;
    int bad = 0;
    const int a = row_adapter(p, r, &bad);
    if (a == -2) continue;
    const int rank = a >= 0 ? adapter_rank(p, a, &bad) : 0;
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx + 16 * j;
      if (n >= p.n) continue;
      float y = acc[i][j];
      if (E4M3) y = y * __ldcg(p.x_scale + r) * __ldcg(p.w_scale + n);
      float z = 0.f;
      for (int q = 0; q < rank; ++q)
        z = fmaf(__ldcg(p.v + static_cast<int64_t>(r) * p.ad.rank_max + q),
                 entry<false>(p.ad.b, (static_cast<int64_t>(a) * p.n + n) * p.ad.rank_max + q), z);
      y += z;
      const int64_t at = r * p.out_stride + n;
      if (p.out_bf16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
      else static_cast<float*>(p.out)[at] = y;
    }
  }
}

template <bool E4M3>
cudaError_t launch_t(const ProjectParams& p, cudaStream_t s) {
  if (p.ad.n_adapters > 0) {
    const cudaError_t e = launch_pdl(shrink_kernel<E4M3>, dim3(p.rows), dim3(256), 0, s, p);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(project_kernel<E4M3>, dim3((p.n + kTile - 1) / kTile, (p.rows + kTile - 1) / kTile), dim3(256), 0, s, p);
}

}  // namespace

size_t project_workspace(int rows, int n, int k, bool x_e4m3, int rank_max) {
  return static_cast<size_t>(rows) * rank_max * sizeof(float);
}

cudaError_t launch_project(const ProjectParams& p, cudaStream_t s) {
  return p.x_e4m3 ? launch_t<true>(p, s) : launch_t<false>(p, s);
}

}  // namespace tts
