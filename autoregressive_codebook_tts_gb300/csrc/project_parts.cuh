// What the projection's kernels share: rows' adapters, tcgen05 and TMA pieces, tensor maps.
#pragma once

#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "cache_view.cuh"
#include "checks.h"
#include "project_tile.h"
#include "serve_kernels.h"

namespace tts {
namespace {

// ---------------------------------------------------------------------------
// The adapter of row r: -1 none, -2 the row is of no request.
// ---------------------------------------------------------------------------
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

// ---------------------------------------------------------------------------
// Tensor-core pieces
// ---------------------------------------------------------------------------
// Shared-memory matrix descriptor: K-major rows of 128 bytes in the 128-byte swizzle (mode 2),
// 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (static_cast<uint64_t>(1) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Issued by one elected lane of a converged warp.
template <bool E4M3>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (E4M3)
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(kFull, mbar_wait(bar, parity));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, float v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(__float_as_uint(v)) : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Box {one 128-byte column, rows, columns} of a matrix seen as [K columns][rows][128 bytes].
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}
// 16 bytes at a shared-memory address
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts16(uint32_t a, const uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// A barrier of the epilogue's threads that also makes an outcome common to them.
__device__ __forceinline__ bool epilogue_all(bool v, int threads) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\tsetp.ne.u32 pi, %1, 0;\n\t"
      "bar.red.and.pred po, 1, %2, pi;\n\tselp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(out) : "r"(static_cast<uint32_t>(v)), "r"(threads) : "memory");
  return out != 0;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void store_out(const ProjectParams& p, int64_t at, float y) {
  if (p.out_bf16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
  else static_cast<float*>(p.out)[at] = y;
}

__device__ __forceinline__ float2 bf16_pair_f32(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// Eight entries of B as four pairs, zero from the rank on.
__device__ __forceinline__ void b_pairs(const uint4 w, int left, float2 (&b)[4]) {
  float f[8];
  unpack_bf16x8(w, f);
  if (left < 8) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = e < left ? f[e] : 0.f;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) b[e] = make_float2(f[2 * e], f[2 * e + 1]);
}
// four entries of v at once, the same address for the whole warp
__device__ __forceinline__ void v_pairs(uint32_t v, float2& a, float2& b) {
  const uint4 x = lds16(v);
  a = make_float2(__uint_as_float(x.x), __uint_as_float(x.y));
  b = make_float2(__uint_as_float(x.z), __uint_as_float(x.w));
}

// cuTensorMapEncodeTiled, looked up once through the runtime (no link against the driver)
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::mutex mtx;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::lock_guard<std::mutex> lock(mtx);
  if (fn == nullptr) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    else
      cudaGetLastError();
  }
  return fn;
}

// A row-major matrix of 1- or 2-byte entries as [K columns][rows][128 bytes] (whole columns), or
// as [1][rows][K] (flat), boxes of `box_rows` rows; raw > 0: boxes of that many columns,
// unswizzled; planes: that many such matrices, one after the other (flat); swizzled: boxes of that many
// 2-byte columns, 16, 32 or 64, in the swizzle of their width.
bool encode(CUtensorMap* map, const void* base, int es, int64_t stride, int k, int rows, int box_rows, int ch, bool flat,
            int raw = 0, int planes = 1, int swizzled = 0) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t cols = kRowBytes / es, pitch = static_cast<cuuint64_t>(stride) * es;
  cuuint64_t dims[3] = {flat ? static_cast<cuuint64_t>(k) : cols, static_cast<cuuint64_t>(rows),
                        flat ? static_cast<cuuint64_t>(planes) : static_cast<cuuint64_t>(k) / cols};
  cuuint64_t strides[2] = {pitch, flat ? pitch * rows : kRowBytes};
  cuuint32_t box[3] = {raw > 0 || swizzled > 0 ? static_cast<cuuint32_t>(raw + swizzled) : static_cast<cuuint32_t>(cols), static_cast<cuuint32_t>(box_rows), flat ? 1u : static_cast<cuuint32_t>(ch)};
  cuuint32_t es3[3] = {1, 1, 1};
  return enc(map, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
             strides, box, es3, CU_TENSOR_MAP_INTERLEAVE_NONE, raw > 0 ? CU_TENSOR_MAP_SWIZZLE_NONE : swizzled == 16 ? CU_TENSOR_MAP_SWIZZLE_32B : swizzled == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launch attributes of a kernel in clusters of (1, S) CTAs.
template <typename Kernel>
int active_clusters(Kernel kern, int S, int threads, int smem) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, S);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = static_cast<unsigned>(S);
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  return n;
}
template <typename Kernel, typename... Args>
cudaError_t launch_clustered(Kernel kern, dim3 grid, int threads, int smem, int S, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = static_cast<unsigned>(S);
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// The same in clusters of two along x: pairs of CTAs.
template <typename Kernel, typename... Args>
cudaError_t launch_pairs(Kernel kern, int grid, int threads, int smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace
}  // namespace tts
