// A shared projection with every request's own low-rank adapter:
//   out[r] = x[r] W^T + scale_a (x[r] A_a^T) B_a^T
//
// Two launches.  The first takes the adapters' narrow products v = scale x A^T (a warp a rank, f32).
// The second is the shared product on the tensor cores with the adapters' wide product added in
// its epilogue:
//   * a tile is 128 rows of W (the MMA's M) by up to 256 rows of x (its N), K in stages of one to
//     four 128-byte columns that TMA brings in the 128-byte swizzle; bf16 and e4m3 differ only in
//     the instruction's kind.  With W as M an accumulator lane is one output column, so that
//     a warp stores 32 neighbouring columns of a row and a thread needs one row of B_a;
//   * few tiles: the K range is split over a cluster, whose partial sums meet in rank order through
//     distributed shared memory.  Many tiles: CTAs walk them, and with up to 160 rows a tile the
//     accumulator is double, so the products of the next tile run under the epilogue;
//   * the epilogue's threads take z = v B_a^T on the CUDA cores, in f32, while the tensor cores work:
//     thread m reads row n = 128 tile + m of B_a through a private ring of asynchronous copies, v
//     comes by bulk copies of 32 rows, and z waits in tensor memory beside the accumulator.  So x A^T
//     is never rounded, a request's adapter never meets another request's row, and what lies behind
//     an adapter's rank is not used.
#include <map>
#include <mutex>
#include <tuple>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "cache_view.cuh"
#include "checks.h"
#include "serve_kernels.h"

namespace tts {
namespace {

constexpr int kM = 128;               // rows of W a tile
constexpr int kRowBytes = 128;        // bytes of K a swizzled row holds
constexpr int kWChunk = kM * kRowBytes;
constexpr int kMaxStages = 8;
constexpr int kMaxCluster = 8;
constexpr int kThreads = 192;         // warps 0-3 epilogue, 4 copies, 5 products
constexpr int kEpi = 128;
constexpr int kTmemCols = 512;
constexpr int kRedLd = kM + 16;       // floats between the rows of a partial
constexpr int kRingVecs = 16;         // 16-byte pieces of B a thread has room for

struct Plan {
  int nb, nbr;          // x rows a tile (a multiple of 16), and that rounded up to 32
  int ch, stages;       // 128-byte columns a stage, stages of the ring
  int n_acc;            // accumulators
  int split;            // CTAs that share a tile's K
  int n_rt, n_nt, n_tiles;
  int n_chunks;         // 128-byte columns of K (the last may be short)
  int flat;             // K is not whole columns: one copy each
  int ring;             // runs of B rows in flight
  int v_off, b_off, bar_off, smem;
  int vec_out;          // out rows take 16-byte (f32) or 8-byte (bf16) stores
};

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
// v[r][j] = scale_a x_scale[r] sum_k x[r][k] A_a[j][k], a warp a rank of a row; zeros from the rank
// to the next multiple of eight, up to where the epilogue reads.
// ---------------------------------------------------------------------------
constexpr int kShrinkWarps = 8;

// eight entries of a row
__device__ __forceinline__ void entries8(const uint8_t* x, int64_t i, float (&f)[8]) {
  const uint2 v = __ldg(reinterpret_cast<const uint2*>(x + i));
  float a[4], b[4];
  E4m3Code::values(v.x, a);
  E4m3Code::values(v.y, b);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[e] = a[e];
    f[4 + e] = b[e];
  }
}
__device__ __forceinline__ void entries8(const __nv_bfloat16* x, int64_t i, float (&f)[8]) {
  unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(x + i)), f);
}

template <typename X>
__global__ void __launch_bounds__(kShrinkWarps * 32) shrink_kernel(const ProjectParams p) {
  grid_wait();
  grid_launch_dependents();
  const int r = blockIdx.x, lane = threadIdx.x & 31, j = blockIdx.y * kShrinkWarps + (threadIdx.x >> 5);
  int bad = 0;
  const int a = row_adapter(p, r, &bad);
  const int rank = a >= 0 ? adapter_rank(p, a, &bad) : 0;
  if (blockIdx.y == 0 && threadIdx.x == 0 && bad != 0) set_err(p.err, bad);
  if (j >= ((rank + 7) & ~7)) return;
  float acc = 0.f;
  if (j < rank) {
    const X* x = static_cast<const X*>(p.x) + r * p.x_stride;
    const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(p.ad.a) + (static_cast<int64_t>(a) * p.ad.rank_max + j) * p.k;
#pragma unroll 4
    for (int k = lane * 8; k < p.k; k += 256) {
      float f[8], g[8];
      entries8(x, k, f);
      entries8(w, k, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc = fmaf(f[e], g[e], acc);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) acc += __shfl_xor_sync(kFull, acc, o);
    if (sizeof(X) == 1) acc *= __ldcg(p.x_scale + r);
    if (p.ad.scale != nullptr) acc *= __ldcg(p.ad.scale + a);
  }
  if (lane == 0) p.v[static_cast<int64_t>(r) * p.ad.rank_max + j] = acc;
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
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr) : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
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
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest n groups of this thread have landed; n + 1 = 1, 2, 4 or 8.
__device__ __forceinline__ void cp_async_wait(int ring) {
  if (ring == 8) asm volatile("cp.async.wait_group 7;" ::: "memory");
  else if (ring == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (ring == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
}
// A barrier of the epilogue's threads that also makes an outcome common to them.
__device__ __forceinline__ bool epilogue_all(bool v) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\tsetp.ne.u32 pi, %1, 0;\n\t"
      "bar.red.and.pred po, 1, 128, pi;\n\tselp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(out) : "r"(static_cast<uint32_t>(v)) : "memory");
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

struct TileInfo {
  int ad[256];       // adapter of the tile's rows: -1 none, -2 no request
  int rank[256];
  float sx[256];
  int run[256];      // rows that share an adapter: first | length << 16, within 32 rows each
  int n_runs;
};

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
__device__ __forceinline__ void v_pairs(const float* v, float2& a, float2& b) {
  const float4 x = *reinterpret_cast<const float4*>(v);
  a = make_float2(x.x, x.y);
  b = make_float2(x.z, x.w);
}

template <bool E4M3>
__global__ void __launch_bounds__(kThreads, 1) project_kernel(const __grid_constant__ CUtensorMap wmap,
                                                              const __grid_constant__ CUtensorMap xmap,
                                                              const ProjectParams p, const Plan q) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ TileInfo s_tile;
  const int stage_bytes = q.ch * (kWChunk + q.nb * kRowBytes);
  float* s_v = reinterpret_cast<float*>(smem + q.v_off);          // [2][32][rank_max]
  unsigned char* s_b = smem + q.b_off;                            // [kRingVecs][128] 16-byte pieces
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + q.bar_off);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* v_full = acc_empty + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(v_full + 2);
  float* red = reinterpret_cast<float*>(smem);   // partial sums, over the ring once it is drained

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = q.split, rank = S > 1 ? static_cast<int>(blockIdx.y) : 0;
  const int n_st = (q.n_chunks + q.ch - 1) / q.ch;
  const int st0 = static_cast<int>(static_cast<int64_t>(rank) * n_st / S);
  const int nst = static_cast<int>(static_cast<int64_t>(rank + 1) * n_st / S) - st0;

  if (tid == 0) {
    for (int i = 0; i < q.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
      mbar_init(&v_full[i], 1);
    }
    mbar_init_fence();
  }
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_u32(s_tmem)), "n"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  // Without adapters this is the call's first kernel: its inputs are an earlier kernel's.  With
  // them, the narrow products' kernel had passed that wait before it let this one start.
  if (p.ad.n_adapters == 0) grid_wait();
  grid_launch_dependents();

  if (warp == 4) {
    // ------------------------------------------------------------------ copies
    if (lane == 0) {
      const int cols = kRowBytes / (E4M3 ? 1 : 2);
      bool ok = true;
      int it = 0;
      for (int tile = blockIdx.x; tile < q.n_tiles && ok; tile += gridDim.x) {
        const int rt = tile % q.n_rt, nt = tile / q.n_rt;
        for (int i = 0; i < nst; ++i, ++it) {
          const int s = it % q.stages;
          if (it >= q.stages && !mbar_wait(&empty[s], static_cast<uint32_t>(it / q.stages - 1) & 1u)) {
            ok = false;
            break;
          }
          unsigned char* w = smem + s * stage_bytes;
          unsigned char* x = w + q.ch * kWChunk;
          const int c0 = (st0 + i) * q.ch;
          mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(stage_bytes));
          if (q.flat) {
            for (int c = 0; c < q.ch; ++c) {
              tma_load(w + c * kWChunk, &wmap, (c0 + c) * cols, nt * kM, 0, &full[s]);
              tma_load(x + c * q.nb * kRowBytes, &xmap, (c0 + c) * cols, rt * q.nb, 0, &full[s]);
            }
          } else {
            tma_load(w, &wmap, 0, nt * kM, c0, &full[s]);
            tma_load(x, &xmap, 0, rt * q.nb, c0, &full[s]);
          }
        }
      }
      if (!ok) set_err(p.err, TTS_EFLAG_TIMEOUT);
      // no copy may still be landing when the CTA leaves
      for (int t = max(0, it - q.stages); t < it; ++t) mbar_wait(&full[t % q.stages], static_cast<uint32_t>(t / q.stages) & 1u);
    }
    __syncwarp();
  } else if (warp == 5) {
    // ---------------------------------------------------------------- products
    // f32 accumulator (bits 4-5 = 1); bf16 operands are 1 at bits 7-9 and 10-12, e4m3 ones 0;
    // both K-major; N >> 3 at bit 17, M >> 4 at bit 24
    const uint32_t idesc = (1u << 4) | (E4M3 ? 0u : (1u << 7) | (1u << 10)) | (static_cast<uint32_t>(q.nb >> 3) << 17) |
                           (static_cast<uint32_t>(kM >> 4) << 24);
    bool ok = true;
    int it = 0, i = 0;
    for (int tile = blockIdx.x; tile < q.n_tiles && ok; tile += gridDim.x, ++i) {
      const int buf = i % q.n_acc, use = i / q.n_acc;
      if (use > 0 && !warp_wait(&acc_empty[buf], static_cast<uint32_t>(use - 1) & 1u)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem + static_cast<uint32_t>(buf * q.nbr);
      for (int st = 0; st < nst; ++st, ++it) {
        const int s = it % q.stages;
        if (!warp_wait(&full[s], static_cast<uint32_t>(it / q.stages) & 1u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t w = smem_u32(smem + s * stage_bytes), x = w + static_cast<uint32_t>(q.ch * kWChunk);
        for (int c = 0; c < q.ch; ++c) {
          const uint64_t ad = smem_desc(w + c * kWChunk), bd = smem_desc(x + c * q.nb * kRowBytes);
#pragma unroll
          for (int k = 0; k < kRowBytes / 32; ++k)   // 32 bytes of K an instruction
            mma<E4M3>(d, ad + 2 * k, bd + 2 * k, idesc, st > 0 || c > 0 || k > 0);
        }
        mma_commit(&empty[s]);   // the stage is free once these products have read it
      }
      mma_commit(&acc_full[buf]);
    }
    if (!ok && lane == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
  } else {
    // ---------------------------------------------------------------- epilogue
    grid_wait();   // v, and whoever read or wrote out before
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t zcol = tmem + static_cast<uint32_t>(q.n_acc * q.nbr) + lane_off;
    const int m = tid, rm = p.ad.rank_max;
    const int per_run = kRingVecs / q.ring;   // 16-byte pieces of a row of B
    const bool with = p.ad.n_adapters > 0;
    const int lo = q.nb * rank / S, hi = q.nb * (rank + 1) / S;   // rows whose adapters this CTA adds
    bool ok = true;
    uint32_t vq = 0;   // chunks of v asked for so far
    int i = 0;
    for (int tile = blockIdx.x; tile < q.n_tiles && ok; tile += gridDim.x, ++i) {
      const int rt = tile % q.n_rt, nt = tile / q.n_rt, r0 = rt * q.nb;
      const int n = nt * kM + m;
      for (int t = tid; t < q.nbr; t += kEpi) {
        const int r = r0 + t;
        int a = -2, k = 0, bad = 0;
        float sx = 0.f;
        if (t < q.nb && r < p.rows) {
          a = row_adapter(p, r, &bad);
          if (a >= 0) k = adapter_rank(p, a, &bad);
          if (E4M3) sx = __ldcg(p.x_scale + r);
        }
        s_tile.ad[t] = a >= 0 && k == 0 ? -1 : a;
        s_tile.rank[t] = k;
        s_tile.sx[t] = sx;
      }
      named_barrier(1, kEpi);
      int n_runs = 0;
      if (with) {
        const int c_lo = lo / 32, c_hi = (hi + 31) / 32;
        auto ask_v = [&](int c, uint32_t seq) {   // 32 rows of v
          const int r = r0 + c * 32, cnt = min(32, p.rows - r);
          const uint32_t bytes = static_cast<uint32_t>(cnt * rm) * 4u;
          mbar_arrive_expect_tx(&v_full[seq & 1], bytes);
          bulk_g2s_plain(s_v + (seq & 1) * 32 * rm, p.v + static_cast<int64_t>(r) * rm, bytes, &v_full[seq & 1]);
        };
        if (warp == 0) {
          int base = 0;
          for (int c = c_lo; c < c_hi; ++c) {
            const int t = c * 32 + lane;
            const int a = t >= lo && t < hi ? s_tile.ad[t] : -3;
            const int prev = __shfl_up_sync(kFull, a, 1);
            const uint32_t edge = __ballot_sync(kFull, lane == 0 || a != prev);
            const uint32_t first = __ballot_sync(kFull, a >= 0 && (edge >> lane & 1u));
            if (first >> lane & 1u) {
              const uint32_t later = lane == 31 ? 0u : edge >> (lane + 1);
              const int len = later != 0 ? __ffs(static_cast<int>(later)) : 32 - lane;
              s_tile.run[base + __popc(first & ((1u << lane) - 1))] = t | (len << 16);
            }
            base += __popc(first);
          }
          if (lane == 0) s_tile.n_runs = base;
        }
        named_barrier(1, kEpi);
        n_runs = s_tile.n_runs;
        const unsigned char* brow = static_cast<const unsigned char*>(p.ad.b) + static_cast<int64_t>(n) * rm * 2;
        auto ask_b = [&](int k) {
          if (k < n_runs && n < p.n) {
            const int t = s_tile.run[k] & 0xffff;
            const unsigned char* src = brow + static_cast<int64_t>(s_tile.ad[t]) * p.n * rm * 2;
            const int have = (s_tile.rank[t] + 7) / 8;
            unsigned char* dst = s_b + (k % q.ring) * per_run * (kEpi * 16) + tid * 16;
            for (int v = 0; v < have; ++v) cp_async16(dst + v * (kEpi * 16), src + v * 16);
          }
          cp_async_commit();
        };
        for (int k = 0; k < q.ring; ++k) ask_b(k);
        int cur = -1, c_next = c_lo;   // the chunk of v in use (copy cur_seq), the next to ask for
        uint32_t cur_seq = 0, seq = vq;
        // (thread 0 asks; all threads count along)
        auto ask_next = [&]() {
          if (c_next < c_hi && r0 + c_next * 32 < p.rows) {
            if (tid == 0) ask_v(c_next, seq);
            ++seq;
          }
          ++c_next;
        };
        const uint32_t seq0 = seq;
        ask_next();
        ask_next();
        for (int k = 0; k < n_runs; ++k) {
          const int run = s_tile.run[k], t0 = run & 0xffff, len = run >> 16, a_rank = s_tile.rank[t0];
          const int c = t0 / 32;
          while (cur < c) {
            // the next chunk of v: its buffer's last readers have passed this barrier
            cur = cur < 0 ? c_lo : cur + 1;
            if (cur > c_lo) {
              named_barrier(1, kEpi);
              ask_next();
            }
            cur_seq = seq0 + static_cast<uint32_t>(cur - c_lo);
            ok = mbar_wait(&v_full[cur_seq & 1], (cur_seq >> 1) & 1u) && ok;
          }
          cp_async_wait(q.ring);
          const float* v = s_v + (cur_seq & 1) * 32 * rm;
          const unsigned char* b = s_b + (k % q.ring) * per_run * (kEpi * 16) + tid * 16;
          const int have = (a_rank + 7) / 8;
          if (len >= 8) {
            float2 z[32];
#pragma unroll
            for (int t = 0; t < 32; ++t) z[t] = make_float2(0.f, 0.f);
            for (int e = 0; e < have; ++e) {
              float2 bp[4];
              b_pairs(lds128(b + e * (kEpi * 16)), a_rank - 8 * e, bp);
#pragma unroll
              for (int t = 0; t < 32; ++t) {
                float2 v0, v1, v2, v3;
                v_pairs(v + t * rm + e * 8, v0, v1);
                v_pairs(v + t * rm + e * 8 + 4, v2, v3);
                z[t] = __ffma2_rn(v0, bp[0], z[t]);
                z[t] = __ffma2_rn(v1, bp[1], z[t]);
                z[t] = __ffma2_rn(v2, bp[2], z[t]);
                z[t] = __ffma2_rn(v3, bp[3], z[t]);
              }
            }
            const int first = t0 - c * 32;
#pragma unroll
            for (int t = 0; t < 32; ++t)
              if (t >= first && t < first + len) tmem_st1(zcol + static_cast<uint32_t>(c * 32 + t), z[t].x + z[t].y);
          } else {
            for (int t = t0; t < t0 + len; ++t) {
              float2 z = make_float2(0.f, 0.f), y = z;
              for (int e = 0; e < have; ++e) {
                float2 bp[4], v0, v1, v2, v3;
                b_pairs(lds128(b + e * (kEpi * 16)), a_rank - 8 * e, bp);
                const float* vt = v + (t - c * 32) * rm + e * 8;
                v_pairs(vt, v0, v1);
                v_pairs(vt + 4, v2, v3);
                z = __ffma2_rn(v0, bp[0], z);
                y = __ffma2_rn(v1, bp[1], y);
                z = __ffma2_rn(v2, bp[2], z);
                y = __ffma2_rn(v3, bp[3], y);
              }
              tmem_st1(zcol + static_cast<uint32_t>(t), (z.x + z.y) + (y.x + y.y));
            }
          }
          ask_b(k + q.ring);
        }
        // copies of chunks that no run needed: waited for, so that every phase is used once
        for (uint32_t w = cur < 0 ? seq0 : cur_seq + 1; w != seq; ++w) ok = mbar_wait(&v_full[w & 1], (w >> 1) & 1u) && ok;
        vq = seq;
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        tmem_wait_st();
      }
      // ---- the accumulator
      const int buf = i % q.n_acc, use = i / q.n_acc;
      ok = mbar_wait(&acc_full[buf], static_cast<uint32_t>(use) & 1u) && ok;
      ok = epilogue_all(ok);
      if (!ok) {
        if (tid == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
        break;
      }
      tc_fence_after();
      const uint32_t dcol = tmem + static_cast<uint32_t>(buf * q.nbr) + lane_off;
      const float sw = E4M3 && n < p.n ? __ldcg(p.w_scale + n) : 0.f;
      for (int c = 0; c < q.nbr / 32; ++c) {
        float acc[32], z[32];
        tmem_ld32(dcol + c * 32, acc);
        const int a = s_tile.ad[c * 32 + lane];
        const int t = c * 32 + lane;
        const uint32_t live = __ballot_sync(kFull, a != -2);
        const uint32_t has = __ballot_sync(kFull, a >= 0 && t >= lo && t < hi);
        if (has != 0) tmem_ld32(zcol + c * 32, z);
        if (E4M3) {
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[j] *= s_tile.sx[c * 32 + j] * sw;
        }
        if (has != 0) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (has >> j & 1u) acc[j] += z[j];
        }
        if (S == 1) {
          if (n < p.n) {
            const int64_t at = static_cast<int64_t>(r0 + c * 32) * p.out_stride + n;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (live >> j & 1u) store_out(p, at + j * p.out_stride, acc[j]);
          }
        } else {
          // (every MMA of this CTA has read the ring)
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c * 32 + j < q.nb) red[(c * 32 + j) * kRedLd + m] = acc[j];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[buf]);
      named_barrier(1, kEpi);   // the tile's notes may change
    }
  }
  if (S > 1) {
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();   // every CTA's partial is in its shared memory
    if (warp < 4) {
      const int rt = static_cast<int>(blockIdx.x) % q.n_rt, nt = static_cast<int>(blockIdx.x) / q.n_rt;
      const int lo = q.nb * rank / S, hi = q.nb * (rank + 1) / S;
      uint32_t peer[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) peer[r] = r < S ? map_shared_rank(red, r) : 0u;
      const int n = nt * kM + lane * 4;
      for (int t = lo + warp; t < hi; t += 4) {
        if (s_tile.ad[t] == -2) continue;
        const uint32_t off = static_cast<uint32_t>((t * kRedLd + lane * 4) * 4);
        float4 part[kMaxCluster];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) part[r] = r < S ? ld_cluster_f4(peer[r] + off) : make_float4(0.f, 0.f, 0.f, 0.f);
        float4 y = part[0];
#pragma unroll
        for (int r = 1; r < kMaxCluster; ++r)
          if (r < S) {
            y.x += part[r].x;
            y.y += part[r].y;
            y.z += part[r].z;
            y.w += part[r].w;
          }
        const int64_t at = static_cast<int64_t>(rt * q.nb + t) * p.out_stride + n;
        if (q.vec_out && n + 3 < p.n) {
          if (p.out_bf16) {
            const __nv_bfloat162 a = __floats2bfloat162_rn(y.x, y.y), b = __floats2bfloat162_rn(y.z, y.w);
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
          } else {
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = y;
          }
        } else {
          if (n < p.n) store_out(p, at, y.x);
          if (n + 1 < p.n) store_out(p, at + 1, y.y);
          if (n + 2 < p.n) store_out(p, at + 2, y.z);
          if (n + 3 < p.n) store_out(p, at + 3, y.w);
        }
      }
    }
    // no CTA leaves while a peer still reads its partial
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
  } else {
    tc_fence_before();
    __syncthreads();
  }
  if (warp == 5) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
  }
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
// as [1][rows][K] (flat), boxes of `box_rows` rows.
bool encode(CUtensorMap* map, const void* base, int es, int64_t stride, int k, int rows, int box_rows, int ch, bool flat) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t cols = kRowBytes / es, pitch = static_cast<cuuint64_t>(stride) * es;
  cuuint64_t dims[3] = {flat ? static_cast<cuuint64_t>(k) : cols, static_cast<cuuint64_t>(rows),
                        flat ? 1 : static_cast<cuuint64_t>(k) / cols};
  cuuint64_t strides[2] = {pitch, flat ? pitch : kRowBytes};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(cols), static_cast<cuuint32_t>(box_rows), flat ? 1u : static_cast<cuuint32_t>(ch)};
  cuuint32_t es3[3] = {1, 1, 1};
  return enc(map, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
             strides, box, es3, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kBarBytes = (2 * kMaxStages + 6) * 8 + 16;

// The dynamic shared memory a CTA of the kernel may take on device `dev`, set as its limit once
// per device; 0 on failure.
template <bool E4M3>
size_t configure(int dev) {
  static std::mutex mtx;
  static size_t budget[64] = {};
  std::lock_guard<std::mutex> lock(mtx);
  if (budget[dev] != 0) return budget[dev];
  int optin = 0;
  cudaFuncAttributes fa;
  if (cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
      cudaFuncGetAttributes(&fa, project_kernel<E4M3>) != cudaSuccess || static_cast<size_t>(optin) <= fa.sharedSizeBytes)
    return 0;
  const size_t b = static_cast<size_t>(optin) - fa.sharedSizeBytes;
  if (cudaFuncSetAttribute(project_kernel<E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(b)) != cudaSuccess)
    return 0;
  budget[dev] = b;
  return b;
}

// Clusters of S CTAs that the device keeps resident at once (cached).
template <bool E4M3>
int max_active_clusters(int dev, int S, int smem) {
  static std::mutex mtx;
  static std::map<std::tuple<int, int, int>, int> cache;
  const auto key = std::make_tuple(dev, S, smem);
  std::lock_guard<std::mutex> lock(mtx);
  const auto it = cache.find(key);
  if (it != cache.end()) return it->second;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, S);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = static_cast<unsigned>(S);
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, project_kernel<E4M3>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  cache[key] = n;
  return n;
}

// Shared memory of a plan: the ring, two chunks of v, the ring of B rows, barriers.
void lay_out(Plan& q, int rank_max, size_t budget) {
  const int stage = q.ch * (kWChunk + q.nb * kRowBytes);
  q.ring = rank_max == 0 ? 1 : rank_max <= 16 ? 8 : rank_max <= 32 ? 4 : rank_max <= 64 ? 2 : 1;
  const int v = 2 * 32 * rank_max * 4, b = rank_max == 0 ? 0 : kRingVecs * kEpi * 16;
  const int fixed = 1024 + v + b + kBarBytes;
  int st = static_cast<int>((budget - fixed) / stage);
  const int per_cta = (q.n_chunks + q.ch - 1) / q.ch;
  st = st > kMaxStages ? kMaxStages : st;
  if (q.n_tiles * q.split <= 1 || q.split > 1) st = st > per_cta ? per_cta : st;
  q.stages = st < 1 ? 1 : st;
  // (a cluster's partial sums take the ring's place)
  int ring = q.stages * stage;
  const int red = q.split > 1 ? q.nb * kRedLd * 4 : 0;
  if (ring < red) ring = (red + 1023) / 1024 * 1024;
  q.v_off = ring;
  q.b_off = ring + v;
  q.bar_off = q.b_off + b;
  q.smem = 1024 + q.bar_off + kBarBytes;
}

template <bool E4M3>
cudaError_t launch_t(const ProjectParams& p, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  const size_t budget = configure<E4M3>(dev);
  if (budget == 0) {
    const cudaError_t le = cudaGetLastError();
    return le != cudaSuccess ? le : cudaErrorInvalidValue;
  }
  const int es = E4M3 ? 1 : 2, rm = p.ad.n_adapters > 0 ? p.ad.rank_max : 0, n_sm = sm_count();
  Plan q = {};
  q.n_nt = (p.n + kM - 1) / kM;
  q.n_chunks = (p.k * es + kRowBytes - 1) / kRowBytes;
  q.flat = p.k * es % kRowBytes != 0;
  // Up to 256 rows are one tile where that leaves every CTA one tile at most; else tiles of up to
  // 160 rows, of which two accumulators and z fit tensor memory.
  const int most = p.rows <= 256 && q.n_nt <= n_sm ? 256 : 160;
  q.n_rt = (p.rows + most - 1) / most;
  q.nb = ((p.rows + q.n_rt - 1) / q.n_rt + 15) / 16 * 16;
  q.n_rt = (p.rows + q.nb - 1) / q.nb;
  q.nbr = (q.nb + 31) / 32 * 32;
  q.n_acc = q.nbr <= 160 ? 2 : 1;
  q.n_tiles = q.n_nt * q.n_rt;
  q.ch = q.nb <= 32 ? 4 : q.nb <= 128 ? 2 : 1;
  q.split = 1;
  if (q.n_tiles < n_sm) {
    // the largest cluster that keeps every tile's resident at once
    const int n_st = (q.n_chunks + q.ch - 1) / q.ch;
    for (int c = n_st < kMaxCluster ? n_st : kMaxCluster; c > 1 && q.split == 1; --c) {
      Plan t = q;
      t.split = c;
      lay_out(t, rm, budget);
      if (static_cast<size_t>(t.smem) <= budget && q.n_tiles <= max_active_clusters<E4M3>(dev, c, t.smem)) q.split = c;
    }
  }
  lay_out(q, rm, budget);
  if (static_cast<size_t>(q.smem) > budget) return cudaErrorInvalidConfiguration;
  const int quantum = p.out_bf16 ? 8 : 16;
  q.vec_out = p.out_stride * (p.out_bf16 ? 2 : 4) % quantum == 0;
  CUtensorMap wmap, xmap;
  if (!encode(&wmap, p.w, es, p.k, p.k, p.n, kM, q.ch, q.flat) ||
      !encode(&xmap, p.x, es, p.x_stride, p.k, p.rows, q.nb, q.ch, q.flat))
    return cudaErrorInvalidValue;
  if (rm > 0) {
    using X = typename std::conditional<E4M3, uint8_t, __nv_bfloat16>::type;
    e = launch_pdl(shrink_kernel<X>, dim3(p.rows, (rm + kShrinkWarps - 1) / kShrinkWarps), dim3(kShrinkWarps * 32), 0, s, p);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = q.split > 1 ? dim3(q.n_tiles, q.split) : dim3(q.n_tiles < n_sm ? q.n_tiles : n_sm);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = q.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = static_cast<unsigned>(q.split);
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, project_kernel<E4M3>, wmap, xmap, p, q);
}

}  // namespace

size_t project_workspace(int rows, int n, int k, bool x_e4m3, int rank_max) {
  return static_cast<size_t>(rows) * rank_max * sizeof(float);
}

cudaError_t launch_project(const ProjectParams& p, cudaStream_t s) {
  return p.x_e4m3 ? launch_t<true>(p, s) : launch_t<false>(p, s);
}

}  // namespace tts
