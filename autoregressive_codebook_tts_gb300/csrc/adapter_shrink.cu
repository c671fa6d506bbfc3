// The adapters' narrow products of a projection: v[r][j] = scale_a x_scale[r] sum_k x[r][k] A_a[j][k].
//
// Few rows: a warp a rank of a row, on the CUDA cores; every adapter's rows are read once a row that
// has it, and that is what bounds it.  Many rows: the tensor cores, 128 rows of x a tile against
// the stacked A of the tile's adapters (as many as fit 128 columns at a time), K split over a
// cluster; a row keeps the columns of its own adapter.  Rows in e4m3 are widened to bf16 in shared
// memory on the way, exactly.  Beside v in f32 the second form leaves v as three bf16 parts, whose
// sum is v, and notes which blocks of 16 rows share one adapter: there the wide product can run on
// the tensor cores too.
//
// K 2048: 32 rows of rank 16 5 us, 96 rows of up to 64 ranks 8 (a round trip for the row's adapter, one
// for its entries); 4093 rows of rank 32 12.5 us, 6000 rows of e4m3 17 (the widening), read from a launch list.
#include <map>
#include <tuple>

#include "project_parts.cuh"

namespace tts {
namespace {

// ---------------------------------------------------------------------------
// v[r][j] = scale_a x_scale[r] sum_k x[r][k] A_a[j][k], a warp a rank of a row; zeros from the rank
// to the next multiple of eight, up to where the epilogue reads.
// ---------------------------------------------------------------------------
constexpr int kShrinkWarps = 8;

// eight entries of a row
template <typename X> struct Raw;
template <> struct Raw<uint8_t> {
  uint2 v;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p) + i));
  }
  __device__ __forceinline__ void values(float (&f)[8]) const {
    float a[4], b[4];
    E4m3Code::values(v.x, a);
    E4m3Code::values(v.y, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = a[e];
      f[4 + e] = b[e];
    }
  }
};
template <> struct Raw<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i));
  }
  __device__ __forceinline__ void values(float (&f)[8]) const { unpack_bf16x8(v, f); }
};

// The row's entries are asked for while its adapter is looked up (three dependent loads), then the
// adapter's, 2048 of K at a time.
template <typename X>
__global__ void __launch_bounds__(kShrinkWarps * 32) shrink_kernel(const ProjectParams p) {
  constexpr int U = 8;
  grid_wait();
  grid_launch_dependents();
  const int r = blockIdx.x, lane = threadIdx.x & 31, j = blockIdx.y * kShrinkWarps + (threadIdx.x >> 5);
  Raw<X> x[U];
  Raw<__nv_bfloat16> w[U];
  const int64_t row = r * p.x_stride;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = u * 256 + lane * 8;
    if (k < p.k) x[u].load(p.x, row + k);
  }
  int bad = 0;
  const int a = row_adapter(p, r, &bad);
  const int rank = a >= 0 ? adapter_rank(p, a, &bad) : 0;
  if (blockIdx.y == 0 && threadIdx.x == 0 && bad != 0) set_err(p.err, bad);
  if (j >= ((rank + 7) & ~7)) return;
  float acc = 0.f;
  if (j < rank) {
    const int64_t at = (static_cast<int64_t>(a) * p.ad.rank_max + j) * p.k;
    for (int k0 = 0; k0 < p.k; k0 += U * 256) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * 256 + lane * 8;
        if (k < p.k) {
          if (k0 > 0) x[u].load(p.x, row + k);
          w[u].load(p.ad.a, at + k);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k0 + u * 256 + lane * 8 < p.k) {
          float f[8], g[8];
          x[u].values(f);
          w[u].values(g);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc = fmaf(f[e], g[e], acc);
        }
      }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) acc += __shfl_xor_sync(kFull, acc, o);
    if (sizeof(X) == 1) acc *= __ldcg(p.x_scale + r);
    if (p.ad.scale != nullptr) acc *= __ldcg(p.ad.scale + a);
  }
  if (lane == 0) p.v[static_cast<int64_t>(r) * p.ad.rank_max + j] = acc;
}

// ---------------------------------------------------------------------------
// Tensor cores
// ---------------------------------------------------------------------------
constexpr int kStackCols = 128;       // columns of the accumulator: ranks of the adapters of a pass
constexpr int kXBytes = kM * kRowBytes;
constexpr int kStackBytes = kStackCols * kRowBytes;
constexpr int kRawBytes = kM * 64;    // 64 e4m3 columns
constexpr int kMaxStages = 6;
constexpr int kMaxCluster = 8;
constexpr int kThreads = 192;         // warps 0-3 rows, 4 copies, 5 products
constexpr int kRows = 128;            // threads of the first

struct ShrinkPlan {
  int stages, split, n_chunks;        // K in chunks of 64 entries
  int per_pass;                       // adapters whose ranks fit the stack
  int red_off, bar_off, smem;
};

struct RowNotes {
  int ad[kM];
  int rank[kM];
  int run_ad[kM];      // adapters of the tile's runs of rows, in order
  int slot_ad[kM];     // and each of them once
  int first[4], leads[4];   // how many of them each warp's threads hold
};

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr) : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// v as three bf16 values of its own sign whose sum it is: eight bits each of the 24, cut off rather than
// rounded, so that none is larger than v.  None is 0 unless v is (a part that would be shares the one
// before it), and an infinity is three: so an infinite entry of B meets what it would have met in v,
// 0 times infinity only where v is 0.  (The parts are exact down to 2^-100; of a smaller v they may
// drop what is below bf16's range.)
__device__ __forceinline__ void parts_of(float v, float (&h)[3]) {
  auto top = [](float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); };
  h[0] = top(v);
  const float rest = v - h[0];
  h[1] = top(rest);
  h[2] = rest - h[1];
  if (!(fabsf(rest) > 0.f)) {   // eight bits, an infinity or NaN
    h[0] = 0.5f * v;
    h[1] = h[2] = 0.25f * v;
  } else if (h[2] == 0.f) {
    h[1] = h[2] = 0.5f * rest;
  }
}
// 16 codes as bf16, exactly
__device__ __forceinline__ void widen16(const uint4 w, uint4& lo, uint4& hi) {
  float f[16];
  CacheElem<CodeE4m3>::values(w, f);
  lo = make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
  hi = make_uint4(bf16_pair(f[8], f[9]), bf16_pair(f[10], f[11]), bf16_pair(f[12], f[13]), bf16_pair(f[14], f[15]));
}

template <bool E4M3>
__global__ void __launch_bounds__(kThreads, 1) shrink_tc_kernel(const __grid_constant__ CUtensorMap amap,
                                                                const __grid_constant__ CUtensorMap xmap,
                                                                const ProjectParams p, const ShrinkPlan q) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ RowNotes s_row;
  constexpr int kStage = kXBytes + kStackBytes + (E4M3 ? kRawBytes : 0);
  const int rm = p.ad.rank_max, red_ld = rm + 4;
  float* red = reinterpret_cast<float*>(smem + q.red_off);   // [128][red_ld] sums of this K range
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + q.bar_off);
  uint64_t* wide = full + kMaxStages;
  uint64_t* empty = wide + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + 1;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(acc_empty + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = q.split, rank = S > 1 ? static_cast<int>(blockIdx.y) : 0;
  const int r0 = blockIdx.x * kM;
  const int c0 = rank * q.n_chunks / S, nc = (rank + 1) * q.n_chunks / S - c0;

  if (tid == 0) {
    for (int i = 0; i < q.stages; ++i) {
      mbar_init(&full[i], 2);   // x, and the adapters' rows
      mbar_init(&wide[i], 4);
      mbar_init(&empty[i], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 4);
    mbar_init_fence();
  }
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_u32(s_tmem)), "n"(kStackCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  grid_wait();
  grid_launch_dependents();

  // ---- the rows' adapters, and the tile's list of them
  if (warp < 4) {
    const int r = r0 + tid;
    int bad = 0, a = -2, k = 0;
    if (r < p.rows) {
      a = row_adapter(p, r, &bad);
      if (a >= 0) k = adapter_rank(p, a, &bad);
    }
    if (k == 0 && a >= 0) a = -1;
    if (bad != 0 && rank == 0) set_err(p.err, bad);
    s_row.ad[tid] = a;
    s_row.rank[tid] = k;
    // a block of 16 rows whose adapters are one: that one; -1 none; -2 several
    int top = a, low = a >= 0 ? a : 0x7fffffff;
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) {
      top = max(top, __shfl_xor_sync(kFull, top, o));
      low = min(low, __shfl_xor_sync(kFull, low, o));
    }
    if (rank == 0 && (lane & 15) == 0 && r < p.rows) p.block_ad[r / 16] = top < 0 ? -1 : top == low ? top : -2;
    // the runs' adapters in order, then those among them that no earlier run has
    const int prev = __shfl_up_sync(kFull, a, 1);
    const bool edge = a >= 0 && (lane == 0 || prev != a);
    const uint32_t e = __ballot_sync(kFull, edge);
    if (lane == 0) s_row.first[warp] = __popc(e);
    named_barrier(1, kRows);
    int at = __popc(e & ((1u << lane) - 1)), edges = 0;
    for (int w = 0; w < 4; ++w) {
      at += w < warp ? s_row.first[w] : 0;
      edges += s_row.first[w];
    }
    if (edge) s_row.run_ad[at] = a;
    named_barrier(1, kRows);
    const int mine = tid < edges ? s_row.run_ad[tid] : -1;
    bool leads = mine >= 0;
    for (int u = 0; u < tid && leads; ++u) leads = s_row.run_ad[u] != mine;
    const uint32_t m = __ballot_sync(kFull, leads);
    if (lane == 0) s_row.leads[warp] = __popc(m);
    named_barrier(1, kRows);
    int base = 0;
    for (int w = 0; w < warp; ++w) base += s_row.leads[w];
    if (leads) s_row.slot_ad[base + __popc(m & ((1u << lane) - 1))] = mine;
  } else if (warp == 4 && lane == 0) {
    // rows of x need no notes
    const int n = nc < q.stages ? nc : q.stages;
    for (int i = 0; i < n; ++i) {
      unsigned char* x = smem + i * kStage;
      mbar_arrive_expect_tx(&full[i], static_cast<uint32_t>(E4M3 ? kRawBytes : kXBytes));
      tma_load(E4M3 ? x + kXBytes + kStackBytes : x, &xmap, (c0 + i) * 64, r0, 0, &full[i]);
    }
  }
  __syncthreads();
  const int n_slots = s_row.leads[0] + s_row.leads[1] + s_row.leads[2] + s_row.leads[3];
  const int passes = (n_slots + q.per_pass - 1) / q.per_pass;

  if (warp == 4) {
    // ------------------------------------------------------------------ copies
    if (lane == 0) {
      bool ok = true;
      int it = 0;
      for (int ps = 0; ps < passes && ok; ++ps) {
        const int cnt = min(q.per_pass, n_slots - ps * q.per_pass);
        for (int i = 0; i < nc; ++i, ++it) {
          const int s = it % q.stages;
          if (it >= q.stages && !mbar_wait(&empty[s], static_cast<uint32_t>(it / q.stages - 1) & 1u)) {
            ok = false;
            break;
          }
          unsigned char* x = smem + s * kStage;
          unsigned char* st = x + kXBytes;
          if (it >= min(nc, q.stages)) {   // (the first were asked for above)
            mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(E4M3 ? kRawBytes : kXBytes));
            tma_load(E4M3 ? st + kStackBytes : x, &xmap, (c0 + i) * 64, r0, 0, &full[s]);
          }
          mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(cnt * rm * kRowBytes));
          for (int k = 0; k < cnt; ++k)
            tma_load(st + k * rm * kRowBytes, &amap, (c0 + i) * 64, s_row.slot_ad[ps * q.per_pass + k] * rm, 0, &full[s]);
        }
      }
      if (!ok) set_err(p.err, TTS_EFLAG_TIMEOUT);
      // no copy may still be landing when the CTA leaves
      if (passes == 0)   // (rows of x that nothing reads: their second arrivals are missing)
        for (; it < min(nc, q.stages); ++it) mbar_arrive(&full[it]);
      for (int t = max(0, it - q.stages); t < it; ++t) mbar_wait(&full[t % q.stages], static_cast<uint32_t>(t / q.stages) & 1u);
    }
    __syncwarp();
  } else if (warp == 5) {
    // ---------------------------------------------------------------- products
    bool ok = true;
    int it = 0;
    for (int ps = 0; ps < passes && ok; ++ps) {
      const int cnt = min(q.per_pass, n_slots - ps * q.per_pass);
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>((cnt * rm + 15) / 16 * 2) << 17) |
                             (static_cast<uint32_t>(kM >> 4) << 24);
      if (ps > 0 && !warp_wait(acc_empty, static_cast<uint32_t>(ps - 1) & 1u)) {
        ok = false;
        break;
      }
      tc_fence_after();
      for (int i = 0; i < nc; ++i, ++it) {
        const int s = it % q.stages;
        if (!warp_wait(&full[s], static_cast<uint32_t>(it / q.stages) & 1u) ||
            (E4M3 && !warp_wait(&wide[s], static_cast<uint32_t>(it / q.stages) & 1u))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t x = smem_u32(smem + s * kStage);
        const uint64_t xd = smem_desc(x), ad = smem_desc(x + kXBytes);
#pragma unroll
        for (int k = 0; k < kRowBytes / 32; ++k) mma<false>(tmem, xd + 2 * k, ad + 2 * k, idesc, i > 0 || k > 0);
        mma_commit(&empty[s]);
      }
      mma_commit(acc_full);
    }
    if (!ok && lane == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
  } else {
    // -------------------------------------------------------------------- rows
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    const int a = s_row.ad[tid];
    bool ok = true;
    int it = 0;
    for (int ps = 0; ps < passes && ok; ++ps) {
      if (E4M3) {
        for (int i = 0; i < nc; ++i, ++it) {
          const int s = it % q.stages;
          ok = mbar_wait(&full[s], static_cast<uint32_t>(it / q.stages) & 1u) && ok;
          unsigned char* x = smem + s * kStage;
          const unsigned char* raw = x + kXBytes + kStackBytes;
          uint4 w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = lds128(raw + (j * kRows + tid) * 16);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // 16 codes of row m, pieces 2 c and 2 c + 1 of its swizzled 128 bytes
            const int m = (j * kRows + tid) / 4, c = tid & 3;
            uint4 lo, hi;
            widen16(w[j], lo, hi);
            *reinterpret_cast<uint4*>(x + m * kRowBytes + (((2 * c) ^ (m & 7)) << 4)) = lo;
            *reinterpret_cast<uint4*>(x + m * kRowBytes + (((2 * c + 1) ^ (m & 7)) << 4)) = hi;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&wide[s]);
        }
      }
      ok = mbar_wait(acc_full, static_cast<uint32_t>(ps) & 1u) && ok;
      ok = epilogue_all(ok, kRows);
      if (!ok) {
        if (tid == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
        break;
      }
      tc_fence_after();
      const int cnt = min(q.per_pass, n_slots - ps * q.per_pass);
      for (int i = 0; i < cnt; ++i) {
        const int mine = s_row.slot_ad[ps * q.per_pass + i];
        if (!__any_sync(kFull, a == mine)) continue;
        for (int j = 0; j < rm; j += 8) {
          float v[8];
          tmem_ld8(tmem + lane_off + static_cast<uint32_t>(i * rm + j), v);
          if (a == mine) {
            *reinterpret_cast<float4*>(red + tid * red_ld + j) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(red + tid * red_ld + j + 4) = make_float4(v[4], v[5], v[6], v[7]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty);
    }
  }
  __syncwarp();
  tc_fence_before();
  if (S > 1) cluster_sync_all();
  else __syncthreads();
  if (n_slots > 0) {
    // the K ranges' sums in rank order, scaled; zeros from the adapter's rank on
    uint32_t peer[kMaxCluster];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) peer[r] = r < S ? map_shared_rank(red, r) : 0u;
    const int lo = kM * rank / S, hi = kM * (rank + 1) / S, per = rm / 8;
    for (int u = tid; u < (hi - lo) * per; u += kThreads) {
      const int t = lo + u / per, j = (u - (u / per) * per) * 8, a = s_row.ad[t], r = r0 + t;
      if (a < 0) continue;
      const uint32_t off = static_cast<uint32_t>((t * red_ld + j) * 4);
      float4 pa[kMaxCluster], pb[kMaxCluster];
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c)
        if (c < S) {
          pa[c] = ld_cluster_f4(peer[c] + off);
          pb[c] = ld_cluster_f4(peer[c] + off + 16);
        }
      float v[8] = {};
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c)
        if (c < S) {
          v[0] += pa[c].x; v[1] += pa[c].y; v[2] += pa[c].z; v[3] += pa[c].w;
          v[4] += pb[c].x; v[5] += pb[c].y; v[6] += pb[c].z; v[7] += pb[c].w;
        }
      const float xs = E4M3 ? __ldcg(p.x_scale + r) : 1.f, as = p.ad.scale == nullptr ? 1.f : __ldcg(p.ad.scale + a);
      const int left = s_row.rank[t] - j;
      float h[3][8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = e < left ? v[e] * xs * as : 0.f;
        float part[3];
        parts_of(v[e], part);
#pragma unroll
        for (int i = 0; i < 3; ++i) h[i][e] = part[i];
      }
      const int64_t at = static_cast<int64_t>(r) * rm + j, all = static_cast<int64_t>(p.rows) * rm;
      *reinterpret_cast<float4*>(p.v + at) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(p.v + at + 4) = make_float4(v[4], v[5], v[6], v[7]);
#pragma unroll
      for (int i = 0; i < 3; ++i)
        *reinterpret_cast<uint4*>(p.v_parts + i * all + at) =
            make_uint4(bf16_pair(h[i][0], h[i][1]), bf16_pair(h[i][2], h[i][3]), bf16_pair(h[i][4], h[i][5]),
                       bf16_pair(h[i][6], h[i][7]));
    }
  }
  // no CTA leaves while a peer still reads its sums
  if (S > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
  if (warp == 5) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kStackCols) : "memory");
  }
}

template <bool E4M3>
size_t configure(int dev) {
  static std::mutex mtx;
  static size_t budget[64] = {};
  std::lock_guard<std::mutex> lock(mtx);
  if (budget[dev] != 0) return budget[dev];
  int optin = 0;
  cudaFuncAttributes fa;
  if (cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
      cudaFuncGetAttributes(&fa, shrink_tc_kernel<E4M3>) != cudaSuccess || static_cast<size_t>(optin) <= fa.sharedSizeBytes)
    return 0;
  const size_t b = static_cast<size_t>(optin) - fa.sharedSizeBytes;
  if (cudaFuncSetAttribute(shrink_tc_kernel<E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(b)) != cudaSuccess)
    return 0;
  budget[dev] = b;
  return b;
}

template <bool E4M3>
int max_active_clusters(int dev, int S, int smem) {
  static std::mutex mtx;
  static std::map<std::tuple<int, int, int>, int> cache;
  const auto key = std::make_tuple(dev, S, smem);
  std::lock_guard<std::mutex> lock(mtx);
  const auto it = cache.find(key);
  if (it != cache.end()) return it->second;
  const int n = active_clusters(shrink_tc_kernel<E4M3>, S, kThreads, smem);
  cache[key] = n;
  return n;
}

template <bool E4M3>
cudaError_t launch_tc(const ProjectParams& p, cudaStream_t s) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  const size_t budget = configure<E4M3>(dev);
  if (budget == 0) {
    const cudaError_t le = cudaGetLastError();
    return le != cudaSuccess ? le : cudaErrorInvalidValue;
  }
  constexpr int kStage = kXBytes + kStackBytes + (E4M3 ? kRawBytes : 0);
  const int rm = p.ad.rank_max, tiles = (p.rows + kM - 1) / kM;
  ShrinkPlan q = {};
  q.n_chunks = (p.k + 63) / 64;
  q.per_pass = kStackCols / rm;
  const int red = kM * (rm + 4) * 4, bars = (3 * kMaxStages + 2) * 8 + 16;
  int st = static_cast<int>((budget - 1024 - red - bars) / kStage);
  q.stages = st > kMaxStages ? kMaxStages : st;
  q.red_off = q.stages * kStage;
  q.bar_off = q.red_off + red;
  q.smem = 1024 + q.bar_off + bars;
  q.split = 1;
  // the largest cluster that keeps every tile's resident at once
  for (int c = q.n_chunks < kMaxCluster ? q.n_chunks : kMaxCluster; c > 1 && q.split == 1; --c)
    if (tiles <= max_active_clusters<E4M3>(dev, c, q.smem)) q.split = c;
  CUtensorMap amap, xmap;
  if (!encode(&amap, p.ad.a, 2, p.k, p.k, p.ad.n_adapters * rm, rm, 1, true) ||
      !encode(&xmap, p.x, E4M3 ? 1 : 2, p.x_stride, p.k, p.rows, kM, 1, true, E4M3 ? 64 : 0))
    return cudaErrorInvalidValue;
  return launch_clustered(shrink_tc_kernel<E4M3>, dim3(tiles, q.split), kThreads, q.smem, q.split, s, amap, xmap, p, q);
}

template <typename X>
cudaError_t launch_few(const ProjectParams& p, cudaStream_t s) {
  const dim3 grid(p.rows, (p.ad.rank_max + kShrinkWarps - 1) / kShrinkWarps);
  return launch_pdl(shrink_kernel<X>, grid, dim3(kShrinkWarps * 32), 0, s, p);
}

}  // namespace

cudaError_t launch_shrink(const ProjectParams& p, cudaStream_t s) {
  if (p.tc) return p.x_e4m3 ? launch_tc<true>(p, s) : launch_tc<false>(p, s);
  return p.x_e4m3 ? launch_few<uint8_t>(p, s) : launch_few<__nv_bfloat16>(p, s);
}

}  // namespace tts
