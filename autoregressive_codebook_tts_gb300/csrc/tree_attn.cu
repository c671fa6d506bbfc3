// Attention of a tree of drafted tokens over a cache, on the CUDA cores in f32 (f32 caches,
// or f32 queries over any cache), and the merge of partial rows that every form of it uses.
//
// An item's query rows (up to RB: nodes times the q heads of the kv head) share every cache
// row, which is read from HBM once, widened (and scaled) to f32 on its way to shared memory.
// Per 64-row tile: scores with two cache rows a thread against RB / 8 query rows (cache rows
// in lanes, query rows broadcast), the online softmax in base 2 with a warp to every eighth
// query row, then P V with four columns a thread.  The window is cut over all CTAs by cost
// (tree_plan.cuh); rows of unfinished items merge in tree_combine_kernel.  f32 cache and query, 16 / 8
// heads: one stream at 2750 rows 24 us, latency; 32 streams of 1500..4000 rows 268 us (2.7 TB/s, 0.40 of
// the measured copy rate); 8 streams of 16 nodes 126 us.
//
// A node row that is not visible must not touch the result even where it holds NaN or
// infinity, and 0 * NaN is NaN: non-finite V entries of node rows are replaced by 0 as they
// are staged, their rows noted, and added at the end to the query rows that see them.
#include <type_traits>

#include "tree_plan.cuh"

namespace tts {
namespace {

constexpr int kThreads = 256, kWarps = 8, kTile = 64;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The f32 value of entry d of a cache row of V.
template <typename KvT, int D>
__device__ __forceinline__ float v_entry(const CacheView& c, int64_t row, int d) {
  if constexpr (CacheElem<KvT>::kScaled) {
    const uint32_t code = static_cast<const uint8_t*>(c.v)[row * D + d];
    return (std::is_same<KvT, CodeI8>::value ? I8Code::value(code) : E4m3Code::value(code)) *
           c.v_scale[row];
  } else {
    return static_cast<float>(static_cast<const KvT*>(c.v)[row * D + d]);
  }
}

__device__ __forceinline__ bool finite_f32(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

template <int D, typename KvT, int RB>
struct TreeSmem {
  float k[kTile][D + 4];    // + 4: a column of 16-byte reads over 32 rows hits every bank once
  float v[kTile][D];
  float q[RB][D];
  float p[RB][kTile];
  float m[RB], l[RB], alpha[RB];
  unsigned long long see[RB];
  unsigned long long bad_v;  // node rows with non-finite V entries (in this piece)
};

template <int D, typename KvT, int RB>
__global__ void __launch_bounds__(kThreads, 2) tree_attn_kernel(const TreeParams p) {
  using E = CacheElem<KvT>;
  constexpr int RW = RB / kWarps;              // query rows of a warp
  constexpr int C4 = D / 4;                    // 4-column groups of a row
  constexpr int VR = kThreads / C4;            // thread groups of the P V product
  constexpr int RV = RB >= VR ? RB / VR : 1;   // its query rows a thread
  extern __shared__ __align__(16) unsigned char raw[];
  auto& s = *reinterpret_cast<TreeSmem<D, KvT, RB>*>(raw);
  const CacheView& c = p.cache;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_wait();
  grid_launch_dependents();
  if (blockIdx.x == 0 && p.err != nullptr) {
    bool any = false;
    for (int b = tid; b < c.B; b += kThreads) {
      bool bad;
      tree_window(p, b, &bad);
      any = any || bad;
    }
    if (any) set_err(p.err, TTS_EFLAG_NVALID);
  }
  const int gs = p.group >> 1;   // log2 of the group (1, 2 or 4)
  PieceWalk walk;
  Piece it;
  walk.init(p, blockIdx.x);
  while (walk.get(p, it)) {
    const int r_first = it.rb * RB, n_total = it.w.past + it.w.nodes;
    // A tile's vectors of K and V: loaded to registers (the first before anything else waits, the
    // next while a tile is worked on), then widened into shared memory.
    constexpr int CV = D / E::kVec;   // 16-byte vectors of a cache row
    constexpr int N = kTile * CV, NV = N / kThreads;
    static_assert(N % kThreads == 0, "whole vectors a thread");
    uint4 kr[NV], vr[NV];
    float sk[NV], sv[NV];
    auto fetch = [&](int tile) {
      const int r0 = tile * kTile, nrow = min(kTile, n_total - r0);
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int i = n * kThreads + tid, r = i / CV, u = i - r * CV;
        kr[n] = vr[n] = make_uint4(0, 0, 0, 0);
        sk[n] = sv[n] = 0.f;
        if (r >= nrow) continue;
        int page = 0;
        if (c.paged) {
          page = cache_page(c, it.b, r0 + r);
          if (page < 0) {
            set_err(p.err, TTS_EFLAG_PAGE);
            page = 0;
          }
        }
        const int64_t row = cache_row(c, it.b, it.g, r0 + r, page);
        kr[n] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(c.k) + row * (D * E::kBytes)) + u);
        vr[n] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(c.v) + row * (D * E::kBytes)) + u);
        if constexpr (E::kScaled) {
          sk[n] = __ldcg(c.k_scale + row);
          sv[n] = __ldcg(c.v_scale + row);
        }
      }
    };
    fetch(it.t0);
    // query rows, zero past the nodes
    for (int i = tid; i < RB * C4; i += kThreads) {
      const int r = i / C4, d4 = i - r * C4, t = (r_first + r) >> gs, h = (r_first + r) & (p.group - 1);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t < it.w.nodes) {
        const int64_t at = (static_cast<int64_t>(it.b) * p.T + t) * p.q_stride + (it.g * p.group + h) * D + d4 * 4;
        if (p.q_bf16) {
          const uint2 u = __ldcg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.q) + at));
          x = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                          __uint_as_float(u.y & 0xffff0000u));
        } else {
          x = __ldcg(reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + at));
        }
      }
      *reinterpret_cast<float4*>(&s.q[r][d4 * 4]) = x;
    }
    if (tid < RB) {
      const int t = (r_first + tid) >> gs;
      s.m[tid] = -INFINITY;
      s.l[tid] = 0.f;
      s.see[tid] = t < it.w.nodes ? seen_nodes(p, it.b, t, it.w.nodes) : 0ull;
    }
    if (tid == 0) s.bad_v = 0;
    float4 o[RV];
#pragma unroll
    for (int i = 0; i < RV; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int oc = tid % C4, og = tid / C4;
    for (int tile = it.t0; tile < it.t1; ++tile) {
      const int r0 = tile * kTile;
      __syncthreads();   // the tile before is consumed
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int i = n * kThreads + tid, r = i / CV, u = i - r * CV;
        float kf[E::kVec], vf[E::kVec];
        E::values(kr[n], kf);
        E::values(vr[n], vf);
        if constexpr (E::kScaled) {
#pragma unroll
          for (int e = 0; e < E::kVec; ++e) {
            kf[e] *= sk[n];
            vf[e] *= sv[n];
          }
        }
        if (r0 + r >= it.w.past && r0 + r < n_total) {
          bool any = false;
#pragma unroll
          for (int e = 0; e < E::kVec; ++e)
            if (!finite_f32(vf[e])) {
              any = true;
              vf[e] = 0.f;
            }
          if (any) atomicOr(&s.bad_v, 1ull << (r0 + r - it.w.past));
        }
#pragma unroll
        for (int e = 0; e < E::kVec; e += 4) {
          *reinterpret_cast<float4*>(&s.k[r][u * E::kVec + e]) = make_float4(kf[e], kf[e + 1], kf[e + 2], kf[e + 3]);
          *reinterpret_cast<float4*>(&s.v[r][u * E::kVec + e]) = make_float4(vf[e], vf[e + 1], vf[e + 2], vf[e + 3]);
        }
      }
      __syncthreads();
      if (tile + 1 < it.t1) fetch(tile + 1);
      // scores of cache rows lane and lane + 32 for the warp's query rows
      float a[RW][2];
#pragma unroll
      for (int i = 0; i < RW; ++i) a[i][0] = a[i][1] = 0.f;
#pragma unroll 4
      for (int d4 = 0; d4 < C4; ++d4) {
        const float4 k0 = *reinterpret_cast<const float4*>(&s.k[lane][d4 * 4]);
        const float4 k1 = *reinterpret_cast<const float4*>(&s.k[lane + 32][d4 * 4]);
#pragma unroll
        for (int i = 0; i < RW; ++i) {
          const float4 x = *reinterpret_cast<const float4*>(&s.q[warp * RW + i][d4 * 4]);
          a[i][0] = fmaf(x.x, k0.x, fmaf(x.y, k0.y, fmaf(x.z, k0.z, fmaf(x.w, k0.w, a[i][0]))));
          a[i][1] = fmaf(x.x, k1.x, fmaf(x.y, k1.y, fmaf(x.z, k1.z, fmaf(x.w, k1.w, a[i][1]))));
        }
      }
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        const int r = warp * RW + i;
        const unsigned long long see = s.see[r];
        bool vis[2];
        float z[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int j = r0 + lane + 32 * k, u = j - it.w.past;
          vis[k] = u < 0 || (u < it.w.nodes && ((see >> u) & 1ull) != 0);
          z[k] = vis[k] ? a[i][k] * p.scale_log2 : -INFINITY;
        }
        float mx = fmaxf(z[0], z[1]);
#pragma unroll
        for (int w = 16; w >= 1; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, w));
        const float m_old = s.m[r], m_new = fmaxf(m_old, mx);
        const float m_use = m_new == -INFINITY ? 0.f : m_new;
        const float e0 = vis[0] ? ex2(z[0] - m_use) : 0.f, e1 = vis[1] ? ex2(z[1] - m_use) : 0.f;
        float sum = e0 + e1;
#pragma unroll
        for (int w = 16; w >= 1; w >>= 1) sum += __shfl_xor_sync(kFull, sum, w);
        s.p[r][lane] = e0;
        s.p[r][lane + 32] = e1;
        __syncwarp();
        if (lane == 0) {
          const float al = m_old == -INFINITY ? 0.f : ex2(m_old - m_use);
          s.alpha[r] = al;
          s.m[r] = m_new;
          s.l[r] = s.l[r] * al + sum;
        }
      }
      __syncthreads();
      if (og < RB) {
#pragma unroll
        for (int i = 0; i < RV; ++i) {
          const float al = s.alpha[og * RV + i];
          o[i].x *= al; o[i].y *= al; o[i].z *= al; o[i].w *= al;
        }
#pragma unroll 2
        for (int j = 0; j < kTile; j += 4) {
          float4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const float4*>(&s.v[j + k][oc * 4]);
#pragma unroll
          for (int i = 0; i < RV; ++i) {
            const float4 w = *reinterpret_cast<const float4*>(&s.p[og * RV + i][j]);
            o[i].x = fmaf(w.x, v[0].x, fmaf(w.y, v[1].x, fmaf(w.z, v[2].x, fmaf(w.w, v[3].x, o[i].x))));
            o[i].y = fmaf(w.x, v[0].y, fmaf(w.y, v[1].y, fmaf(w.z, v[2].y, fmaf(w.w, v[3].y, o[i].y))));
            o[i].z = fmaf(w.x, v[0].z, fmaf(w.y, v[1].z, fmaf(w.z, v[2].z, fmaf(w.w, v[3].z, o[i].z))));
            o[i].w = fmaf(w.x, v[0].w, fmaf(w.y, v[1].w, fmaf(w.z, v[2].w, fmaf(w.w, v[3].w, o[i].w))));
          }
        }
      }
    }
    // visible non-finite V entries (their weights are above 0, or the row is NaN anyway)
    if (og < RB && s.bad_v != 0) {
#pragma unroll
      for (int i = 0; i < RV; ++i) {
        unsigned long long bits = s.bad_v & s.see[og * RV + i];
        while (bits != 0) {
          const int u = __ffsll(static_cast<long long>(bits)) - 1;
          bits &= bits - 1;
          const int pos = it.w.past + u;
          const int page = c.paged ? max(cache_page(c, it.b, pos), 0) : 0;
          const int64_t row = cache_row(c, it.b, it.g, pos, page);
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[e] = v_entry<KvT, D>(c, row, oc * 4 + e);
            if (finite_f32(x[e])) x[e] = 0.f;
          }
          o[i].x += x[0]; o[i].y += x[1]; o[i].z += x[2]; o[i].w += x[3];
        }
      }
    }
    if (og < RB) {
#pragma unroll
      for (int i = 0; i < RV; ++i) {
        const int r = og * RV + i, t = (r_first + r) >> gs, h = (r_first + r) & (p.group - 1);
        if (t >= it.w.nodes) continue;
        if (it.complete()) {
          const float l = s.l[r];
          // nothing seen: 0; only scores of -inf: NaN, as the formula's 0 / 0
          const float inv = l == 0.f ? (it.w.past > 0 || s.see[r] != 0 ? __uint_as_float(0x7fc00000u) : 0.f) : 1.f / l;
          store_tree_row4(p, it.b, t, it.g * p.group + h, D, oc * 4, o[i], inv);
        } else {
          const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + it.slot();
          *reinterpret_cast<float4*>(p.part + (slot * RB + r) * D + oc * 4) = o[i];
          if (oc == 0) p.ml[slot * RB + r] = make_float2(s.m[r], s.l[r]);
        }
      }
    }
    __syncthreads();   // the query rows and statistics are read
  }
}

// Merges the pieces of an item's row in CTA order: M = max m, L = sum l 2^(m - M),
// out = sum O 2^(m - M) / L.  One warp a row, the row's columns in its lanes; 32 pieces at a
// time, a lane each for their statistics, their rows eight loads in flight.
template <int D>
__global__ void __launch_bounds__(kThreads) tree_combine_kernel(const TreeParams p) {
  constexpr int PL = D / 32;   // columns a lane
  using Vec = typename std::conditional<PL == 4, float4, float2>::type;
  grid_wait();
  grid_launch_dependents();
  const CacheView& c = p.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_stream = c.n_kv_heads * p.n_rb;
  const int b = blockIdx.x / per_stream, k = blockIdx.x - b * per_stream;
  const int g = k / p.n_rb, rb = k - g * p.n_rb;
  Axis axis;
  int at_b = b, before;
  axis.find(p, 0, at_b, before);
  const TreeWindow w = axis.window(p, b);
  const int tiles = tree_tiles(p, w);
  if (tiles == 0) return;
  const int per = cost_per_cta(axis.total, p.n_cta), cost = item_cost(p, tiles);
  const int start = before + cost * k;
  const int c0 = start / per, c1 = (start + cost - 1) / per;
  // the CTAs whose pieces hold tiles are consecutive, first .. c1; the first whose range ends past
  // tile 0.  (A range that starts in the item's fixed units has no tiles of its own before it.)
  int first = c0;
  while (first < c1 && tile_at(p, per * (first + 1) - start, tiles) == 0) ++first;
  if (tile_at(p, per * (first + 1) - start, tiles) >= tiles) return;   // finished by one CTA
  for (int r = blockIdx.y * kWarps + warp; r < p.rows; r += gridDim.y * kWarps) {
    const int t = (rb * p.rows + r) >> (p.group >> 1), h = (rb * p.rows + r) & (p.group - 1);
    if (t >= w.nodes) break;
    float M = -INFINITY, L = 0.f, acc[PL];
#pragma unroll
    for (int e = 0; e < PL; ++e) acc[e] = 0.f;
    for (int x0 = first; x0 <= c1; x0 += 32) {
      const int x = x0 + lane;
      const int t0 = tile_at(p, per * x - start, tiles), t1 = tile_at(p, per * (x + 1) - start, tiles);
      // row of the lane's piece in the partials (any row, and no weight, where it has no tiles)
      const bool has = x <= c1 && t0 < t1;
      const int at = ((has ? x : first) * 2 + (has && t0 > 0 ? 0 : 1)) * p.rows + r;
      const float2 ml = has ? __ldcg(p.ml + at) : make_float2(-INFINITY, 0.f);
      const int n = min(32, c1 + 1 - x0);
      // the first rows travel with the statistics
      constexpr int BATCH = 8;
      Vec v[BATCH];
      auto fetch = [&](int j0) {
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
          const int src = __shfl_sync(kFull, at, (j0 + j) & 31);
          const bool live = __shfl_sync(kFull, static_cast<int>(has), (j0 + j) & 31) != 0 && j0 + j < n;
          v[j] = Vec{};
          if (live) v[j] = __ldcg(reinterpret_cast<const Vec*>(p.part + static_cast<int64_t>(src) * D) + lane);
        }
      };
      fetch(0);
      float top = ml.x;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      const float M1 = fmaxf(M, top), use = M1 == -INFINITY ? 0.f : M1;
      if (M1 > M && M > -INFINITY) {
        const float a = ex2(M - M1);
        L *= a;
#pragma unroll
        for (int e = 0; e < PL; ++e) acc[e] *= a;
      }
      M = M1;
      // a piece that saw nothing (all masked) has maximum -inf and weight 0; one that only saw NaN
      // scores (which no maximum holds) passes its NaN on
      const float wt = ml.x == -INFINITY ? (ml.y != ml.y ? 1.f : 0.f) : ex2(ml.x - use);
      float sum = ml.y * wt;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      L += sum;
      for (int j0 = 0; j0 < n; j0 += BATCH) {
        if (j0 > 0) fetch(j0);
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
          const float e = __shfl_sync(kFull, wt, (j0 + j) & 31);
          if (j0 + j < n) {
            acc[0] = fmaf(v[j].x, e, acc[0]);
            acc[1] = fmaf(v[j].y, e, acc[1]);
            if constexpr (PL == 4) {
              acc[2] = fmaf(v[j].z, e, acc[2]);
              acc[3] = fmaf(v[j].w, e, acc[3]);
            }
          }
        }
      }
    }
    const bool sees = w.past > 0 || seen_nodes(p, b, t, w.nodes) != 0;
    const float inv = L == 0.f ? (sees ? __uint_as_float(0x7fc00000u) : 0.f) : 1.f / L;
    const int64_t at = ((static_cast<int64_t>(b) * p.T + t) * p.n_q_heads + g * p.group + h) * D + lane * PL;
    if (p.q_bf16) {
#pragma unroll
      for (int e = 0; e < PL; e += 2) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
        *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.out) + at + e) = v;
      }
    } else {
#pragma unroll
      for (int e = 0; e < PL; e += 2)
        *reinterpret_cast<float2*>(static_cast<float*>(p.out) + at + e) = make_float2(acc[e] * inv, acc[e + 1] * inv);
    }
  }
}

template <int D, typename KvT, int RB>
cudaError_t launch_t(const TreeParams& p, cudaStream_t s) {
  auto kern = tree_attn_kernel<D, KvT, RB>;
  constexpr size_t smem = sizeof(TreeSmem<D, KvT, RB>);
  // (idempotent: the attribute is the same on every call)
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(p.n_cta), dim3(kThreads), smem, s, p);
}
template <int D, typename KvT>
cudaError_t launch_r(const TreeParams& p, cudaStream_t s) {
  if (p.rows == 8) return launch_t<D, KvT, 8>(p, s);
  if (p.rows == 16) return launch_t<D, KvT, 16>(p, s);
  if (p.rows == 32) return launch_t<D, KvT, 32>(p, s);
  return cudaErrorInvalidValue;
}
template <int D>
cudaError_t launch_kv(const TreeParams& p, int kv_dtype, cudaStream_t s) {
  switch (kv_dtype) {
    case TTS_F32: return launch_r<D, float>(p, s);
    case TTS_BF16: return launch_r<D, __nv_bfloat16>(p, s);
    case TTS_I8: return launch_r<D, CodeI8>(p, s);
    default: return launch_r<D, CodeE4m3>(p, s);
  }
}

}  // namespace

cudaError_t launch_tree_attn(const TreeParams& p, int kv_dtype, int head_dim, cudaStream_t s) {
  return head_dim == 64 ? launch_kv<64>(p, kv_dtype, s) : launch_kv<128>(p, kv_dtype, s);
}

cudaError_t launch_tree_combine(const TreeParams& p, int head_dim, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.cache.B) * p.cache.n_kv_heads * p.n_rb, (p.rows + kWarps - 1) / kWarps);
  return head_dim == 64 ? launch_pdl(tree_combine_kernel<64>, grid, dim3(kThreads), 0, s, p)
                        : launch_pdl(tree_combine_kernel<128>, grid, dim3(kThreads), 0, s, p);
}

}  // namespace tts
