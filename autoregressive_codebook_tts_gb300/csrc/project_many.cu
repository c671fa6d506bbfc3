// The shared projection of many rows, with the adapters' wide products beside it, on pairs of SMs.
//
// Many rows bound the product by the tensor cores, and those by the operands that have to reach
// them: an SM takes 64 bytes a clock from L2.  Two CTAs therefore share a tile of 256 rows of W by up
// to 256 rows of x (cta_group::2): each brings its own 128 rows of W and half the rows of x.  The
// accumulator is double, so that a tile's products run under the epilogue of the last one (some 6000
// clocks, as long as the products of a tile of e4m3); with adapters that leaves room for 160 rows a
// tile, 416 clocks of L2 for 320 of products a column of 128 bytes.  A pair walks neighbouring tiles of
// the same rows of x, whose notes it takes once.
//
// K 2048, us: without adapters 4096 rows x 4096 columns in bf16 40.2 (1.71 PFLOP/s; the library's
// product 36.5), 6000 x 12288 in e4m3 92.7; 4093 rows of 7 requests x 4096, rank 32, bf16 78; 6000 rows x
// 12288 in e4m3, rank 16, of 5 requests 180, of 40 278.  (With two parts of v for bf16 outputs 76, 171 and
// 256; of that form 224 rows and one accumulator took 79, 202 and 247, 4093 rows of 40 requests
// with rank 64 124 against 105, 1000 rows of ten 90 against 72: runs then have more room, but each epilogue
// stands between two tiles' products.)
//
// z = v B_a^T: rows of a tile that lie together and share an adapter are a run.  A run has columns of
// its own (its rows, up to a multiple of 32), so its product meets no other adapter's rows, and what
// the columns behind it hold is not read.  v comes as its three bf16 parts.  Entries of B behind the
// adapter's rank are overwritten with zeros in shared memory before the product reads them.  Runs that
// find no room are added on the CUDA cores in the epilogue.
//
// Warps: 0-7 epilogue, 8 copies, 9 products (of the pair's first CTA), 10 notes (each row's
// adapter, runs and their columns, a tile ahead), 11 the zeros behind the ranks, 12 copies of B and v,
// which have stages of their own, as narrow as the ranks allow: they come while the tile's shared
// products run.
#include <cstdint>

#include "project_parts.cuh"

namespace tts {
namespace {

constexpr int kMaxNb = 256;
constexpr int kMaxRuns = 16;
constexpr int kThreads = 416;
constexpr int kCopyWarp = 8, kMmaWarp = 9, kNoteWarp = 10, kZeroWarp = 11, kZCopyWarp = 12;
constexpr int kMaxZSlots = 4;         // stages of B and v
constexpr int kMaxStages = 8;
constexpr int kTmemCols = 512;
constexpr int kWChunk = kM * kRowBytes;

constexpr int kNoZ = -1, kByRow = -2;

struct ManyPlan {
  int nb;                   // rows of x a tile, a multiple of 32
  int ch, stages;
  int n_rt, n_nt, n_tiles;
  int n_chunks, flat;
  int parts;                // 0: no adapters
  int zw, z_slots;          // ranks a stage of B and v holds (16, 32 or 64), such stages
  int z_off, bar_off, smem;
};

struct Notes {
  int ad[kMaxNb];           // -1 none, -2 no request
  int rank[kMaxNb];
  int zcol[kMaxNb];         // the row's column of z, -1 none
  __align__(16) float sx[kMaxNb];
  int run_ad[kMaxRuns], run_rank[kMaxRuns], run_first[kMaxRuns], run_n[kMaxRuns], run_col[kMaxRuns];
  int n_runs;
  // of each 16 rows: those of requests; where z of all of them begins (kNoZ: none has any; kByRow: some
  // have, or not in one piece, or some rows are of no request)
  uint32_t live[kMaxNb / 16];
  int z_at[kMaxNb / 16];
};

// ---- pairs of CTAs
template <bool E4M3>
__device__ __forceinline__ void mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (E4M3)
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
// One arrival at this barrier of both CTAs once the products issued so far are done.
__device__ __forceinline__ void commit2(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}"
      ::"r"(smem_u32(bar)), "h"(static_cast<uint16_t>(3)) : "memory");
}
// A copy into this CTA's shared memory that counts at a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load2(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
// Arrives at a barrier of either CTA; what it tells of was read, not written.
__device__ __forceinline__ void arrive_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ bool warp_wait_cluster(uint64_t* bar, uint32_t parity) {
  return __all_sync(kFull, mbar_wait_cluster(bar, parity, kWaitLimitCycles));
}
// 16 columns of this thread's lane; to be used after a wait that names them.
__device__ __forceinline__ void tmem_ask16(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_wait16(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
                 "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               ::"memory");
}
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, float& v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=f"(v) : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_wait(float (&a)[4], float (&b)[4]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(a[0]), "+f"(a[1]), "+f"(a[2]), "+f"(a[3]), "+f"(b[0]), "+f"(b[1]), "+f"(b[2]), "+f"(b[3])::"memory");
}

// Where byte i of rows of 2 zw bytes lies in their swizzle: the 16-byte pieces of 128 bytes trade
// places with each other (rows of 128, 64, 32 bytes).
__device__ __forceinline__ int swizzled(int i, int zw) {
  const int mask = zw == 64 ? 0x70 : zw == 32 ? 0x30 : 0x10;
  return i ^ ((i >> 3) & mask);
}
// Descriptor of K-major rows of 2 zw bytes in that swizzle (modes 2, 4, 6), 8-row groups one after
// the other.
__device__ __forceinline__ uint64_t z_desc(uint32_t addr, int zw) {
  const uint64_t mode = zw == 64 ? 2 : zw == 32 ? 4 : 6;
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (static_cast<uint64_t>(1) << 16) |
         (static_cast<uint64_t>(zw) << 32) | (static_cast<uint64_t>(1) << 46) | (mode << 61);
}

// z of four rows of the tile (row[u] < 0: none) for output column n, on the CUDA cores.
__device__ __forceinline__ void z_of_rows(const ProjectParams& p, const Notes& note, int t0, int r0, int n, const int (&row)[4],
                                          float (&z)[4]) {
  const int rm = p.ad.rank_max;
  int rank[4], most = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    rank[u] = row[u] >= 0 && n < p.n ? note.rank[t0 + row[u]] : 0;
    most = max(most, rank[u]);
  }
  for (int e = 0; e < most; e += 8) {
    uint4 w[4];
    float4 va[4], vb[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (e < rank[u]) {
        const int a = note.ad[t0 + row[u]];
        w[u] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.ad.b) +
                                                     (static_cast<int64_t>(a) * p.n + n) * rm + e));
        const float4* v = reinterpret_cast<const float4*>(p.v + static_cast<int64_t>(r0 + row[u]) * rm + e);
        va[u] = __ldcg(v);
        vb[u] = __ldcg(v + 1);
      }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (e < rank[u]) {
        float2 bp[4];
        b_pairs(w[u], rank[u] - e, bp);
        z[u] = fmaf(va[u].x, bp[0].x, z[u]);
        z[u] = fmaf(va[u].y, bp[0].y, z[u]);
        z[u] = fmaf(va[u].z, bp[1].x, z[u]);
        z[u] = fmaf(va[u].w, bp[1].y, z[u]);
        z[u] = fmaf(vb[u].x, bp[2].x, z[u]);
        z[u] = fmaf(vb[u].y, bp[2].y, z[u]);
        z[u] = fmaf(vb[u].z, bp[3].x, z[u]);
        z[u] = fmaf(vb[u].w, bp[3].y, z[u]);
      }
  }
}

template <bool E4M3>
__global__ void __launch_bounds__(kThreads, 1) project_many_kernel(const __grid_constant__ CUtensorMap wmap,
                                                                   const __grid_constant__ CUtensorMap xmap,
                                                                   const __grid_constant__ CUtensorMap bmap,
                                                                   const __grid_constant__ CUtensorMap vmap,
                                                                   const ProjectParams p, const ManyPlan q) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  // (the same offset in both CTAs: their shared memory begins alike)
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ Notes s_note[2];
  const int half = q.nb / 2, x_chunk = half * kRowBytes;
  const int stage_bytes = q.ch * (kWChunk + x_chunk), z_row = q.zw * 2;
  const int z_bytes = (kM + q.parts * half) * z_row;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + q.bar_off);  // (the first CTA's)
  uint64_t* empty = full + kMaxStages;
  uint64_t* z_full = empty + kMaxStages;                           // (the first CTA's)
  uint64_t* zl = z_full + kMaxZSlots;                                 // B and v have landed here,
  uint64_t* zr = zl + kMaxZSlots;                                     // (the first CTA's) and in the second CTA
  uint64_t* z_empty = zr + kMaxZSlots;
  uint64_t* acc_full = z_empty + kMaxZSlots;
  uint64_t* acc_empty = acc_full + 2;                              // (the first CTA's)
  uint64_t* note_full = acc_empty + 2;
  uint64_t* note_empty = note_full + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(note_empty + 2);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank());
  // this pair's tiles, neighbours along W first
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  const int tile0 = static_cast<int>(static_cast<int64_t>(pair) * q.n_tiles / pairs);
  const int tile1 = static_cast<int>(static_cast<int64_t>(pair + 1) * q.n_tiles / pairs);
  const int nst = (q.n_chunks + q.ch - 1) / q.ch;

  if (tid == 0) {
    for (int i = 0; i < q.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < q.z_slots; ++i) {
      mbar_init(&z_full[i], 1);
      mbar_init(&zl[i], 1);
      mbar_init(&zr[i], 1);
      mbar_init(&z_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 16);
      mbar_init(&note_full[i], 1);
      mbar_init(&note_empty[i], q.parts > 0 ? 11 : 8);   // epilogue 8; copies, products, zeros
    }
    mbar_init_fence();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_u32(s_tmem)), "n"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_sync_all();   // both CTAs' barriers and tensor memory are there
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  if (p.ad.n_adapters == 0) grid_wait();   // (else the narrow products' kernel has waited)
  grid_launch_dependents();

  const uint32_t zbase = static_cast<uint32_t>(2 * q.nb);
  // a tile's notes: the i-th tile of this CTA, to be given back with note_done
  auto note_wait = [&](int i) { return warp_wait(&note_full[i & 1], static_cast<uint32_t>(i >> 1) & 1u); };
  auto note_done = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&note_empty[i & 1]);
  };

  if (warp == kCopyWarp) {
    // ------------------------------------------------------------------ copies
    const int cols = kRowBytes / (E4M3 ? 1 : 2);
    bool ok = true;
    int it = 0, i = 0;
    auto next_stage = [&]() {
      const int s = it % q.stages;
      return it < q.stages || warp_wait(&empty[s], static_cast<uint32_t>(it / q.stages - 1) & 1u);
    };
    for (int tile = tile0; tile < tile1 && ok; ++tile, ++i) {
      const int rt = tile / q.n_nt, nt = tile - rt * q.n_nt;
      const int w0 = nt * 2 * kM + rank * kM, x0 = rt * q.nb + rank * half;
      for (int st = 0; st < nst && ok; ++st, ++it) {
        ok = next_stage();
        if (!ok) break;
        if (lane == 0) {
          const int s = it % q.stages;
          unsigned char* w = smem + s * stage_bytes;
          unsigned char* x = w + q.ch * kWChunk;
          const uint32_t bar = map_shared_rank(&full[s], 0);
          // the first CTA's barrier counts the bytes of both
          if (rank == 0) mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(2 * stage_bytes));
          const int c0 = st * q.ch;
          if (q.flat) {
            for (int c = 0; c < q.ch; ++c) {
              tma_load2(w + c * kWChunk, &wmap, (c0 + c) * cols, w0, 0, bar);
              tma_load2(x + c * x_chunk, &xmap, (c0 + c) * cols, x0, 0, bar);
            }
          } else {
            tma_load2(w, &wmap, 0, w0, c0, bar);
            tma_load2(x, &xmap, 0, x0, c0, bar);
          }
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
    // no copy may still be landing, and no product reading, when the CTA leaves
    for (int t = max(0, it - q.stages); t < it; ++t) warp_wait(&empty[t % q.stages], static_cast<uint32_t>(t / q.stages) & 1u);
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- products
    bool ok = true;
    int it = 0, iz = 0, i = 0;
    const uint32_t idesc = (1u << 4) | (E4M3 ? 0u : (1u << 7) | (1u << 10)) | (static_cast<uint32_t>(q.nb >> 3) << 17) |
                           (static_cast<uint32_t>(2 * kM >> 4) << 24);
    for (int tile = tile0; tile < tile1 && ok; ++tile, ++i) {
      if (rank != 0) {   // the first CTA issues for both
        if (q.parts > 0) {
          ok = note_wait(i);
          note_done(i);
        }
        continue;
      }
      const int buf = i & 1;
      if (i > 1 && !warp_wait_cluster(&acc_empty[buf], static_cast<uint32_t>(i / 2 - 1) & 1u)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem + static_cast<uint32_t>(buf * q.nb);
      for (int st = 0; st < nst && ok; ++st, ++it) {
        const int s = it % q.stages;
        if (!warp_wait(&full[s], static_cast<uint32_t>(it / q.stages) & 1u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t w = smem_u32(smem + s * stage_bytes), x = w + static_cast<uint32_t>(q.ch * kWChunk);
        for (int c = 0; c < q.ch; ++c) {
          const uint64_t ad = smem_desc(w + c * kWChunk), bd = smem_desc(x + c * x_chunk);
#pragma unroll
          for (int k = 0; k < kRowBytes / 32; ++k) mma2<E4M3>(d, ad + 2 * k, bd + 2 * k, idesc, st > 0 || c > 0 || k > 0);
        }
        commit2(&empty[s]);
      }
      if (q.parts > 0) {
        // z's products, 16 to 64 ranks at a time, behind the shared ones (asked for in between, they
        // cost those more than they saved); the last tile's z has to be read first
        ok = note_wait(i) && ok;
        const Notes& note = s_note[buf];
        const int runs = ok ? note.n_runs : 0;
        if (i > 0 && runs > 0) ok = warp_wait_cluster(&acc_empty[buf ^ 1], static_cast<uint32_t>((i - 1) / 2) & 1u);
        tc_fence_after();
        for (int k = 0; k < runs && ok; ++k) {
          const uint32_t zi = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(note.run_n[k] >> 3) << 17) |
                              (static_cast<uint32_t>(2 * kM >> 4) << 24);
          const int ranks = note.run_rank[k];
          const uint32_t zd = tmem + zbase + static_cast<uint32_t>(note.run_col[k]);
          for (int j = 0; j < ranks; j += q.zw, ++iz) {
            const int s = iz % q.z_slots;
            ok = warp_wait(&z_full[s], static_cast<uint32_t>(iz / q.z_slots) & 1u);
            if (!ok) break;
            tc_fence_after();
            const uint32_t w = smem_u32(smem + q.z_off + s * z_bytes);
            const int steps = (min(q.zw, ranks - j) + 15) / 16;
            for (int h = 0; h < q.parts; ++h) {
              const uint64_t ad = z_desc(w, q.zw), bd = z_desc(w + static_cast<uint32_t>((kM + h * half) * z_row), q.zw);
              for (int e = 0; e < steps; ++e) mma2<false>(zd, ad + 2 * e, bd + 2 * e, zi, j > 0 || h > 0 || e > 0);
            }
            commit2(&z_empty[s]);
          }
        }
        note_done(i);
      }
      commit2(&acc_full[buf]);
    }
    if (!ok && lane == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
  } else if (warp == kNoteWarp) {
    // ------------------------------------------------------------------- notes
    bool ok = true;
    int i = 0;
    constexpr int kC = kMaxNb / 32;
    const int zcols = kTmemCols - 2 * q.nb;
    for (int tile = tile0; tile < tile1 && ok; ++tile, ++i) {
      if (i > 1 && !warp_wait(&note_empty[i & 1], static_cast<uint32_t>(i / 2 - 1) & 1u)) {
        ok = false;
        break;
      }
      Notes& note = s_note[i & 1];
      if (i > 1 && tile / q.n_nt == (tile - 2) / q.n_nt) {   // the same rows
        if (lane == 0) mbar_arrive(&note_full[i & 1]);
        continue;
      }
      const int r0 = tile / q.n_nt * q.nb;
      int ad[kC], k[kC];
      float sx[kC];
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const int t = c * 32 + lane, r = r0 + t;
        const bool in = t < q.nb && r < p.rows;
        ad[c] = !in ? -2 : p.row_stream == nullptr ? r : __ldcg(p.row_stream + r);
        sx[c] = E4M3 && in ? __ldcg(p.x_scale + r) : 0.f;
      }
#pragma unroll
      for (int c = 0; c < kC; ++c)
        // (any negative adapter is none; -2 is for rows of no request)
        ad[c] = ad[c] < 0 ? -2 : p.ad.n_adapters == 0 || ad[c] >= p.n_streams ? -1 : max(__ldcg(p.stream_adapter + ad[c]), -1);
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        if (ad[c] >= p.ad.n_adapters) ad[c] = -1;
        k[c] = ad[c] < 0 ? 0 : p.ad.rank == nullptr ? p.ad.rank_max : __ldcg(p.ad.rank + ad[c]);
      }
      uint32_t edge[kC];
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const int t = c * 32 + lane;
        k[c] = min(max(k[c], 0), p.ad.rank_max);
        if (ad[c] >= 0 && k[c] == 0) ad[c] = -1;
        int prev = __shfl_up_sync(kFull, ad[c], 1);
        const int last = c > 0 ? __shfl_sync(kFull, ad[c > 0 ? c - 1 : 0], 31) : -3;
        if (lane == 0) prev = last;
        edge[c] = __ballot_sync(kFull, ad[c] != prev);
        if (t < q.nb) {
          note.ad[t] = ad[c];
          note.rank[t] = k[c];
          note.sx[t] = sx[c];
          note.zcol[t] = -1;
        }
      }
      __syncwarp();
      // runs get columns of z: those of eight rows or more first, then, with what is left, the others
      int n_runs = 0, col = 0;
      if (q.parts > 0)
        for (int pass = 0; pass < 2; ++pass) {
          int first = 0;
          while (first < q.nb) {
            // the next edge behind `first`
            int end = q.nb;
#pragma unroll
            for (int c = kC - 1; c >= 0; --c) {
              const int from = first + 1 - c * 32;
              const uint32_t m = from >= 32 ? 0u : from <= 0 ? edge[c] : edge[c] >> from << from;
              if (m != 0) end = min(end, c * 32 + __ffs(static_cast<int>(m)) - 1);
            }
            const int a = note.ad[first], len = end - first, n = (len + 31) / 32 * 32;
            if (a >= 0 && (pass == 0) == (len >= 8) && col + n <= zcols && n_runs < kMaxRuns) {
              for (int t = first + lane; t < end; t += 32) note.zcol[t] = col + t - first;
              if (lane == 0) {
                note.run_ad[n_runs] = a;
                note.run_rank[n_runs] = note.rank[first];
                note.run_first[n_runs] = first;
                note.run_n[n_runs] = n;
                note.run_col[n_runs] = col;
              }
              ++n_runs;
              col += n;
            }
            first = end;
          }
        }
      __syncwarp();
      for (int c = 0; c < q.nb / 16; ++c) {
        const int t = c * 16 + (lane & 15), a = note.ad[t], zc = note.zcol[t];
        const uint32_t live = __ballot_sync(kFull, a != -2) & 0xffffu;
        const int base = __shfl_sync(kFull, zc, 0);
        const bool none = __all_sync(kFull, a == -1 || q.parts == 0), all = __all_sync(kFull, zc >= 0 && zc - (lane & 15) == base);
        if (lane == 0) {
          note.live[c] = live;
          note.z_at[c] = live != 0xffffu ? kByRow : none ? kNoZ : all ? static_cast<int>(zbase) + base : kByRow;
        }
      }
      if (lane == 0) note.n_runs = n_runs;
      __syncwarp();
      if (lane == 0) mbar_arrive(&note_full[i & 1]);
    }
    if (!ok && lane == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
  } else if (warp == kZeroWarp) {
    // ------------------------------------------------- zeros behind the ranks
    bool ok = true;
    int iz = 0, i = 0;
    uint32_t phase = 0;   // of each slot's zl and zr
    if (q.parts > 0)
      for (int tile = tile0; tile < tile1 && ok; ++tile, ++i) {
        ok = note_wait(i);
        const Notes& note = s_note[i & 1];
        const int runs = ok ? note.n_runs : 0;
        for (int k = 0; k < runs && ok; ++k) {
          const int ranks = note.run_rank[k];
          for (int j = 0; j < ranks; j += q.zw, ++iz) {
            const int s = iz % q.z_slots, left = min(q.zw, ranks - j);
            if (left % 16 == 0) continue;
            if (!warp_wait(&zl[s], phase >> s & 1u)) {
              ok = false;
              break;
            }
            unsigned char* b = smem + q.z_off + s * z_bytes;
            for (int m = lane; m < kM; m += 32)
              for (int e = left; e < ((left + 15) & ~15); ++e)
                *reinterpret_cast<uint16_t*>(b + swizzled(m * z_row + e * 2, q.zw)) = 0;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (rank == 0) {
              // both CTAs' operands: the products may read them
              if (!warp_wait_cluster(&zr[s], phase >> s & 1u)) {
                ok = false;
                break;
              }
              if (lane == 0) mbar_arrive(&z_full[s]);
            } else if (lane == 0) {
              mbar_arrive_remote(map_shared_rank(&zr[s], 0));
            }
            phase ^= 1u << s;
          }
        }
        note_done(i);
      }
    if (!ok && lane == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
  } else if (warp == kZCopyWarp) {
    // ------------------------------ B rows and v's parts of runs, 64 ranks a stage
    bool ok = true;
    int iz = 0, i = 0;
    if (q.parts > 0) {
      grid_wait();   // (v)
      for (int tile = tile0; tile < tile1 && ok; ++tile, ++i) {
        const int rt = tile / q.n_nt, nt = tile - rt * q.n_nt, w0 = nt * 2 * kM + rank * kM;
        ok = note_wait(i);
        const Notes& note = s_note[i & 1];
        const int runs = ok ? note.n_runs : 0;
        for (int k = 0; k < runs && ok; ++k) {
          const int n2 = note.run_n[k] / 2, bytes = (kM + q.parts * n2) * z_row;
          for (int j = 0; j < note.run_rank[k]; j += q.zw, ++iz) {
            const int s = iz % q.z_slots;
            if (iz >= q.z_slots && !warp_wait(&z_empty[s], static_cast<uint32_t>(iz / q.z_slots - 1) & 1u)) {
              ok = false;
              break;
            }
            if (lane == 0) {
              unsigned char* b = smem + q.z_off + s * z_bytes;
              // where zeros have to be written first the stage is announced here, else with the pair's
              uint32_t bar = smem_u32(&zl[s]);
              if (min(q.zw, note.run_rank[k] - j) % 16 == 0) {
                bar = map_shared_rank(&z_full[s], 0);
                if (rank == 0) mbar_arrive_expect_tx(&z_full[s], static_cast<uint32_t>(2 * bytes));
              } else {
                mbar_arrive_expect_tx(&zl[s], static_cast<uint32_t>(bytes));
              }
              tma_load2(b, &bmap, j, note.run_ad[k] * p.n + w0, 0, bar);
              for (int h = 0; h < q.parts; ++h)
                for (int t = 0; t < n2; t += 16)
                  tma_load2(b + (kM + h * half + t) * z_row, &vmap, j,
                            rt * q.nb + note.run_first[k] + rank * n2 + t, h, bar);
            }
            __syncwarp();
          }
        }
        note_done(i);
      }
      // no copy may still be landing, and no product reading, when the CTA leaves
      for (int t = max(0, iz - q.z_slots); t < iz; ++t) warp_wait(&z_empty[t % q.z_slots], static_cast<uint32_t>(t / q.z_slots) & 1u);
    }
    if (!ok && lane == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
  } else {
    // ---------------------------------------------------------------- epilogue
    grid_wait();
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int t0 = warp < 4 ? 0 : half, chunks = half / 16;   // this warp's columns
    bool ok = true;
    int i = 0;
    for (int tile = tile0; tile < tile1 && ok; ++tile, ++i) {
      const int rt = tile / q.n_nt, nt = tile - rt * q.n_nt, r0 = rt * q.nb + t0;
      const int n = nt * 2 * kM + rank * kM + (warp & 3) * 32 + lane;
      const float sw = E4M3 && n < p.n ? __ldcg(p.w_scale + n) : 0.f;
      const Notes& note = s_note[i & 1];
      ok = note_wait(i);
      // (16 rows each) those taken by rows
      const uint32_t by_row = __ballot_sync(kFull, lane < chunks && note.z_at[t0 / 16 + (lane < chunks ? lane : 0)] == kByRow);
      ok = warp_wait(&acc_full[i & 1], static_cast<uint32_t>(i / 2) & 1u) && ok;
      if (!ok) {
        if (lane == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
        break;
      }
      tc_fence_after();
      const uint32_t dcol = tmem + static_cast<uint32_t>((i & 1) * q.nb) + lane_off;
      const int64_t row0 = static_cast<int64_t>(r0) * p.out_stride + n;
      // Rows where runs meet or end, four at a time; those whose run found no columns get z here.
#pragma unroll 1
      for (uint32_t some = by_row; some != 0; some &= some - 1) {
        const int c = __ffs(static_cast<int>(some)) - 1;
#pragma unroll 1
        for (uint32_t left = note.live[t0 / 16 + c]; left != 0;) {
          int row[4], alone[4];
          float y[4], z[4], zs[4] = {};
          bool any = false;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            row[u] = __ffs(static_cast<int>(left)) - 1;   // -1: none left
            left &= left - 1;
            const int t = t0 + c * 16 + max(row[u], 0), zc = note.zcol[t];
            tmem_ld1(dcol + static_cast<uint32_t>(t), y[u]);
            // (a row without z has no column there: any of the accumulator's instead)
            tmem_ld1(zc >= 0 ? tmem + zbase + static_cast<uint32_t>(zc) + lane_off : dcol + static_cast<uint32_t>(t), z[u]);
            alone[u] = q.parts > 0 && row[u] >= 0 && note.ad[t] >= 0 && zc < 0 ? row[u] : -1;
            any = any || alone[u] >= 0;
          }
          tmem_wait(y, z);
          if (any) z_of_rows(p, note, t0 + c * 16, r0 + c * 16, n, alone, zs);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (row[u] >= 0) {
              const int t = t0 + c * 16 + row[u];
              if (E4M3) y[u] *= note.sx[t] * sw;
              y[u] += note.zcol[t] >= 0 ? z[u] : zs[u];
              if (n < p.n) store_out(p, row0 + (c * 16 + row[u]) * p.out_stride, y[u]);
            }
        }
      }
      // The others 16 columns at a time; the next ones' loads are in flight while these are stored.
      float acc[16], z[16];
      auto load = [&](int c) {
        const int z_at = note.z_at[t0 / 16 + c];
        if (z_at != kByRow) tmem_ask16(dcol + static_cast<uint32_t>(t0 + c * 16), acc);
        if (z_at >= 0) tmem_ask16(tmem + static_cast<uint32_t>(z_at) + lane_off, z);
      };
      load(0);
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        const int z_at = note.z_at[t0 / 16 + c];
        tmem_wait16(acc);
        tmem_wait16(z);
        float y[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] = acc[j];
        if (E4M3) {
          const float2 w2 = make_float2(sw, sw);
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(&note.sx[t0 + c * 16 + j]);
            const float2 u = __fmul2_rn(make_float2(y[j], y[j + 1]), __fmul2_rn(make_float2(f.x, f.y), w2));
            const float2 v = __fmul2_rn(make_float2(y[j + 2], y[j + 3]), __fmul2_rn(make_float2(f.z, f.w), w2));
            y[j] = u.x;
            y[j + 1] = u.y;
            y[j + 2] = v.x;
            y[j + 3] = v.y;
          }
        }
        if (z_at >= 0) {
#pragma unroll
          for (int j = 0; j < 16; ++j) y[j] += z[j];
        }
        if (c + 1 < chunks) {
          load(c + 1);
        } else {
          // accumulator and z may be overwritten
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_relaxed(map_shared_rank(&acc_empty[i & 1], 0));
        }
        if (z_at != kByRow && n < p.n) {
          const int64_t at = row0 + c * 16 * p.out_stride;
          if (p.out_bf16) {
            __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) + at;
#pragma unroll
            for (int j = 0; j < 16; ++j) to[j * p.out_stride] = __float2bfloat16_rn(y[j]);
          } else {
            float* to = static_cast<float*>(p.out) + at;
#pragma unroll
            for (int j = 0; j < 16; ++j) to[j * p.out_stride] = y[j];
          }
        }
      }
      note_done(i);
    }
  }
  __syncwarp();
  tc_fence_before();
  // no CTA leaves while the other may still signal it, read its operands or land in its memory
  cluster_sync_all();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
  }
}

constexpr int kBars = (2 * kMaxStages + 4 * kMaxZSlots + 8) * 8 + 16;

template <bool E4M3>
size_t configure(int dev) {
  static std::mutex mtx;
  static size_t budget[64] = {};
  std::lock_guard<std::mutex> lock(mtx);
  if (budget[dev] != 0) return budget[dev];
  int optin = 0;
  cudaFuncAttributes fa;
  if (cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
      cudaFuncGetAttributes(&fa, project_many_kernel<E4M3>) != cudaSuccess || static_cast<size_t>(optin) <= fa.sharedSizeBytes)
    return 0;
  const size_t b = static_cast<size_t>(optin) - fa.sharedSizeBytes;
  if (cudaFuncSetAttribute(project_many_kernel<E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(b)) !=
      cudaSuccess)
    return 0;
  budget[dev] = b;
  return b;
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
  const int es = E4M3 ? 1 : 2, rm = p.ad.n_adapters > 0 ? p.ad.rank_max : 0, n_pairs = sm_count() / 2;
  ManyPlan q = {};
  q.n_nt = (p.n + 2 * kM - 1) / (2 * kM);
  q.n_chunks = (p.k * es + kRowBytes - 1) / kRowBytes;
  q.flat = p.k * es % kRowBytes != 0;
  // The rows a tile that make the least of waves times a tile's time: products (2 nb clocks a column
  // of 128 bytes) or L2 (256 + nb).  With adapters two accumulators and z share tensor memory.
  int64_t best = INT64_MAX;
  // 160 rows leave columns for two runs a tile, 128 for five.
  const int widest = rm == 0 ? kMaxNb : p.n_streams <= p.rows / 320 ? 160 : 128;
  for (int nb = 96; nb <= widest; nb += 32) {
    const int64_t tiles = static_cast<int64_t>(q.n_nt) * ((p.rows + nb - 1) / nb);
    const int64_t cost = (tiles + n_pairs - 1) / n_pairs * (2 * nb > 256 + nb ? 2 * nb : 256 + nb);
    if (cost <= best) {
      best = cost;
      q.nb = nb;
    }
  }
  q.n_rt = (p.rows + q.nb - 1) / q.nb;
  q.n_tiles = q.n_nt * q.n_rt;
  q.parts = rm == 0 ? 0 : 3;   // (bf16 outputs too need all: terms of z may cancel)
  // Larger copies stream faster: two columns of K a stage and three such stages, and as many of B and
  // v as then fit (one at least).
  const int chunk = kWChunk + q.nb / 2 * kRowBytes, room = static_cast<int>(budget) - 1024 - kBars;
  q.zw = rm <= 16 ? 16 : rm <= 32 ? 32 : 64;
  const int z_bytes = q.parts == 0 ? 0 : (kM + q.parts * (q.nb / 2)) * q.zw * 2;
  q.z_slots = z_bytes == 0 ? 0 : (room - 6 * chunk) / z_bytes;
  q.z_slots = q.z_slots > kMaxZSlots ? kMaxZSlots : z_bytes > 0 && q.z_slots < 1 ? 1 : q.z_slots;
  const int z = q.z_slots * z_bytes;
  q.ch = (room - z) / (2 * chunk) >= 3 ? 2 : 1;
  q.stages = (room - z) / (q.ch * chunk);
  q.stages = q.stages > kMaxStages ? kMaxStages : q.stages;
  q.z_off = q.stages * q.ch * chunk;
  q.bar_off = q.z_off + z;
  q.smem = 1024 + q.bar_off + kBars;
  CUtensorMap wmap, xmap, bmap, vmap;
  if (!encode(&wmap, p.w, es, p.k, p.k, p.n, kM, q.ch, q.flat) ||
      !encode(&xmap, p.x, es, p.x_stride, p.k, p.rows, q.nb / 2, q.ch, q.flat))
    return cudaErrorInvalidValue;
  bmap = vmap = wmap;
  if (q.parts > 0 && (!encode(&bmap, p.ad.b, 2, rm, rm, p.ad.n_adapters * p.n, kM, 1, true, 0, 1, q.zw) ||
                      !encode(&vmap, p.v_parts, 2, rm, rm, p.rows, 16, 1, true, 0, 3, q.zw)))
    return cudaErrorInvalidValue;
  if (rm > 0) {
    e = launch_shrink(p, s);
    if (e != cudaSuccess) return e;
  }
  const int grid = 2 * (q.n_tiles < n_pairs ? q.n_tiles : n_pairs);
  return launch_pairs(project_many_kernel<E4M3>, grid, kThreads, q.smem, s, wmap, xmap, bmap, vmap, p, q);
}

}  // namespace

// Whether the pairs' tiles of 160 rows would fill the device, which smaller tiles split over K do
// for fewer rows; and whether requests have 32 rows and more, as runs need.
bool project_is_many(const ProjectParams& p) {
  const int64_t tiles = static_cast<int64_t>((p.n + 2 * kM - 1) / (2 * kM)) * ((p.rows + 159) / 160);
  return p.rows > 256 && tiles >= sm_count() / 2 &&
         (p.ad.n_adapters == 0 || (p.row_stream != nullptr && p.n_streams <= p.rows / 32));
}

cudaError_t launch_project_many(const ProjectParams& p, cudaStream_t s) {
  return p.x_e4m3 ? launch_t<true>(p, s) : launch_t<false>(p, s);
}

}  // namespace tts
