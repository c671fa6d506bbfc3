// The shared projection of many rows, with the adapters' wide products beside it, on pairs of SMs.
//
// Many rows bound the product by the tensor cores, and those by the operands that have to reach
// them.  Two CTAs therefore share a tile of 256 rows of W by up to 160 rows of x (cta_group::2): each
// brings its own 128 rows of W and half the rows of x, 26 bytes a kiloflop instead of the 36 of a
// CTA by itself.  The accumulator is double, so that a tile's products run under the epilogue of
// the last one; what is left of tensor memory holds z = v B_a^T.
//
// z: rows of a tile that lie together and share an adapter are a run.  A run has columns of its own
// (its rows, up to a multiple of 32), so its product meets no other adapter's rows, and what the
// columns behind it hold is not read.  v comes as bf16 parts (two for bf16 outputs, all three for
// f32 ones).  Entries of B behind the adapter's rank are overwritten with zeros in shared memory
// before the product reads them.  Runs that find no room are added on the CUDA cores in the
// epilogue.
//
// Warps: 0-3 epilogue, 4 copies, 5 products (of the pair's first CTA), 6 notes (each row's
// adapter, runs and their columns, a tile ahead), 7 the zeros behind the ranks.
#include <map>
#include <tuple>

#include "project_parts.cuh"

namespace tts {
namespace {

constexpr int kMaxNb = 160;
constexpr int kMaxRuns = 16;
constexpr int kThreads = 256;
constexpr int kEpi = 128;
constexpr int kMaxStages = 8;
constexpr int kTmemCols = 512;
constexpr int kWChunk = kM * kRowBytes;
constexpr int kRing = 16;             // 16-byte pieces of B a thread of the epilogue has room for
constexpr int kMaxAhead = 8;

struct ManyPlan {
  int nb;                   // rows of x a tile, a multiple of 32
  int ch, stages;
  int n_rt, n_nt, n_tiles;
  int n_chunks, flat;
  int parts;                // 0: no adapters
  int v_off, b_off, z_off, bar_off, smem;
};

struct Notes {
  int ad[kMaxNb];           // -1 none, -2 no request
  int rank[kMaxNb];
  int zcol[kMaxNb];         // the row's column of z, -1 none
  float sx[kMaxNb];
  int run_ad[kMaxRuns], run_rank[kMaxRuns], run_first[kMaxRuns], run_n[kMaxRuns], run_col[kMaxRuns];
  int n_runs;
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
__device__ __forceinline__ bool warp_wait_cluster(uint64_t* bar, uint32_t parity) {
  return __all_sync(kFull, mbar_wait_cluster(bar, parity, kWaitLimitCycles));
}
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, float& v) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  v = __uint_as_float(r);
}
__device__ __forceinline__ void cp_async_wait(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    case 7: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 8;" ::: "memory"); break;
  }
}

// z of the rows `todo` of a chunk of 32 on the CUDA cores, into s_z[row][thread]: thread m streams
// its row of each B_a through a ring of 16-byte pieces.
__device__ __noinline__ void z_on_cuda_cores(const ProjectParams& p, const Notes& note, int c, int r0, int n, uint32_t todo,
                                             float* s_v, unsigned char* s_b, float* s_z) {
  const int tid = threadIdx.x, rm = p.ad.rank_max;
  named_barrier(1, kEpi);   // the last chunk's rows of v have been read
  for (int i = tid; i < 32 * rm / 4; i += kEpi) {
    const int t = i / (rm / 4), r = r0 + c * 32 + t;
    if (todo >> t & 1u) cp_async16(s_v + i * 4, p.v + static_cast<int64_t>(r) * rm + (i - t * (rm / 4)) * 4);
  }
  cp_async_commit();
  uint32_t next = todo;
  int ahead = 0, put = 0, room = kRing, get = 0;
  auto ask = [&](int done) {
    while (next != 0 && ahead - done < kMaxAhead) {
      const int t = c * 32 + __ffs(static_cast<int>(next)) - 1, have = (note.rank[t] + 7) / 8;
      if (have > room) break;
      if (n < p.n) {
        const unsigned char* src = static_cast<const unsigned char*>(p.ad.b) + (static_cast<int64_t>(note.ad[t]) * p.n + n) * rm * 2;
        for (int v = 0, at = put; v < have; ++v) {
          cp_async16(s_b + (at * kEpi + tid) * 16, src + v * 16);
          at = at + 1 == kRing ? 0 : at + 1;
        }
      }
      cp_async_commit();
      put = put + have >= kRing ? put + have - kRing : put + have;
      room -= have;
      ++ahead;
      next &= next - 1;
    }
  };
  ask(0);
  cp_async_wait(ahead);     // v
  named_barrier(1, kEpi);
  int k = 0;
  for (uint32_t left = todo; left != 0; left &= left - 1, ++k) {
    const int j = __ffs(static_cast<int>(left)) - 1, rank = note.rank[c * 32 + j], have = (rank + 7) / 8;
    cp_async_wait(ahead - k - 1);
    const float* vt = s_v + j * rm;
    float2 z = make_float2(0.f, 0.f), y = z;
    for (int e = 0, at = get; e < have; ++e) {
      float2 bp[4], v0, v1, v2, v3;
      b_pairs(lds128(s_b + (at * kEpi + tid) * 16), rank - 8 * e, bp);
      at = at + 1 == kRing ? 0 : at + 1;
      v_pairs(vt + e * 8, v0, v1);
      v_pairs(vt + e * 8 + 4, v2, v3);
      z = __ffma2_rn(v0, bp[0], z);
      y = __ffma2_rn(v1, bp[1], y);
      z = __ffma2_rn(v2, bp[2], z);
      y = __ffma2_rn(v3, bp[3], y);
    }
    s_z[j * kEpi + tid] = (z.x + z.y) + (y.x + y.y);
    get = get + have >= kRing ? get + have - kRing : get + have;
    room += have;
    ask(k + 1);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
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
  const int stage_bytes = q.ch * (kWChunk + x_chunk);
  float* s_v = reinterpret_cast<float*>(smem + q.v_off);
  unsigned char* s_b = smem + q.b_off;
  float* s_z = reinterpret_cast<float*>(smem + q.z_off);          // [32][128]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + q.bar_off);  // (the first CTA's)
  uint64_t* zl = full + kMaxStages;                                // B and v parts have landed here
  uint64_t* empty = zl + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + 2;                              // (the first CTA's)
  uint64_t* note_full = acc_empty + 2;
  uint64_t* note_empty = note_full + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(note_empty + 2);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  const int nst = (q.n_chunks + q.ch - 1) / q.ch;

  if (tid == 0) {
    for (int i = 0; i < q.stages; ++i) {
      mbar_init(&full[i], 2);
      mbar_init(&zl[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 8);
      mbar_init(&note_full[i], 1);
      mbar_init(&note_empty[i], q.parts > 0 ? 7 : 4);   // epilogue 4; copies, products, zeros
    }
    mbar_init_fence();
  }
  if (warp == 5) {
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

  if (warp == 4) {
    // ------------------------------------------------------------------ copies
    const int cols = kRowBytes / (E4M3 ? 1 : 2);
    bool ok = true;
    int it = 0, i = 0;
    auto next_stage = [&]() {
      const int s = it % q.stages;
      return it < q.stages || warp_wait(&empty[s], static_cast<uint32_t>(it / q.stages - 1) & 1u);
    };
    for (int tile = pair; tile < q.n_tiles && ok; tile += pairs, ++i) {
      const int rt = tile % q.n_rt, nt = tile / q.n_rt;
      const int w0 = nt * 2 * kM + rank * kM, x0 = rt * q.nb + rank * half;
      for (int st = 0; st < nst; ++st, ++it) {
        ok = next_stage();
        if (!ok) break;
        if (lane == 0) {
          const int s = it % q.stages;
          unsigned char* w = smem + s * stage_bytes;
          unsigned char* x = w + q.ch * kWChunk;
          const uint32_t bar = map_shared_rank(&full[s], 0);
          // the first CTA's barrier counts the bytes of both
          if (rank == 0) mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(2 * stage_bytes));
          else mbar_arrive_remote(bar);
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
      if (q.parts == 0 || !ok) continue;
      if (i == 0) grid_wait();   // v's parts
      ok = note_wait(i);
      const Notes& note = s_note[i & 1];
      const int runs = ok ? note.n_runs : 0;
      for (int k = 0; k < runs && ok; ++k)
        for (int j = 0; j < note.run_rank[k] && ok; j += 64)
          for (int h = 0; h < q.parts; ++h, ++it) {
            ok = next_stage();
            if (!ok) break;
            if (lane == 0) {
              const int s = it % q.stages, n2 = note.run_n[k] / 2;
              unsigned char* w = smem + s * stage_bytes;
              unsigned char* x = w + q.ch * kWChunk;
              mbar_arrive_expect_tx(&zl[s], static_cast<uint32_t>(kWChunk + n2 * kRowBytes));
              tma_load(w, &bmap, j, note.run_ad[k] * p.n + w0, 0, &zl[s]);
              for (int t = 0; t < n2; t += 16)
                tma_load(x + t * kRowBytes, &vmap, j, rt * q.nb + note.run_first[k] + rank * n2 + t, h, &zl[s]);
            }
            __syncwarp();
          }
      note_done(i);
    }
    if (!ok && lane == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
    // no copy may still be landing, and no product reading, when the CTA leaves
    for (int t = max(0, it - q.stages); t < it; ++t) warp_wait(&empty[t % q.stages], static_cast<uint32_t>(t / q.stages) & 1u);
  } else if (warp == 5) {
    // ---------------------------------------------------------------- products
    bool ok = true;
    int it = 0, i = 0;
    const uint32_t idesc = (1u << 4) | (E4M3 ? 0u : (1u << 7) | (1u << 10)) | (static_cast<uint32_t>(q.nb >> 3) << 17) |
                           (static_cast<uint32_t>(2 * kM >> 4) << 24);
    for (int tile = pair; tile < q.n_tiles && ok; tile += pairs, ++i) {
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
      for (int st = 0; st < nst; ++st, ++it) {
        const int s = it % q.stages;
        if (!warp_wait_cluster(&full[s], static_cast<uint32_t>(it / q.stages) & 1u)) {
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
      if (q.parts > 0 && ok) {
        ok = note_wait(i);
        // the last tile's z has to be read first
        if (i > 0 && !warp_wait_cluster(&acc_empty[(i - 1) & 1], static_cast<uint32_t>((i - 1) / 2) & 1u)) ok = false;
        tc_fence_after();
        const Notes& note = s_note[buf];
        const int runs = ok ? note.n_runs : 0;
        for (int k = 0; k < runs && ok; ++k) {
          const uint32_t zi = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(note.run_n[k] >> 3) << 17) |
                              (static_cast<uint32_t>(2 * kM >> 4) << 24);
          const int ranks = note.run_rank[k];
          const uint32_t zd = tmem + zbase + static_cast<uint32_t>(note.run_col[k]);
          for (int j = 0; j < ranks && ok; j += 64)
            for (int h = 0; h < q.parts; ++h, ++it) {
              const int s = it % q.stages;
              if (!warp_wait_cluster(&full[s], static_cast<uint32_t>(it / q.stages) & 1u)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t w = smem_u32(smem + s * stage_bytes);
              const uint64_t ad = smem_desc(w), bd = smem_desc(w + static_cast<uint32_t>(q.ch * kWChunk));
              const int steps = (min(64, ranks - j) + 15) / 16;
              for (int e = 0; e < steps; ++e) mma2<false>(zd, ad + 2 * e, bd + 2 * e, zi, j > 0 || h > 0 || e > 0);
              commit2(&empty[s]);
            }
        }
        note_done(i);
      }
      commit2(&acc_full[buf]);
    }
    if (!ok && lane == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
  } else if (warp == 6) {
    // ------------------------------------------------------------------- notes
    bool ok = true;
    int i = 0;
    constexpr int kC = kMaxNb / 32;
    const int zcols = kTmemCols - 2 * q.nb;
    for (int tile = pair; tile < q.n_tiles && ok; tile += pairs, ++i) {
      if (i > 1 && !warp_wait(&note_empty[i & 1], static_cast<uint32_t>(i / 2 - 1) & 1u)) {
        ok = false;
        break;
      }
      Notes& note = s_note[i & 1];
      const int r0 = (tile % q.n_rt) * q.nb;
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
        ad[c] = ad[c] < 0 ? -2 : p.ad.n_adapters == 0 || ad[c] >= p.n_streams ? -1 : __ldcg(p.stream_adapter + ad[c]);
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        if (ad[c] >= p.ad.n_adapters || ad[c] == -1 || ad[c] < -2) ad[c] = -1;
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
      if (lane == 0) note.n_runs = n_runs;
      __syncwarp();
      if (lane == 0) mbar_arrive(&note_full[i & 1]);
    }
    if (!ok && lane == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
  } else if (warp == 7) {
    // ------------------------------------------------- zeros behind the ranks
    bool ok = true;
    int it = 0, i = 0;
    uint32_t phase = 0;   // of each stage's zl
    if (q.parts > 0)
      for (int tile = pair; tile < q.n_tiles && ok; tile += pairs, ++i) {
        it += nst;
        ok = note_wait(i);
        const Notes& note = s_note[i & 1];
        const int runs = ok ? note.n_runs : 0;
        for (int k = 0; k < runs && ok; ++k) {
          const int ranks = note.run_rank[k];
          for (int j = 0; j < ranks && ok; j += 64)
            for (int h = 0; h < q.parts; ++h, ++it) {
              const int s = it % q.stages;
              if (!warp_wait(&zl[s], phase >> s & 1u)) {
                ok = false;
                break;
              }
              phase ^= 1u << s;
              const int left = min(64, ranks - j);
              if (left % 16 != 0) {
                unsigned char* b = smem + s * stage_bytes;
                for (int m = lane; m < kM; m += 32)
                  for (int e = left; e < ((left + 15) & ~15); ++e)
                    *reinterpret_cast<uint16_t*>(b + m * kRowBytes + (((e >> 3) ^ (m & 7)) << 4) + (e & 7) * 2) = 0;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              }
              __syncwarp();
              if (lane == 0) mbar_arrive_remote(map_shared_rank(&full[s], 0));
            }
        }
        note_done(i);
      }
    if (!ok && lane == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
  } else {
    // ---------------------------------------------------------------- epilogue
    grid_wait();
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    bool ok = true;
    int i = 0;
    for (int tile = pair; tile < q.n_tiles && ok; tile += pairs, ++i) {
      const int rt = tile % q.n_rt, nt = tile / q.n_rt, r0 = rt * q.nb, buf = i & 1;
      const int n = nt * 2 * kM + rank * kM + tid;
      const float sw = E4M3 && n < p.n ? __ldcg(p.w_scale + n) : 0.f;
      ok = mbar_wait(&note_full[buf], static_cast<uint32_t>(i >> 1) & 1u);
      ok = mbar_wait(&acc_full[buf], static_cast<uint32_t>(i >> 1) & 1u) && ok;
      ok = epilogue_all(ok);
      if (!ok) {
        if (tid == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
        break;
      }
      tc_fence_after();
      const Notes& note = s_note[buf];
      const uint32_t dcol = tmem + static_cast<uint32_t>(buf * q.nb) + lane_off;
      for (int c = 0; c < q.nb / 32; ++c) {
        float acc[32];
        tmem_ld32(dcol + c * 32, acc);
        const int a = note.ad[c * 32 + lane], zc = note.zcol[c * 32 + lane];
        const uint32_t live = __ballot_sync(kFull, a != -2);
        const uint32_t on_tc = __ballot_sync(kFull, zc >= 0), on_cc = __ballot_sync(kFull, a >= 0 && zc < 0 && q.parts > 0);
        if (E4M3) {
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[j] *= note.sx[c * 32 + j] * sw;
        }
        if (on_tc != 0) {
          // one run: its columns lie together
          const int f = __ffs(static_cast<int>(on_tc)) - 1, base = __shfl_sync(kFull, zc, f) - f;
          const bool one = __all_sync(kFull, zc < 0 || zc - lane == base) && static_cast<int>(zbase) + base + 32 <= kTmemCols;
          if (one) {
            float z[32];
            tmem_ld32(tmem + static_cast<uint32_t>(static_cast<int>(zbase) + base) + lane_off, z);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (on_tc >> j & 1u) acc[j] += z[j];
          } else {
            for (uint32_t left = on_tc; left != 0; left &= left - 1) {
              const int j = __ffs(static_cast<int>(left)) - 1;
              float z;
              tmem_ld1(tmem + zbase + static_cast<uint32_t>(__shfl_sync(kFull, zc, j)) + lane_off, z);
              s_z[j * kEpi + tid] = z;
            }
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (on_tc >> j & 1u) acc[j] += s_z[j * kEpi + tid];
          }
        }
        if (on_cc != 0) {
          z_on_cuda_cores(p, note, c, r0, n, on_cc, s_v, s_b, s_z);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (on_cc >> j & 1u) acc[j] += s_z[j * kEpi + tid];
        }
        if (n < p.n) {
          const int64_t at = static_cast<int64_t>(r0 + c * 32) * p.out_stride + n;
          if (p.out_bf16) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (live >> j & 1u) static_cast<__nv_bfloat16*>(p.out)[at + j * p.out_stride] = __float2bfloat16_rn(acc[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (live >> j & 1u) static_cast<float*>(p.out)[at + j * p.out_stride] = acc[j];
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_remote(map_shared_rank(&acc_empty[buf], 0));
        mbar_arrive(&note_empty[buf]);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  // no CTA leaves while the other may still signal it, read its operands or land in its memory
  cluster_sync_all();
  if (warp == 5) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
  }
}

constexpr int kBars = (3 * kMaxStages + 8) * 8 + 16;

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
  q.n_rt = (p.rows + kMaxNb - 1) / kMaxNb;
  q.nb = ((p.rows + q.n_rt - 1) / q.n_rt + 31) / 32 * 32;
  q.n_rt = (p.rows + q.nb - 1) / q.nb;
  q.n_tiles = q.n_nt * q.n_rt;
  q.parts = rm == 0 ? 0 : p.out_bf16 ? 2 : 3;
  const int v = 32 * rm * 4, b = rm > 0 ? kRing * kEpi * 16 : 0, z = rm > 0 ? 32 * kEpi * 4 : 0;
  const int left = static_cast<int>(budget) - 1024 - v - b - z - kBars;
  // larger copies stream faster: two columns of K a stage where three such stages fit
  for (q.ch = 2; q.ch >= 1; --q.ch) {
    const int stage = q.ch * (kWChunk + q.nb / 2 * kRowBytes);
    q.stages = left / stage > kMaxStages ? kMaxStages : left / stage;
    q.v_off = q.stages * stage;
    if (q.stages >= 3) break;
  }
  if (q.ch < 1) return cudaErrorInvalidConfiguration;
  q.b_off = q.v_off + v;
  q.z_off = q.b_off + b;
  q.bar_off = q.z_off + z;
  q.smem = 1024 + q.bar_off + kBars;
  CUtensorMap wmap, xmap, bmap, vmap;
  if (!encode(&wmap, p.w, es, p.k, p.k, p.n, kM, q.ch, q.flat) ||
      !encode(&xmap, p.x, es, p.x_stride, p.k, p.rows, q.nb / 2, q.ch, q.flat))
    return cudaErrorInvalidValue;
  bmap = vmap = wmap;
  if (q.parts > 0 && (!encode(&bmap, p.ad.b, 2, rm, rm, p.ad.n_adapters * p.n, kM, 1, true) ||
                      !encode(&vmap, p.v_parts, 2, rm, rm, p.rows, 16, 1, true, 0, 3)))
    return cudaErrorInvalidValue;
  if (rm > 0) {
    e = launch_shrink(p, s);
    if (e != cudaSuccess) return e;
  }
  const int grid = 2 * (q.n_tiles < n_pairs ? q.n_tiles : n_pairs);
  return launch_pairs(project_many_kernel<E4M3>, grid, kThreads, q.smem, s, wmap, xmap, bmap, vmap, p, q);
}

}  // namespace

// Whether the pairs' tiles fill the device: fewer leave SMs idle, which smaller tiles split over K
// do not.
bool project_is_many(int rows, int n) {
  const int64_t tiles = static_cast<int64_t>((n + 2 * kM - 1) / (2 * kM)) * ((rows + kMaxNb - 1) / kMaxNb);
  return rows > kMaxNb && tiles >= sm_count() / 2;
}

cudaError_t launch_project_many(const ProjectParams& p, cudaStream_t s) {
  return p.x_e4m3 ? launch_t<true>(p, s) : launch_t<false>(p, s);
}

}  // namespace tts
