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
//   * the epilogue's warps take z = v B_a^T on the CUDA cores, in f32, while the tensor cores work: a
//     group of four warps covers the 128 columns; a warp loads 32 rows of a B_a into registers while it
//     works on the last ones, and lays them out in shared memory; v comes by one bulk copy, and z waits
//     in tensor memory beside the accumulator.  So x A^T is never rounded, a request's adapter never
//     meets another request's row, and what lies behind an adapter's rank is not used.  (Asynchronous
//     copies to shared memory took a wavefront a lane, however the lanes shared the rows, 16 bytes a
//     clock; TMA boxes of 32 rows no less: 35 us of the 57 that 96 requests with adapters of up to 64
//     ranks, 12288 columns, took either way.)  A group has about four rows, as far as four groups go.
#include <map>
#include <tuple>

#include "project_parts.cuh"
#include "project_plan.h"

namespace tts {
namespace {

constexpr int kTmemCols = 512;

// Neighbouring blocks of 16 rows that share an adapter.
struct BlockRun {
  int ad, first, count;   // blocks [first, first + count) of the tile
};
// The next run of blocks from `at` on with one adapter; lane b of the warp holds block b's adapter
// (negative: none, or several).  Converged warp; false when there is none.
__device__ __forceinline__ bool next_run(int mine, int blocks, int at, BlockRun& run) {
  const int lane = threadIdx.x & 31;
  const uint32_t some = __ballot_sync(kFull, mine >= 0 && lane >= at && lane < blocks);
  if (some == 0) return false;
  run.first = __ffs(static_cast<int>(some)) - 1;
  run.ad = __shfl_sync(kFull, mine, run.first);
  const uint32_t other = __ballot_sync(kFull, (mine != run.ad || lane >= blocks) && lane > run.first);
  run.count = (other != 0 ? __ffs(static_cast<int>(other)) - 1 : 32) - run.first;
  return true;
}

struct TileInfo {
  int ad[256];       // adapter of the tile's rows: -1 none, -2 no request
  int rank[256];
  float sx[256];
  bool one[256];     // the row's block of 16 shares one adapter
};

// Block `lane` of a tile: the adapter its rows share, negative for none, several or no such block.
__device__ __forceinline__ int tile_block(const ProjectParams& p, const Plan& q, int rt, int lane) {
  const int r = rt * q.nb + lane * 16;
  return lane < q.nb / 16 && r < p.rows ? __ldcg(p.block_ad + r / 16) : -1;
}

template <bool E4M3, bool WIDE>
__global__ void __launch_bounds__(max_threads(WIDE), 1) project_kernel(const __grid_constant__ CUtensorMap wmap,
                                                              const __grid_constant__ CUtensorMap xmap,
                                                              const __grid_constant__ CUtensorMap bmap,
                                                              const __grid_constant__ CUtensorMap vmap,
                                                              const ProjectParams p, const Plan q) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ TileInfo s_tile;
  const int stage_bytes = q.ch * (kWChunk + q.nb * kRowBytes);
  float* s_v = reinterpret_cast<float*>(smem + q.v_off);          // [v_rows][rank_max]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + q.bar_off);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* v_full = acc_empty + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(v_full + 1);
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
      mbar_init(&acc_empty[i], 4 * q.groups);
    }
    mbar_init(v_full, 1);
    mbar_init_fence();
  }
  const int copy_warp = 4 * q.groups, mma_warp = copy_warp + 1;
  if (warp == mma_warp) {
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

  if (warp == copy_warp) {
    // ------------------------------------------------------------------ copies
    const int cols = kRowBytes / (E4M3 ? 1 : 2);
    bool ok = true, waited = false;
    int it = 0;
    // a free stage, once its last products have read it
    auto next_stage = [&]() {
      const int s = it % q.stages;
      return it < q.stages || warp_wait(&empty[s], static_cast<uint32_t>(it / q.stages - 1) & 1u);
    };
    for (int tile = blockIdx.x; tile < q.n_tiles && ok; tile += gridDim.x) {
      const int rt = tile % q.n_rt, nt = tile / q.n_rt;
      for (int i = 0; i < nst; ++i, ++it) {
        ok = next_stage();
        if (!ok) break;
        if (lane == 0) {
          const int s = it % q.stages;
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
        __syncwarp();
      }
      if (q.parts == 0 || rank != 0 || !ok) continue;
      // B rows and parts of v for blocks that share an adapter, 64 ranks a stage
      if (!waited) grid_wait();
      waited = true;
      const int mine = tile_block(p, q, rt, lane);
      BlockRun run;
      for (int at = 0; ok && next_run(mine, q.nb / 16, at, run); at = run.first + run.count) {
        int bad = 0;
        const int ranks = adapter_rank(p, run.ad, &bad);
        for (int j = 0; j < ranks && ok; j += 64)
          for (int h = 0; h < q.parts; ++h, ++it) {
            ok = next_stage();
            if (!ok) break;
            if (lane == 0) {
              const int s = it % q.stages;
              unsigned char* w = smem + s * stage_bytes;
              mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(kWChunk + q.nb * kRowBytes));
              tma_load(w, &bmap, j, run.ad * p.n + nt * kM, 0, &full[s]);
              tma_load(w + q.ch * kWChunk, &vmap, j, rt * q.nb, h, &full[s]);
            }
            __syncwarp();
          }
      }
    }
    if (!ok && lane == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
    // no copy may still be landing when the CTA leaves
    for (int t = max(0, it - q.stages); t < it; ++t) warp_wait(&full[t % q.stages], static_cast<uint32_t>(t / q.stages) & 1u);
    __syncwarp();
  } else if (warp == mma_warp) {
    // ---------------------------------------------------------------- products
    // f32 accumulator (bits 4-5 = 1); bf16 operands are 1 at bits 7-9 and 10-12, e4m3 ones 0;
    // both K-major; N >> 3 at bit 17, M >> 4 at bit 24
    const uint32_t idesc = (1u << 4) | (E4M3 ? 0u : (1u << 7) | (1u << 10)) | (static_cast<uint32_t>(q.nb >> 3) << 17) |
                           (static_cast<uint32_t>(kM >> 4) << 24);
    bool ok = true, waited = false;
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
      if (q.parts > 0 && rank == 0 && ok) {
        // z of blocks that share an adapter, beside the accumulators; the last tile's z has to be
        // read first
        if (!waited) grid_wait();
        waited = true;
        if (i > 0 && !warp_wait(&acc_empty[(i - 1) % q.n_acc], static_cast<uint32_t>((i - 1) / q.n_acc) & 1u)) ok = false;
        tc_fence_after();
        const int mine = tile_block(p, q, tile % q.n_rt, lane);
        const uint32_t zd = tmem + static_cast<uint32_t>(q.n_acc * q.nbr);
        BlockRun run;
        for (int at = 0; ok && next_run(mine, q.nb / 16, at, run); at = run.first + run.count) {
          int bad = 0;
          const int ranks = adapter_rank(p, run.ad, &bad);
          const uint32_t zi = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(run.count * 2) << 17) |
                              (static_cast<uint32_t>(kM >> 4) << 24);
          for (int j = 0; j < ranks && ok; j += 64)
            for (int h = 0; h < q.parts; ++h, ++it) {
              const int s = it % q.stages;
              if (!warp_wait(&full[s], static_cast<uint32_t>(it / q.stages) & 1u)) {
                ok = false;
                break;
              }
              unsigned char* b = smem + s * stage_bytes;
              const int left = min(64, ranks - j);
              if (left % 16 != 0) {
                // what lies behind the rank is not this adapter's: zeros up to the instruction's 16
                for (int m = lane; m < kM; m += 32)
                  for (int e = left; e < ((left + 15) & ~15); ++e)
                    *reinterpret_cast<uint16_t*>(b + m * kRowBytes + (((e >> 3) ^ (m & 7)) << 4) + (e & 7) * 2) = 0;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
              }
              tc_fence_after();
              const uint64_t ad = smem_desc(smem_u32(b));
              const uint64_t bd = smem_desc(smem_u32(b) + q.ch * kWChunk + run.first * 16 * kRowBytes);
              for (int k = 0; k < (left + 15) / 16; ++k)
                mma<false>(zd + run.first * 16, ad + 2 * k, bd + 2 * k, zi, j > 0 || h > 0 || k > 0);
              mma_commit(&empty[s]);
            }
        }
      }
      mma_commit(&acc_full[buf]);
    }
    if (!ok && lane == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
  } else {
    // ---------------------------------------------------------------- epilogue
    const int group = warp >> 2, quad = warp & 3, n_epi = 128 * q.groups;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t zcol = tmem + static_cast<uint32_t>(q.n_acc * q.nbr) + lane_off;
    const int m = quad * 32 + lane, rm = p.ad.rank_max;
    const bool with = p.ad.n_adapters > 0;
    const int lo = q.nb * rank / S, hi = q.nb * (rank + 1) / S;   // rows whose adapters this CTA adds,
    const int glo = lo + (hi - lo) * group / q.groups, ghi = lo + (hi - lo) * (group + 1) / q.groups;   // and this group
    const uint32_t s_b = smem_u32(smem + q.b_off) + warp * (q.pieces * 512);   // this warp's 32 rows of B, piece by piece
    bool ok = true, waited = !with;
    int i = 0;
    for (int tile = blockIdx.x; tile < q.n_tiles && ok; tile += gridDim.x, ++i) {
      const int rt = tile % q.n_rt, nt = tile / q.n_rt, r0 = rt * q.nb;
      const int n = nt * kM + m;
      for (int t = tid; t < q.nbr; t += n_epi) {
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
      epilogue_all(true, n_epi);
      if (q.parts > 0) {
        // blocks that share an adapter are the tensor cores'
        for (int c = warp; c < q.nbr / 32; c += 4 * q.groups) {
          const int a = s_tile.ad[c * 32 + lane];
          int top = a, low = a >= 0 ? a : 0x7fffffff;
#pragma unroll
          for (int o = 8; o >= 1; o >>= 1) {
            top = max(top, __shfl_xor_sync(kFull, top, o));
            low = min(low, __shfl_xor_sync(kFull, low, o));
          }
          s_tile.one[c * 32 + lane] = top >= 0 && top == low;
        }
        epilogue_all(true, n_epi);
      }
      if (with) {
        const unsigned char* brow = static_cast<const unsigned char*>(p.ad.b) + static_cast<int64_t>(n - lane) * rm * 2;
        const int rows_in = min(32, p.n - (n - lane));   // of this warp's 32
        const uint32_t pool_step = static_cast<uint32_t>(p.n) * rm * 2;   // (at most 2^28)
        bool v_here = false;
        for (int base = glo; base < ghi; base += 32) {
          // runs of rows that share an adapter
          const int t = base + lane;
          const int a = t < ghi && !(q.parts > 0 && s_tile.one[t]) ? max(s_tile.ad[t], -1) : -1;
          const int k = a >= 0 ? s_tile.rank[t] : 0, prev = __shfl_up_sync(kFull, a, 1);
          const uint32_t edge = __ballot_sync(kFull, lane == 0 || a != prev);
          const uint32_t first = __ballot_sync(kFull, a >= 0 && (lane == 0 || a != prev));
          // A run's B rows, into registers: neighbouring lanes take neighbouring pieces of a row.  Piece e
          // of row l then lies at place l ^ (e & mix) of the piece's 512 bytes, so that neither a row's
          // pieces as they are stored nor the rows' as they are read meet in a bank.
          constexpr int kPieces = WIDE ? 16 : 8;
          uint4 w[kPieces];
          auto shift_of = [](int have) { return have > 8 ? 4 : have > 4 ? 3 : have > 2 ? 2 : have - 1; };
          auto ask_b = [&](int l) {
            const int of = __shfl_sync(kFull, a, l), have = (__shfl_sync(kFull, k, l) + 7) >> 3;
            const int sh = shift_of(have), step = 32 >> sh, e = lane & ((1 << sh) - 1), row = lane >> sh;
            const unsigned char* src = brow + static_cast<uint64_t>(static_cast<uint32_t>(of)) * pool_step + row * rm * 2 + e * 16;
#pragma unroll
            for (int c = 0; c < kPieces; ++c)
              if (c < 1 << sh && e < have && row + c * step < rows_in)
                w[c] = __ldcg(reinterpret_cast<const uint4*>(src + c * step * rm * 2));
          };
          if (first != 0) ask_b(__ffs(static_cast<int>(first)) - 1);
          if (!waited) {
            grid_wait();   // v, and whoever read or wrote out before
            waited = true;
          }
          if (!v_here) {
            if (tid == 0) {
              const int cnt = min(hi, p.rows - r0) - lo;
              if (cnt > 0) {
                mbar_arrive_expect_tx(v_full, static_cast<uint32_t>(cnt * rm) * 4u);
                bulk_g2s_plain(s_v, p.v + static_cast<int64_t>(r0 + lo) * rm, static_cast<uint32_t>(cnt * rm) * 4u, v_full);
              } else {
                mbar_arrive(v_full);
              }
            }
            ok = mbar_wait(v_full, static_cast<uint32_t>(i) & 1u) && ok;
            v_here = true;
          }
          for (uint32_t left = first; left != 0; left &= left - 1) {
            const int l = __ffs(static_cast<int>(left)) - 1, ranks = __shfl_sync(kFull, k, l), have = (ranks + 7) >> 3;
            const uint32_t later = edge >> l >> 1;
            const int end = base + (later != 0 ? l + __ffs(static_cast<int>(later)) : 32);
            const int sh = shift_of(have), step = 32 >> sh, mix = min(7, step - 1);
            __syncwarp();   // (the last run has been read)
            {
              const int e = lane & ((1 << sh) - 1), row = lane >> sh;
              const uint32_t dst = s_b + e * 512 + ((row ^ (e & mix)) << 4);
#pragma unroll
              for (int c = 0; c < kPieces; ++c)
                if (c < 1 << sh && e < have) sts16(dst + c * step * 16, w[c]);
            }
            __syncwarp();
            if (left & (left - 1)) ask_b(__ffs(static_cast<int>(left & (left - 1))) - 1);
            const uint32_t b = s_b;
            if (ranks & 7) {
              // zeros behind the rank, where v's are
              const uint32_t tail = b + (have - 1) * 512 + ((lane ^ ((have - 1) & mix)) << 4);
              const uint4 w = lds16(tail);
              const int keep = ranks & 7;
              const uint32_t odd = keep & 1 ? 0xffffu : 0u;   // of the word in which the rank ends
              sts16(tail, make_uint4(keep > 1 ? w.x : w.x & odd, keep > 3 ? w.y : keep > 1 ? w.y & odd : 0u,
                                     keep > 5 ? w.z : keep > 3 ? w.z & odd : 0u, keep > 5 ? w.w & odd : 0u));
            }
            for (int t = base + l; t < end; ++t) {
              float2 z = make_float2(0.f, 0.f), y = z;
              const uint32_t vt = smem_u32(s_v) + (t - lo) * rm * 4;
#pragma unroll 4
              for (int e = 0; e < have; ++e) {
                float2 va, vb, vc, vd;
                const uint4 w = lds16(b + e * 512 + ((lane ^ (e & mix)) << 4));
                v_pairs(vt + e * 32, va, vb);
                v_pairs(vt + e * 32 + 16, vc, vd);
                z = __ffma2_rn(va, bf16_pair_f32(w.x), z);
                y = __ffma2_rn(vb, bf16_pair_f32(w.y), y);
                z = __ffma2_rn(vc, bf16_pair_f32(w.z), z);
                y = __ffma2_rn(vd, bf16_pair_f32(w.w), y);
              }
              tmem_st1(zcol + static_cast<uint32_t>(t), (z.x + z.y) + (y.x + y.y));
            }
          }
        }
        if (!waited) grid_wait();
        waited = true;
        if (!v_here && tid == 0) mbar_arrive(v_full);   // (no row here has an adapter: the phase is used all the same)
        tmem_wait_st();
        tc_fence_before();
      }
      // ---- the accumulator
      const int buf = i % q.n_acc, use = i / q.n_acc;
      ok = mbar_wait(&acc_full[buf], static_cast<uint32_t>(use) & 1u) && ok;
      ok = epilogue_all(ok, n_epi);
      if (!ok) {
        if (tid == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
        break;
      }
      tc_fence_after();
      const uint32_t dcol = tmem + static_cast<uint32_t>(buf * q.nbr) + lane_off;
      const float sw = E4M3 && n < p.n ? __ldcg(p.w_scale + n) : 0.f;
      for (int c = group; c < q.nbr / 16; c += q.groups) {
        float acc[16], z[16];
        tmem_ld16(dcol + c * 16, acc);
        const int t = c * 16 + (lane & 15), a = s_tile.ad[t];
        const uint32_t live = __ballot_sync(kFull, a != -2);
        // (z of a block that shares an adapter is with the cluster's first CTA)
        const bool one = q.parts > 0 && s_tile.one[t];
        const uint32_t has = __ballot_sync(kFull, a >= 0 && (one ? rank == 0 : t >= lo && t < hi));
        if (has != 0) tmem_ld16(zcol + c * 16, z);
        if (E4M3) {
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[j] *= s_tile.sx[c * 16 + j] * sw;
        }
        if (has != 0) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (has >> j & 1u) acc[j] += z[j];
        }
        if (S == 1) {
          if (n < p.n) {
            const int64_t at = static_cast<int64_t>(r0 + c * 16) * p.out_stride + n;
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (live >> j & 1u) store_out(p, at + j * p.out_stride, acc[j]);
          }
        } else if (c * 16 < q.nb) {
          // (every MMA of this CTA has read the ring)
#pragma unroll
          for (int j = 0; j < 16; ++j) red[(c * 16 + j) * kRedLd + m] = acc[j];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[buf]);
      epilogue_all(true, n_epi);   // the tile's notes and v may change
    }
  }
  if (S > 1) {
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();   // every CTA's partial is in its shared memory
    if (warp < copy_warp) {
      const int rt = static_cast<int>(blockIdx.x) % q.n_rt, nt = static_cast<int>(blockIdx.x) / q.n_rt;
      const int lo = q.nb * rank / S, hi = q.nb * (rank + 1) / S;
      uint32_t peer[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) peer[r] = r < S ? map_shared_rank(red, r) : 0u;
      const int n = nt * kM + lane * 4;
      for (int t = lo + warp; t < hi; t += copy_warp) {
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
  if (warp == mma_warp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
  }
}

// The dynamic shared memory a CTA of the kernel may take on device `dev`, set as its limit once
// per device; 0 on failure.
template <bool E4M3, bool WIDE>
size_t configure(int dev) {
  static std::mutex mtx;
  static size_t budget[64] = {};
  std::lock_guard<std::mutex> lock(mtx);
  if (budget[dev] != 0) return budget[dev];
  int optin = 0;
  cudaFuncAttributes fa;
  if (cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
      cudaFuncGetAttributes(&fa, project_kernel<E4M3, WIDE>) != cudaSuccess || static_cast<size_t>(optin) <= fa.sharedSizeBytes)
    return 0;
  const size_t b = static_cast<size_t>(optin) - fa.sharedSizeBytes;
  if (cudaFuncSetAttribute(project_kernel<E4M3, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(b)) != cudaSuccess)
    return 0;
  budget[dev] = b;
  return b;
}

// Clusters of S CTAs that the device keeps resident at once (cached).
template <bool E4M3, bool WIDE>
int max_active_clusters(int dev, int S, int smem) {
  static std::mutex mtx;
  static std::map<std::tuple<int, int, int>, int> cache;
  const auto key = std::make_tuple(dev, S, smem);
  std::lock_guard<std::mutex> lock(mtx);
  const auto it = cache.find(key);
  if (it != cache.end()) return it->second;
  const int n = active_clusters(project_kernel<E4M3, WIDE>, S, max_threads(WIDE), smem);
  cache[key] = n;
  return n;
}

template <bool E4M3, bool WIDE>
cudaError_t launch_t(const ProjectParams& p, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  const size_t budget = configure<E4M3, WIDE>(dev);
  if (budget == 0) {
    const cudaError_t le = cudaGetLastError();
    return le != cudaSuccess ? le : cudaErrorInvalidValue;
  }
  const int es = E4M3 ? 1 : 2, rm = p.ad.n_adapters > 0 ? p.ad.rank_max : 0, n_sm = sm_count();
  Plan q;
  const bool fits = plan_rows(q, p.rows, p.n, p.k, es, rm, p.tc != 0, budget, n_sm,
                              [&](int split, int smem) { return max_active_clusters<E4M3, WIDE>(dev, split, smem); });
  if (!fits) return cudaErrorInvalidConfiguration;
  const int quantum = p.out_bf16 ? 8 : 16;
  q.vec_out = p.out_stride * (p.out_bf16 ? 2 : 4) % quantum == 0;
  CUtensorMap wmap, xmap, bmap, vmap;
  if (!encode(&wmap, p.w, es, p.k, p.k, p.n, kM, q.ch, q.flat) ||
      !encode(&xmap, p.x, es, p.x_stride, p.k, p.rows, q.nb, q.ch, q.flat))
    return cudaErrorInvalidValue;
  bmap = vmap = wmap;
  if (q.parts > 0 && (!encode(&bmap, p.ad.b, 2, rm, rm, p.ad.n_adapters * p.n, kM, 1, true) ||
                      !encode(&vmap, p.v_parts, 2, rm, rm, p.rows, q.nb, 1, true, 0, 3)))
    return cudaErrorInvalidValue;
  if (rm > 0) {
    e = launch_shrink(p, s);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid = q.split > 1 ? dim3(q.n_tiles, q.split) : dim3(q.n_tiles < n_sm ? q.n_tiles : n_sm);
  return launch_clustered(project_kernel<E4M3, WIDE>, grid, 128 * q.groups + 64, q.smem, q.split, s, wmap, xmap, bmap, vmap, p, q);
}

}  // namespace

// From this many rows on the adapters' products may run on the tensor cores.
bool project_tc(int rows) { return rows >= 128; }

size_t project_workspace(int rows, int rank_max) {
  const size_t v = static_cast<size_t>(rows) * rank_max;
  return project_tc(rows) ? round256(v * 4) + round256(v * 2 * 3) + round256((static_cast<size_t>(rows) + 15) / 16 * 4)
                          : round256(v * 4);
}

cudaError_t launch_project(const ProjectParams& given, void* workspace, cudaStream_t s) {
  ProjectParams p = given;
  // on the tensor cores where requests have eight rows and more
  p.tc = p.ad.n_adapters > 0 && project_tc(p.rows) && p.row_stream != nullptr && p.n_streams <= p.rows / 8;
  if (p.ad.n_adapters > 0) {
    const size_t v = static_cast<size_t>(p.rows) * p.ad.rank_max;
    unsigned char* at = static_cast<unsigned char*>(workspace);
    p.v = reinterpret_cast<float*>(at);
    p.v_parts = reinterpret_cast<__nv_bfloat16*>(at + round256(v * 4));
    p.block_ad = reinterpret_cast<int32_t*>(at + round256(v * 4) + round256(v * 2 * 3));
  }
  if (project_is_many(p)) return launch_project_many(p, s);
  const bool wide = p.ad.n_adapters > 0 && p.ad.rank_max > 64;
  if (p.x_e4m3) return wide ? launch_t<true, true>(p, s) : launch_t<true, false>(p, s);
  return wide ? launch_t<false, true>(p, s) : launch_t<false, false>(p, s);
}

}  // namespace tts
