// How the projection of few rows is cut into tiles, stages and clusters (plain C++: the launch asks
// for it, and a host program can).
#pragma once

#include <cstddef>
#include <cstdint>

#include "project_tile.h"

namespace tts {
namespace {

constexpr int kWChunk = kM * kRowBytes;
constexpr int kMaxStages = 8;
constexpr int kMaxCluster = 8;
// Groups of four epilogue warps; then a warp for copies, one for products.  WIDE: ranks over 64.
constexpr int max_groups(bool wide) { return wide ? 3 : 4; }
constexpr int max_threads(bool wide) { return max_groups(wide) * 128 + 64; }
constexpr int kRedLd = kM + 16;       // floats between the rows of a partial
constexpr int kMaxV = 64 * 1024;      // bytes of v a CTA holds at most
// Shared memory that a CTA asks for at least.  A CTA waits for tensor memory until whoever has it on its
// SM leaves, and then for its cluster at a barrier: two CTAs that so wait for one another, of one cluster
// or of clusters that cross, must not meet on an SM, nor one of no cluster wait there between two that
// are of one.  This is more than half of an SM's, and more than a clustered CTA of gemv_mma.cu leaves (it
// takes 73 KB at least; the other clustered kernels with tensor memory take 180 KB and more).  All
// columns are asked for, so no SM could work on two CTAs anyway.
constexpr int kLeastSmem = 160 * 1024;

struct Plan {
  int nb, nbr;          // x rows a tile (a multiple of 16), and that rounded up to 32
  int ch, stages;       // 128-byte columns a stage, stages of the ring
  int n_acc;            // accumulators
  int split;            // CTAs that share a tile's K
  int n_rt, n_nt, n_tiles;
  int n_chunks;         // 128-byte columns of K (the last may be short)
  int flat;             // K is not whole columns: one copy each
  int groups;           // of epilogue warps
  int pieces;           // 16-byte pieces of a row of B a warp has room for
  int parts;            // bf16 parts of v that meet B on the tensor cores (0: none do)
  int v_off, b_off, bar_off, smem;
  int vec_out;          // out rows take 16-byte (f32) or 8-byte (bf16) stores
};

constexpr int kBarBytes = (2 * kMaxStages + 5) * 8 + 16;

// Shared memory of a plan: the ring of operands, v, the rings of B rows, barriers.
void lay_out(Plan& q, int rank_max, size_t budget) {
  const int rows = (q.nb + q.split - 1) / q.split;   // whose adapters a CTA adds
  const int v = (rows * rank_max * 4 + 127) / 128 * 128;
  const int want = (rows + 3) / 4, most = rank_max > 64 || v > kMaxV / 2 ? max_groups(true) : max_groups(false);
  q.groups = rank_max == 0 ? 1 : want < most ? want : most;
  q.pieces = rank_max == 0 ? 0 : rank_max <= 16 ? 2 : rank_max <= 32 ? 4 : rank_max <= 64 ? 8 : 16;
  const int b = q.groups * 4 * q.pieces * 512;
  const int fixed = 1024 + v + b + kBarBytes, chunk = kWChunk + q.nb * kRowBytes;
  // two stages at least, where one column of K a stage leaves room for them
  while (q.ch > 1 && static_cast<int>(budget) - fixed < 2 * q.ch * chunk) q.ch /= 2;
  const int stage = q.ch * chunk;
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
  if (q.smem < kLeastSmem) q.smem = kLeastSmem;
}

// The plan of rows x (n columns of W, k entries of es bytes) with adapters of up to rm ranks (0: none; tc:
// their products on the tensor cores too); resident(S, smem): clusters of S such CTAs that the device
// keeps at once.  False where a CTA's shared memory would not fit.
template <typename Resident>
bool plan_rows(Plan& q, int rows, int n, int k, int es, int rm, bool tc, size_t budget, int n_sm, Resident resident) {
  q = Plan{};
  q.n_nt = (n + kM - 1) / kM;
  q.n_chunks = (k * es + kRowBytes - 1) / kRowBytes;
  q.flat = k * es % kRowBytes != 0;
  // Up to 256 rows are one tile where that leaves every CTA one tile at most; else tiles of up to
  // 160 rows, of which two accumulators and z fit tensor memory.
  int most = rows <= 256 && q.n_nt <= n_sm ? 256 : 160;
  if (most * rm * 4 > kMaxV) most = 128;   // (whose v fits)
  q.n_rt = (rows + most - 1) / most;
  // Adapters on the CUDA cores take a tile's time row by row, W's stream some 16 rows': where a cluster
  // cannot share a tile, the cut that makes the least of waves times that.  96 requests x 12288 columns (96 tiles,
  // or 288 of 32 rows): 51.9 us whole, 47.6 in three; 200 requests 60 and 57; 24000 columns 58 and 50 in two;
  // but 16384 columns (128 tiles) 38.8 whole, 41 in two.
  if (rm > 0 && !tc && 2 * q.n_nt * q.n_rt > n_sm) {
    int64_t best = INT64_MAX;
    int cut = q.n_rt;
    for (int c = q.n_rt; c <= 4 * q.n_rt; ++c) {
      const int nb = ((rows + c - 1) / c + 15) / 16 * 16;
      const int64_t tiles = static_cast<int64_t>(q.n_nt) * ((rows + nb - 1) / nb), cost = (tiles + n_sm - 1) / n_sm * (nb + 16);
      if (cost < best) {
        best = cost;
        cut = c;
      }
    }
    q.n_rt = cut;
  }
  q.nb = ((rows + q.n_rt - 1) / q.n_rt + 15) / 16 * 16;
  q.n_rt = (rows + q.nb - 1) / q.nb;
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
      if (static_cast<size_t>(t.smem) <= budget && q.n_tiles <= resident(c, t.smem)) q.split = c;
    }
  }
  lay_out(q, rm, budget);
  // (bf16 outputs too need all three: terms of z may cancel)
  q.parts = tc ? 3 : 0;
  return static_cast<size_t>(q.smem) <= budget;
}

}  // namespace
}  // namespace tts
