// How the tree attention's work is cut over a launch's CTAs, on the device: the windows are
// device data, so every warp that needs the cut derives it from them, the same way.
//
// Items (stream, kv head, row block), in this order, are laid end to end on a cost axis: an
// item costs p.fixed (its query rows, epilogue and partials) plus kTileCost per tile of its
// window.  CTA r takes the units [r per, (r + 1) per); a piece of an item is the tiles
// whose units fall into a CTA's range.  An item that one CTA takes whole is finished there;
// the pieces of others leave partial rows, which the combine launch merges in CTA order.
// A CTA has at most one piece that starts inside its item (its first: slot 0) and one that
// starts at tile 0 and ends early (its last: slot 1).
#pragma once

#include "cache_view.cuh"
#include "draft_kernels.h"

namespace tts {

constexpr int kTileCost = 4;

// A stream's committed rows and nodes, clamped into the cache; *bad when they had to be.
struct TreeWindow {
  int past, nodes;
};
__device__ __forceinline__ TreeWindow tree_window(const TreeParams& p, int b, bool* bad) {
  const int past = __ldcg(p.n_past + b), nodes = p.n_nodes == nullptr ? p.T : __ldcg(p.n_nodes + b);
  TreeWindow w;
  w.past = min(max(past, 0), p.cache.capacity);
  w.nodes = min(min(max(nodes, 0), p.T), p.cache.capacity - w.past);
  if (bad != nullptr) *bad = w.past != past || w.nodes != nodes;
  return w;
}

// Tiles of a stream's window (0: no nodes, nothing to do).
__device__ __forceinline__ int tree_tiles(const TreeParams& p, TreeWindow w) {
  return w.nodes == 0 ? 0 : (w.past + w.nodes + p.tile - 1) / p.tile;
}
// (units fit 32 bits: the entry point refuses more)
__device__ __forceinline__ int item_cost(const TreeParams& p, int tiles) { return p.fixed + tiles * kTileCost; }
__device__ __forceinline__ int stream_cost(const TreeParams& p, int b) {
  return item_cost(p, tree_tiles(p, tree_window(p, b, nullptr))) * (p.cache.n_kv_heads * p.n_rb);
}

// First tile at or after unit x of an item.
__device__ __forceinline__ int tile_at(const TreeParams& p, int x, int tiles) {
  return min(max(x - p.fixed + kTileCost - 1, 0) / kTileCost, tiles);
}

// Sum of the costs of streams [b0, b1), by a whole warp.
__device__ __forceinline__ int cost_of(const TreeParams& p, int b0, int b1) {
  const int lane = threadIdx.x & 31;
  int sum = 0;
  for (int b = b0 + lane; b < b1; b += 32) sum += stream_cost(p, b);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  return sum;
}

// (The axis is shorter than 2^30: an item costs at most (capacity + 192) / 2 over its row blocks, and
// the entry point refuses B * n_kv_heads * (capacity + 192) from 2^31 on.  The last
// ranges may end past the axis, by fewer than n_cta units: all ends stay below 2^31.)
__device__ __forceinline__ int cost_per_cta(int total, int n_cta) { return (total + n_cta - 1) / n_cta; }

struct Piece {
  int b, g, rb;      // the item
  TreeWindow w;
  int tiles;         // of the item
  int t0, t1;        // the piece: tiles [t0, t1)
  __device__ __forceinline__ bool complete() const { return t0 == 0 && t1 == tiles; }
  __device__ __forceinline__ int slot() const { return t0 > 0 ? 0 : 1; }
};

// Where on the cost axis a stream lies, and how long the axis is.  By a whole warp; up to 32
// streams take one round trip to memory (this stands before everything else a launch does).
struct Axis {
  int lane_past, lane_nodes;   // up to 32 streams: lane b's window
  int total;

  __device__ __forceinline__ TreeWindow window(const TreeParams& p, int b) const {
    if (p.cache.B > 32) return tree_window(p, b, nullptr);
    return {__shfl_sync(kFull, lane_past, b), __shfl_sync(kFull, lane_nodes, b)};
  }
  // Sums the axis; `start`: of stream b (b >= 0), or with b < 0 b becomes the stream that holds
  // unit lo(per_cta) * cta (B when none does).
  __device__ void find(const TreeParams& p, int cta, int& b, int& start) {
    const int lane = threadIdx.x & 31, B = p.cache.B;
    lane_past = lane_nodes = 0;
    if (B <= 32) {
      int own = 0;
      if (lane < B) {
        const TreeWindow w = tree_window(p, lane, nullptr);
        lane_past = w.past;
        lane_nodes = w.nodes;
        own = item_cost(p, tree_tiles(p, w)) * (p.cache.n_kv_heads * p.n_rb);
      }
      int end = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, end, o);
        if (lane >= o) end += x;
      }
      total = __shfl_sync(kFull, end, 31);
      if (b < 0) {
        const unsigned over = __ballot_sync(kFull, end > cost_per_cta(total, p.n_cta) * cta);
        b = over == 0 ? B : __ffs(static_cast<int>(over)) - 1;
      }
      start = b < B ? __shfl_sync(kFull, end - own, b) : total;
      return;
    }
    total = cost_of(p, 0, B);
    if (b >= 0) {
      start = cost_of(p, 0, b);
      return;
    }
    const int lo = cost_per_cta(total, p.n_cta) * cta;
    start = 0;
    b = B;
    for (int b0 = 0; b0 < B; b0 += 32) {
      const int own = b0 + lane < B ? stream_cost(p, b0 + lane) : 0;
      int end = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, end, o);
        if (lane >= o) end += x;
      }
      const unsigned over = __ballot_sync(kFull, start + end > lo);
      if (over != 0) {
        const int at = __ffs(static_cast<int>(over)) - 1;
        b = b0 + at;
        start += __shfl_sync(kFull, end - own, at);
        break;
      }
      start += __shfl_sync(kFull, end, 31);
    }
  }
};

// The pieces of one CTA, in order.  Every call is by a whole warp.
struct PieceWalk {
  Axis axis;
  int lo, hi;        // the CTA's units
  int start;         // where item `next` starts
  int b, next;       // stream, and item of the stream (g * n_rb + rb), of the next item
  TreeWindow w;
  int tiles;

  __device__ __forceinline__ void set_stream(const TreeParams& p) {
    if (b < p.cache.B) {
      w = p.whole ? tree_window(p, b, nullptr) : axis.window(p, b);
      tiles = tree_tiles(p, w);
    }
  }

  __device__ void init(const TreeParams& p, int cta) {
    if (p.whole) {
      // items dealt out one by one
      b = cta / (p.cache.n_kv_heads * p.n_rb);
      next = cta % (p.cache.n_kv_heads * p.n_rb);
      lo = start = 0;
      hi = 1;
      set_stream(p);
      return;
    }
    b = -1;
    axis.find(p, cta, b, start);
    const int per = cost_per_cta(axis.total, p.n_cta);
    lo = per * cta;
    hi = lo + per;
    next = 0;
    set_stream(p);
    if (b < p.cache.B) {
      const int c = item_cost(p, tiles);
      next = (lo - start) / c;
      start += c * next;
    }
  }

  __device__ bool get(const TreeParams& p, Piece& out) {
    while (b < p.cache.B && start < hi) {
      out.b = b;
      out.g = next / p.n_rb;
      out.rb = next - out.g * p.n_rb;
      out.w = w;
      out.tiles = tiles;
      if (p.whole) {
        out.t0 = 0;
        out.t1 = tiles;
        start = hi;
        return tiles > 0;
      }
      out.t0 = tile_at(p, lo - start, tiles);
      out.t1 = tile_at(p, hi - start, tiles);
      start += item_cost(p, tiles);
      if (++next == p.cache.n_kv_heads * p.n_rb) {
        next = 0;
        ++b;
        set_stream(p);
      }
      if (out.t0 < out.t1) return true;
    }
    return false;
  }
};

// The nodes a node sees, as bits.
__device__ __forceinline__ uint64_t seen_nodes(const TreeParams& p, int b, int t, int nodes) {
  const uint64_t all = nodes >= 64 ? ~0ull : (1ull << nodes) - 1;
  const uint64_t m = p.mask == nullptr ? (t >= 63 ? ~0ull : (2ull << t) - 1)
                                       : __ldcg(reinterpret_cast<const unsigned long long*>(p.mask) +
                                                static_cast<int64_t>(b) * p.T + t);
  return m & all;
}

// Four columns of an output row times inv, in the output's type.
__device__ __forceinline__ void store_tree_row4(const TreeParams& p, int b, int t, int h, int D, int col, float4 o,
                                                float inv) {
  const int64_t at = ((static_cast<int64_t>(b) * p.T + t) * p.n_q_heads + h) * D + col;
  if (p.q_bf16) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(o.x * inv, o.y * inv), y = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  }
}

}  // namespace tts
