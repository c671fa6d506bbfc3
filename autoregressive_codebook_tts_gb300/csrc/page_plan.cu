// Pages and row maps of a step of many requests, planned on the device.
//
// The plan is three scans over the streams (pages returned, pages needed, rows) around reads of
// the few table entries that a step can touch, so it is bound by latency: one cluster of eight
// CTAs does it in one launch.  The CTAs share the counting of table entries (a warp a stream) and
// tell each other through distributed shared memory; each then scans all streams by itself, which
// costs less than another exchange.  Pages are returned, then (a cluster barrier later) taken from
// the list's end, then (another) read for the row maps.  Long maps are filled by a launch of their
// own over the whole GPU.
//
// A step of 64 streams takes 8.5 us, one of 512 streams with 38 k rows 13.0, of which the second launch has
// some 4: chains of dependent reads (about 0.7 us each) and barriers, the code of each phase fetched once.
// (One CTA, without the exchange: 9.6 and 37 us.)
#include "common.cuh"
#include "serve_kernels.h"

namespace tts {
namespace {

constexpr int kCtas = 8;
constexpr int kThreads = 512;
constexpr int kPlanWarps = kThreads / 32;
constexpr int kAllWarps = kCtas * kPlanWarps;
constexpr int kFillThreads = 256;
// Maps of more rows than this are filled by a second launch.
constexpr int kOneLaunchRows = 16384;

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Inclusive sums over the block of two values a thread, each held at its cap (so that 32 bits hold
// them; the caps are at most 2^30 + 1); returns the sum of a before this thread.  (Held at the cap
// too: the inclusive sum less the thread's own would be too small there.)
__device__ __forceinline__ uint32_t block_scan(uint32_t& a, uint32_t& b, uint32_t cap_a, uint32_t cap_b, uint2* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  a = min(a, cap_a);
  b = min(b, cap_b);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(kFull, a, o), y = __shfl_up_sync(kFull, b, o);
    if (lane >= o) {
      a = min(a + x, cap_a);
      b = min(b + y, cap_b);
    }
  }
  if (lane == 31) s_warp[warp] = make_uint2(a, b);
  uint32_t before = __shfl_up_sync(kFull, a, 1);
  if (lane == 0) before = 0;
  __syncthreads();
  for (int w = 0; w < warp; ++w) {
    a = min(a + s_warp[w].x, cap_a);
    b = min(b + s_warp[w].y, cap_b);
    before = min(before + s_warp[w].x, cap_a);
  }
  __syncthreads();
  return before;
}

// The map entries of row r, which is of stream b (or of none: b < 0).
template <typename Past>
__device__ __forceinline__ void map_row(const PagePlanParams& p, int r, int b, int t, Past past) {
  int pos = 0;
  int64_t slot = -1;
  if (b >= 0) {
    pos = past(b) + t;
    const int page = __ldcg(p.table + static_cast<int64_t>(b) * p.bt_stride + (pos >> p.page_shift));
    if (page >= 0 && page < p.n_pages)
      slot = (static_cast<int64_t>(page) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
    else
      set_err(p.err, TTS_EFLAG_PAGE);
  }
  p.row_stream[r] = b;
  p.row_pos[r] = pos;
  p.row_slot[r] = slot;
}

// The stream of packed row r: the last b with start[b] <= r that has rows; start[B] > r.
template <typename Start>
__device__ __forceinline__ int stream_of(Start start, int B, int r) {
  int lo = 0, hi = B;   // start[lo] <= r < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start(mid) <= r) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <typename Start, typename Rows, typename Past>
__device__ __forceinline__ void fill_maps(const PagePlanParams& p, int first, int step, Start start, Rows rows, Past past) {
  const int total = p.T > 0 ? 0 : start(p.B);
  for (int r = first; r < p.max_rows; r += step) {
    if (p.T > 0) {
      const int b = r / p.T, t = r - b * p.T;
      map_row(p, r, t < rows(b) ? b : -1, t, past);
    } else if (r < total) {
      const int b = stream_of(start, p.B, r);
      map_row(p, r, b, r - start(b), past);
    } else {
      map_row(p, r, -1, 0, past);
    }
  }
}

__global__ void __launch_bounds__(kThreads) page_plan_kernel(const PagePlanParams p, int fill) {
  extern __shared__ uint32_t s_dyn[];
  uint32_t* s_give = s_dyn;             // [B] pages a stream returns, then where they go on the list
  uint32_t* s_need = s_dyn + p.B;       // [B] pages a stream needs
  uint32_t* s_from = s_dyn + 2 * p.B;   // [B] pages needed before it
  int* s_rows = reinterpret_cast<int*>(s_dyn + 3 * p.B);    // [B] rows granted
  int* s_start = reinterpret_cast<int*>(s_dyn + 4 * p.B);   // [B + 1]
  int* s_new = reinterpret_cast<int*>(s_dyn + 5 * p.B + 1);   // [B] n_new and n_past: asked for once
  int* s_past = s_new + p.B;
  __shared__ uint2 s_warp[kPlanWarps];
  __shared__ uint2 s_carry;
  __shared__ uint32_t s_used;
  grid_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_rank());
  const int gw = warp * kCtas + rank;   // this warp among the cluster's
  const int per = p.capacity >> p.page_shift;
  const int listed = __ldcg(p.n_free);
  for (int b = tid; b < p.B; b += kThreads) {
    const int fresh = __ldcg(p.n_new + b), past = __ldcg(p.n_past + b);
    s_new[b] = fresh;
    s_past[b] = past;
  }
  const int n_free = min(max(listed, 0), p.n_pages);
  int flags = n_free != listed ? TTS_EFLAG_NVALID : 0;
  auto wants = [&](int past, int fresh) {
    return fresh > 0 && past >= 0 && past <= p.capacity - fresh && (p.T == 0 || fresh <= p.T);
  };
  auto holds = [&](int page) { return page >= 0 && page < p.n_pages; };

  // 1. table entries counted, a warp a stream, and told to every CTA
  const uint32_t give_at = map_shared_rank(s_give, lane & (kCtas - 1));
  const uint32_t need_at = map_shared_rank(s_need, lane & (kCtas - 1));
  cluster_sync_all();   // every CTA of the cluster has begun: its shared memory may be written
  for (int b = gw; b < p.B; b += kAllWarps) {
    const int fresh = s_new[b], past = s_past[b];
    const int32_t* row = p.table + static_cast<int64_t>(b) * p.bt_stride;
    const bool ended = fresh < 0;
    uint32_t give = 0, need = 0;
    if (ended || wants(past, fresh)) {
      const int lo = ended ? 0 : past >> p.page_shift;
      const int hi = ended ? per : ((past + fresh - 1) >> p.page_shift) + 1;
      uint32_t held = 0;
#pragma unroll 4
      for (int i = lo + lane; i < hi; i += 32) held += holds(__ldcg(row + i));
      held = __reduce_add_sync(kFull, held);
      if (ended) give = held;
      else need = static_cast<uint32_t>(hi - lo) - held;
    }
    if (lane < kCtas) {
      st_cluster_u32(give_at + b * 4, give);
      st_cluster_u32(need_at + b * 4, need);
    }
  }
  cluster_sync_all();

  // 2. sums over the streams: pages returned and needed
  const uint32_t cap = static_cast<uint32_t>(p.n_pages) + 1;
  uint32_t freed = 0, asked = 0;   // of the streams before this batch
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int b = b0 + tid;
    const uint32_t give = b < p.B ? s_give[b] : 0, need = b < p.B ? s_need[b] : 0;
    uint32_t x = give, y = need;
    const uint32_t ahead = block_scan(x, y, cap, cap, s_warp);
    if (tid == kThreads - 1) s_carry = make_uint2(x, y);
    if (b < p.B) {
      s_give[b] = min(freed + ahead, cap);
      s_from[b] = min(asked + y, cap);   // (with its own for now)
    }
    __syncthreads();
    freed = min(freed + s_carry.x, cap);
    asked = min(asked + s_carry.y, cap);
    __syncthreads();
  }
  // (the list overflows only where a page is listed or held twice)
  const uint32_t kept = min(freed, static_cast<uint32_t>(p.n_pages - n_free));
  if (kept < freed) flags |= TTS_EFLAG_PAGE;
  const uint32_t top = n_free + kept;

  // 3. rows granted.  The sum that max_rows bounds is held one past it; up to there it is exact,
  // and behind the first stream that does not fit every later sum is over it too.
  const uint32_t most = p.T > 0 ? 0 : static_cast<uint32_t>(p.max_rows), over = most + 1;
  uint32_t before = 0, total = 0;
  if (tid == 0) s_used = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int b = b0 + tid;
    uint32_t need = 0, upto = 0;
    int rows = 0;
    if (b < p.B) {
      const int fresh = s_new[b], past = s_past[b];
      need = s_need[b];
      upto = s_from[b];
      if (wants(past, fresh)) {
        if (need == 0 || upto <= top) rows = fresh;
        else flags |= TTS_EFLAG_PAGE;
      } else if (fresh > 0) {
        flags |= TTS_EFLAG_NVALID;
      }
    }
    const uint32_t count = p.T > 0 ? 0 : min(static_cast<uint32_t>(rows), over);
    uint32_t x = count, y = 0;
    block_scan(x, y, over, over, s_warp);
    const uint32_t sum = min(before + x, over);
    const bool fits = sum <= most;
    if (rows > 0 && !fits) {
      rows = 0;
      flags |= TTS_EFLAG_NVALID;
    }
    if (b < p.B) {
      s_rows[b] = rows;
      s_start[b] = p.T > 0 ? b * p.T : (fits ? static_cast<int>(sum - count) : -1);
      s_from[b] = upto - min(need, upto);
      // the pages taken are those up to the last stream that was given any
      if (rows > 0 && need > 0) atomicMax(&s_used, upto);
    }
    // the largest sum that fits, and the sum of all
    uint32_t best = __reduce_max_sync(kFull, fits && b < p.B ? sum : 0u);
    if (lane == 0) s_warp[warp] = make_uint2(best, 0);
    if (tid == kThreads - 1) s_carry = make_uint2(sum, 0);
    __syncthreads();
    for (int w = 0; w < kPlanWarps; ++w) total = max(total, s_warp[w].x);
    before = s_carry.x;
    __syncthreads();
  }
  const uint32_t used = s_used;
  for (int b = tid; b <= p.B; b += kThreads) {
    if (b == p.B) s_start[b] = p.T > 0 ? p.B * p.T : static_cast<int>(total);
    else if (s_start[b] < 0) s_start[b] = static_cast<int>(total);
  }
  __syncthreads();
  if (rank == 0) {
    for (int b = tid; b <= p.B; b += kThreads) {
      if (b < p.B) p.n_rows[b] = s_rows[b];
      p.row_start[b] = s_start[b];
    }
    if (tid == 0) *p.n_free = static_cast<int>(top - used);   // (every CTA has read it)
    if (flags != 0) set_err(p.err, flags);
  }

  // 4. pages of ended streams to the list
  for (int b = gw; b < p.B; b += kAllWarps) {
    if (s_new[b] >= 0 || freed == 0) continue;
    int32_t* row = p.table + static_cast<int64_t>(b) * p.bt_stride;
    uint32_t at = n_free + s_give[b];
    for (int i0 = 0; i0 < per; i0 += 32) {
      const int i = i0 + lane;
      const int page = i < per ? __ldcg(row + i) : -1;
      const bool held = holds(page);
      const uint32_t m = __ballot_sync(kFull, held);
      const uint32_t to = at + __popc(m & ((1u << lane) - 1));
      if (held) {
        if (to < static_cast<uint32_t>(p.n_pages)) p.free_pages[to] = page;
        row[i] = -1;
      }
      at += __popc(m);
    }
  }
  if (freed != 0) cluster_sync_all();   // (the same in every CTA)
  // 5. pages from the list's end to the entries in need
  for (int b = gw; b < p.B; b += kAllWarps) {
    if (s_rows[b] == 0 || s_need[b] == 0) continue;
    const int past = s_past[b];
    int32_t* row = p.table + static_cast<int64_t>(b) * p.bt_stride;
    const int lo = past >> p.page_shift, hi = ((past + s_rows[b] - 1) >> p.page_shift) + 1;
    uint32_t from = s_from[b];
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      const bool lacks = i < hi && !holds(__ldcg(row + i));
      const uint32_t m = __ballot_sync(kFull, lacks);
      if (lacks) row[i] = __ldcg(p.free_pages + (top - 1 - from - __popc(m & ((1u << lane) - 1))));
      from += __popc(m);
    }
  }
  if (fill) {
    if (used != 0) cluster_sync_all();
    fill_maps(p, rank * kThreads + tid, kCtas * kThreads, [&](int b) { return s_start[b]; },
              [&](int b) { return s_rows[b]; }, [&](int b) { return s_past[b]; });
  }
}

__global__ void __launch_bounds__(kFillThreads) page_fill_kernel(const PagePlanParams p) {
  extern __shared__ int s_begin[];   // [B + 1], packed rows
  grid_wait();
  grid_launch_dependents();
  if (p.T == 0) {
    for (int b = threadIdx.x; b <= p.B; b += kFillThreads) s_begin[b] = __ldcg(p.row_start + b);
    __syncthreads();
  }
  fill_maps(p, blockIdx.x * kFillThreads + threadIdx.x, gridDim.x * kFillThreads, [&](int b) { return s_begin[b]; },
            [&](int b) { return __ldcg(p.n_rows + b); }, [&](int b) { return __ldcg(p.n_past + b); });
}

}  // namespace

cudaError_t launch_page_plan(const PagePlanParams& p, cudaStream_t s) {
  const size_t smem = (7 * static_cast<size_t>(p.B) + 1) * sizeof(uint32_t);
  const bool fill = p.max_rows <= kOneLaunchRows;
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024)
    e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (7 * TTS_MAX_PLAN_STREAMS + 1) * sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, page_plan_kernel, p, static_cast<int>(fill));
  if (e != cudaSuccess || fill) return e;
  const int blocks = (p.max_rows + kFillThreads - 1) / kFillThreads;
  const size_t begin = p.T == 0 ? (static_cast<size_t>(p.B) + 1) * sizeof(int) : 0;
  return launch_pdl(page_fill_kernel, dim3(blocks < 1216 ? blocks : 1216), dim3(kFillThreads), begin, s, p);
}

}  // namespace tts
