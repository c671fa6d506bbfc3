// Cache rows of drafted decoding: rows written into a cache (quantised for the 8-bit
// dtypes), read back from it, and moved inside it when a tree's path is accepted.
//
// All three only move bytes, so they are bound by HBM on long inputs and by launch latency
// on one decode step.  A row of head_dim entries is held by the lanes of an eighth to half a
// warp, so a row's largest magnitude is a few shuffles and nothing goes through shared memory.
// K and V of a row go through the same lane (two loads in flight at least); many rows to read
// are read two a lane.
//
// 16 x 1024 rows of 8 heads, bf16 into int8: 37 us (2.7 TB/s; 0.68 of the issue slots, the quantiser's);
// 36.8 k rows back to bf16: 47 us (4.8 TB/s, 0.73 of the measured copy rate; waits on loads).  One row
// of 32 streams: 2.4 and 1.8 us, a launch.  Both of the first took 208 us with
// codes by double division and narrower lanes.
#include "cache_view.cuh"
#include "draft_kernels.h"

namespace tts {
namespace {

constexpr int kWarps = 8;

template <typename SrcT> struct Src;
template <> struct Src<float> {
  static constexpr int kVec = 8;   // entries of a lane: 32 bytes
  static __device__ __forceinline__ void load(const void* p, int64_t i, float (&f)[8]) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 v = __ldcs(q), w = __ldcs(q + 1);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; f[4] = w.x; f[5] = w.y; f[6] = w.z; f[7] = w.w;
  }
};
template <> struct Src<__nv_bfloat16> {
  static constexpr int kVec = 16;
  static __device__ __forceinline__ void load(const void* p, int64_t i, float (&f)[16]) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i);
    const uint4 v = __ldcs(q), w = __ldcs(q + 1);
    float a[8], b[8];
    unpack_bf16x8(v, a);
    unpack_bf16x8(w, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[e] = a[e];
      f[8 + e] = b[e];
    }
  }
};

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// N entries of a lane into the cache row at element i.
template <int N>
__device__ __forceinline__ void store_row(float* p, int64_t i, const float (&x)[N]) {
#pragma unroll
  for (int e = 0; e < N; e += 4) *reinterpret_cast<float4*>(p + i + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
}
template <int N>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, int64_t i, const float (&x)[N]) {
#pragma unroll
  for (int e = 0; e < N; e += 8)
    *reinterpret_cast<uint4*>(p + i + e) = make_uint4(bf16_pair(x[e], x[e + 1]), bf16_pair(x[e + 2], x[e + 3]),
                                                      bf16_pair(x[e + 4], x[e + 5]), bf16_pair(x[e + 6], x[e + 7]));
}
template <typename Code, int N>
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t i, const float (&x)[N], float s, bool zero) {
  uint32_t w[N / 4] = {};
  if (!zero) codes<Code>(x, s, w);
  if constexpr (N == 8) {
    *reinterpret_cast<uint2*>(p + i) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<uint4*>(p + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <typename KvT> struct CodeOf { using type = void; };
template <> struct CodeOf<CodeI8> { using type = I8Code; };
template <> struct CodeOf<CodeE4m3> { using type = E4m3Code; };

// One head row: quantised (a group of LPR lanes agrees on the scale) or converted.
template <typename KvT, int VE, int LPR>
__device__ __forceinline__ void write_head_row(void* cache, float* scale, int64_t row, int D, int lr, bool live,
                                               const float (&x)[VE]) {
  const int64_t at = row * D + lr * VE;
  if constexpr (CacheElem<KvT>::kScaled) {
    // magnitudes order as their bits do; infinities and NaN are the largest
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < VE; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
    for (int o = LPR / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
    if (!live) return;
    using Code = typename CodeOf<KvT>::type;
    const bool bad = top >= 0x7f800000u;
    const float s = bad ? __uint_as_float(0x7fc00000u) : __uint_as_float(top) * (1.0f / Code::kTop);
    store_codes<Code>(static_cast<uint8_t*>(cache), at, x, s, bad || s == 0.f);
    if (lr == 0) scale[row] = s;
  } else {
    if (live) store_row(static_cast<KvT*>(cache), at, x);
  }
}

// Head row i of stream b: (t, g) with g fastest, K and V together.
template <typename SrcT, typename KvT, int D>
__global__ void __launch_bounds__(kWarps * 32) kv_write_kernel(const KvRowsParams p) {
  constexpr int VE = Src<SrcT>::kVec, LPR = D / VE, RPW = 32 / LPR;
  grid_wait();
  grid_launch_dependents();
  const CacheView& c = p.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lr = lane % LPR;
  const int b = blockIdx.y;
  const uint32_t i = (blockIdx.x * kWarps + warp) * RPW + lane / LPR;
  __shared__ int s_start, s_rows;
  if (threadIdx.x == 0) {
    // (once a block: every block of a stream asks the same two words of L2)
    s_start = __ldcg(p.start + b);
    s_rows = p.n_rows == nullptr ? p.T : __ldcg(p.n_rows + b);
    if (blockIdx.x == 0 && (s_rows < 0 || s_rows > p.T)) set_err(p.err, TTS_EFLAG_NVALID);
  }
  __syncthreads();
  const int64_t start = s_start;
  const int nr = s_rows;
  const int t = static_cast<int>(i / c.n_kv_heads), g = static_cast<int>(i) - t * c.n_kv_heads;
  const int64_t pos = start + t;
  const bool first = g == 0 && lr == 0;   // the thread that reports for (b, t)
  bool live = t < min(nr, p.T);
  float xk[VE] = {}, xv[VE] = {};
  if (live) {
    const int64_t src = (static_cast<int64_t>(b) * p.T + t) * p.row_stride + static_cast<int64_t>(g) * D + lr * VE;
    Src<SrcT>::load(p.k, src, xk);
    Src<SrcT>::load(p.v, src, xv);
  }
  if (live && (pos < 0 || pos >= c.capacity)) {
    if (first) set_err(p.err, TTS_EFLAG_POS_RANGE);
    live = false;
  }
  int page = 0;
  if (live && c.paged) {
    page = cache_page(c, b, static_cast<int>(pos));
    if (page < 0) {
      if (first) set_err(p.err, TTS_EFLAG_PAGE);
      live = false;
    }
  }
  const int64_t row = cache_row(c, b, g, live ? static_cast<int>(pos) : 0, live ? page : 0);
  write_head_row<KvT, VE, LPR>(c.k, c.k_scale, row, D, lr, live, xk);
  write_head_row<KvT, VE, LPR>(c.v, c.v_scale, row, D, lr, live, xv);
}

// The entries of a lane as read from the cache: 16 bytes (f32: 32).
template <typename KvT> struct LaneRow;
template <> struct LaneRow<float> {
  static constexpr int kVec = 8;
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    a = __ldcg(q);
    b = __ldcg(q + 1);
  }
  __device__ __forceinline__ void values(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};
template <> struct LaneRow<__nv_bfloat16> {
  static constexpr int kVec = 8;
  uint4 a;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    a = __ldcg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i));
  }
  __device__ __forceinline__ void values(float (&f)[8]) const { unpack_bf16x8(a, f); }
};
template <typename KvT> struct LaneCodes {
  static constexpr int kVec = 16;
  uint4 a;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    a = __ldcg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + i));
  }
  __device__ __forceinline__ void values(float (&f)[16]) const { CacheElem<KvT>::values(a, f); }
};
template <> struct LaneRow<CodeI8> : LaneCodes<CodeI8> {};
template <> struct LaneRow<CodeE4m3> : LaneCodes<CodeE4m3> {};

template <int N>
__device__ __forceinline__ void stream_out(float* p, int64_t i, const float (&f)[N]) {
#pragma unroll
  for (int e = 0; e < N; e += 4)
    __stcs(reinterpret_cast<float4*>(p + i + e), make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]));
}
template <int N>
__device__ __forceinline__ void stream_out(__nv_bfloat16* p, int64_t i, const float (&f)[N]) {
#pragma unroll
  for (int e = 0; e < N; e += 8)
    __stcs(reinterpret_cast<uint4*>(p + i + e), make_uint4(bf16_pair(f[e], f[e + 1]), bf16_pair(f[e + 2], f[e + 3]),
                                                           bf16_pair(f[e + 4], f[e + 5]), bf16_pair(f[e + 6], f[e + 7])));
}

template <typename KvT, typename OutT, int D, int U>
__global__ void __launch_bounds__(kWarps * 32) kv_read_kernel(const KvRowsParams p) {
  constexpr int VE = LaneRow<KvT>::kVec, LPR = D / VE, RPW = 32 / LPR;
  grid_wait();
  grid_launch_dependents();
  const CacheView& c = p.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lr = lane % LPR;
  const int b = blockIdx.y;
  const uint32_t n = static_cast<uint32_t>(p.T) * c.n_kv_heads;   // head rows of a stream (below 2^31)
  const uint32_t i0 = (blockIdx.x * kWarps + warp) * (RPW * U) + lane / LPR;
  __shared__ int s_start, s_rows;
  if (threadIdx.x == 0) {
    // (once a block: every block of a stream asks the same two words of L2)
    s_start = __ldcg(p.start + b);
    s_rows = p.n_rows == nullptr ? p.T : __ldcg(p.n_rows + b);
    if (blockIdx.x == 0 && (s_rows < 0 || s_rows > p.T)) set_err(p.err, TTS_EFLAG_NVALID);
  }
  __syncthreads();
  const int64_t start = s_start;
  const int nr = s_rows;
  int64_t dst[U];
  LaneRow<KvT> k[U], v[U];
  float sk[U], sv[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = i0 + u * RPW;
    dst[u] = -1;
    sk[u] = sv[u] = 1.f;
    if (i >= n) continue;
    const int t = static_cast<int>(i / c.n_kv_heads), g = static_cast<int>(i) - t * c.n_kv_heads;
    const int64_t r = static_cast<int64_t>(b) * p.T + t;
    if (t >= nr) continue;
    const bool first = g == 0 && lr == 0;
    const int64_t pos = start + t;
    if (pos < 0 || pos >= c.capacity) {
      if (first) set_err(p.err, TTS_EFLAG_POS_RANGE);
      continue;
    }
    int page = 0;
    if (c.paged) {
      page = cache_page(c, b, static_cast<int>(pos));
      if (page < 0) {
        if (first) set_err(p.err, TTS_EFLAG_PAGE);
        continue;
      }
    }
    const int64_t row = cache_row(c, b, g, static_cast<int>(pos), page);
    dst[u] = r * p.row_stride + static_cast<int64_t>(g) * D + lr * VE;
    k[u].load(c.k, row * D + lr * VE);
    v[u].load(c.v, row * D + lr * VE);
    if constexpr (CacheElem<KvT>::kScaled) {
      sk[u] = __ldcg(c.k_scale + row);
      sv[u] = __ldcg(c.v_scale + row);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (dst[u] < 0) continue;
    float f[VE];
    k[u].values(f);
#pragma unroll
    for (int e = 0; e < VE; ++e) f[e] = CacheElem<KvT>::kScaled ? f[e] * sk[u] : f[e];
    stream_out(static_cast<OutT*>(p.k_out), dst[u], f);
    v[u].values(f);
#pragma unroll
    for (int e = 0; e < VE; ++e) f[e] = CacheElem<KvT>::kScaled ? f[e] * sv[u] : f[e];
    stream_out(static_cast<OutT*>(p.v_out), dst[u], f);
  }
}

// Rows a lane takes at once: U when one each would already be over four blocks an SM.
template <int RPW, int U>
dim3 row_grid(const KvRowsParams& p, bool& many) {
  const int64_t n = static_cast<int64_t>(p.T) * p.cache.n_kv_heads;
  many = n * p.cache.B > static_cast<int64_t>(p.n_sm) * 4 * kWarps * RPW;
  const int64_t per = static_cast<int64_t>(kWarps) * RPW * (many ? U : 1);
  return dim3(static_cast<unsigned>((n + per - 1) / per), p.cache.B);
}

template <typename SrcT, typename KvT, int D>
cudaError_t launch_write(const KvRowsParams& p, cudaStream_t s) {
  constexpr int per = kWarps * (32 / (D / Src<SrcT>::kVec));
  const int64_t n = static_cast<int64_t>(p.T) * p.cache.n_kv_heads;
  const dim3 grid(static_cast<unsigned>((n + per - 1) / per), p.cache.B);
  return launch_pdl(kv_write_kernel<SrcT, KvT, D>, grid, dim3(kWarps * 32), 0, s, p);
}
template <typename SrcT, typename KvT>
cudaError_t launch_write_d(const KvRowsParams& p, cudaStream_t s) {
  return p.head_dim == 64 ? launch_write<SrcT, KvT, 64>(p, s) : launch_write<SrcT, KvT, 128>(p, s);
}
template <typename SrcT>
cudaError_t launch_write_kv(const KvRowsParams& p, cudaStream_t s) {
  switch (p.kv_dtype) {
    case TTS_F32: return launch_write_d<SrcT, float>(p, s);
    case TTS_BF16: return launch_write_d<SrcT, __nv_bfloat16>(p, s);
    case TTS_I8: return launch_write_d<SrcT, CodeI8>(p, s);
    default: return launch_write_d<SrcT, CodeE4m3>(p, s);
  }
}

template <typename KvT, typename OutT, int D>
cudaError_t launch_read(const KvRowsParams& p, cudaStream_t s) {
  constexpr int RPW = 32 / (D / LaneRow<KvT>::kVec);
  bool many;
  const dim3 grid = row_grid<RPW, 2>(p, many);
  return many ? launch_pdl(kv_read_kernel<KvT, OutT, D, 2>, grid, dim3(kWarps * 32), 0, s, p)
              : launch_pdl(kv_read_kernel<KvT, OutT, D, 1>, grid, dim3(kWarps * 32), 0, s, p);
}
template <typename KvT, typename OutT>
cudaError_t launch_read_d(const KvRowsParams& p, cudaStream_t s) {
  return p.head_dim == 64 ? launch_read<KvT, OutT, 64>(p, s) : launch_read<KvT, OutT, 128>(p, s);
}
template <typename KvT>
cudaError_t launch_read_out(const KvRowsParams& p, cudaStream_t s) {
  return p.row_bf16 ? launch_read_d<KvT, __nv_bfloat16>(p, s) : launch_read_d<KvT, float>(p, s);
}

// ---------------------------------------------------------------------------
// The accepted path's rows move forward: slot n_past + path[i] -> n_past + i.  One warp per
// (stream, kv head, K or V).  path ascends strictly, so path[i] >= i and a later source is
// never an earlier destination; the rows of a batch are all read before any of them is
// written (a warp barrier between), so batches in ascending order move the path exactly.
// ---------------------------------------------------------------------------
template <int ROW_BYTES>
__global__ void __launch_bounds__(32) commit_kernel(const CommitParams p) {
  constexpr int LPR = ROW_BYTES / 16, RPW = 32 / LPR, U = 8;
  grid_wait();
  grid_launch_dependents();
  const CacheView& c = p.cache;
  const int lane = threadIdx.x, lr = lane % LPR;
  const int b = blockIdx.y, g = blockIdx.x >> 1;
  const bool is_v = blockIdx.x & 1;
  const bool report = lane == 0 && blockIdx.x == 0;
  const int n = __ldcg(p.n_accept + b);
  if (n < 0 || n > p.T) {
    if (report) set_err(p.err, TTS_EFLAG_ID_RANGE);
    return;
  }
  if (n == 0) return;
  // lane i holds path entries i and i + 32 (T <= 64)
  const int32_t* path = p.path + static_cast<int64_t>(b) * p.path_stride;
  const int p0 = lane < n ? __ldcg(path + lane) : 0x7fffffff;
  const int p1 = lane + 32 < n ? __ldcg(path + lane + 32) : 0x7fffffff;
  const int prev0 = __shfl_up_sync(kFull, p0, 1), last0 = __shfl_sync(kFull, p0, 31);
  int prev1 = __shfl_up_sync(kFull, p1, 1);
  if (lane == 0) prev1 = last0;
  const bool bad = (lane < n && (p0 < 0 || p0 >= p.T || (lane > 0 && p0 <= prev0))) ||
                   (lane + 32 < n && (p1 >= p.T || p1 <= prev1));
  if (__any_sync(kFull, bad)) {
    if (report) set_err(p.err, TTS_EFLAG_ID_RANGE);
    return;
  }
  const int past = __ldcg(p.n_past + b);
  const int last = __shfl_sync(kFull, n > 32 ? p1 : p0, (n - 1) & 31);
  if (past < 0 || past > c.capacity - 1 - last) {
    if (report) set_err(p.err, TTS_EFLAG_POS_RANGE);
    return;
  }
  // the cache rows of this lane's two entries (destination and source)
  int64_t d0 = -1, s0 = -1, d1 = -1, s1 = -1;
  bool bad_page = false;
  auto rows_of = [&](int i, int from, int64_t& dst, int64_t& src) {
    const int pd = c.paged ? cache_page(c, b, past + i) : 0, ps = c.paged ? cache_page(c, b, past + from) : 0;
    bad_page = bad_page || pd < 0 || ps < 0;
    dst = cache_row(c, b, g, past + i, max(pd, 0));
    src = cache_row(c, b, g, past + from, max(ps, 0));
  };
  if (lane < n) rows_of(lane, p0, d0, s0);
  if (lane + 32 < n) rows_of(lane + 32, p1, d1, s1);
  if (__any_sync(kFull, bad_page)) {
    if (report) set_err(p.err, TTS_EFLAG_PAGE);
    return;
  }
  unsigned char* base = static_cast<unsigned char*>(is_v ? c.v : c.k);
  float* scale = is_v ? c.v_scale : c.k_scale;
  float x0 = 0.f, x1 = 0.f;
  if (scale != nullptr) {
    if (d0 >= 0) x0 = __ldcg(scale + s0);
    if (d1 >= 0) x1 = __ldcg(scale + s1);
  }
  for (int i0 = 0; i0 < n; i0 += RPW * U) {
    uint4 v[U];
    int64_t dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * RPW + lane / LPR;
      const int64_t da = __shfl_sync(kFull, d0, i & 31), db = __shfl_sync(kFull, d1, i & 31);
      const int64_t sa = __shfl_sync(kFull, s0, i & 31), sb = __shfl_sync(kFull, s1, i & 31);
      const int64_t src = i < 32 ? sa : sb;
      dst[u] = i >= n ? -1 : (i < 32 ? da : db);
      if (dst[u] == src) dst[u] = -1;   // already in place
      if (dst[u] >= 0) v[u] = __ldcg(reinterpret_cast<const uint4*>(base + src * ROW_BYTES) + lr);
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (dst[u] >= 0) *(reinterpret_cast<uint4*>(base + dst[u] * ROW_BYTES) + lr) = v[u];
    __syncwarp();
  }
  if (scale != nullptr) {
    // every lane's scales were read before the barriers above
    if (d0 >= 0) scale[d0] = x0;
    if (d1 >= 0) scale[d1] = x1;
  }
}

}  // namespace

cudaError_t launch_kv_write(const KvRowsParams& p, cudaStream_t s) {
  return p.row_bf16 ? launch_write_kv<__nv_bfloat16>(p, s) : launch_write_kv<float>(p, s);
}

cudaError_t launch_kv_read(const KvRowsParams& p, cudaStream_t s) {
  switch (p.kv_dtype) {
    case TTS_F32: return launch_read_out<float>(p, s);
    case TTS_BF16: return launch_read_out<__nv_bfloat16>(p, s);
    case TTS_I8: return launch_read_out<CodeI8>(p, s);
    default: return launch_read_out<CodeE4m3>(p, s);
  }
}

cudaError_t launch_commit(const CommitParams& p, cudaStream_t s) {
  const dim3 grid(2 * p.cache.n_kv_heads, p.cache.B);
  switch (p.row_bytes) {
    case 64: return launch_pdl(commit_kernel<64>, grid, dim3(32), 0, s, p);
    case 128: return launch_pdl(commit_kernel<128>, grid, dim3(32), 0, s, p);
    case 256: return launch_pdl(commit_kernel<256>, grid, dim3(32), 0, s, p);
    case 512: return launch_pdl(commit_kernel<512>, grid, dim3(32), 0, s, p);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tts
