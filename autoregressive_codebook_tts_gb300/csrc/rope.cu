// Rotary positions: rows of q and k heads rotated (half or interleaved pairs, all or part of
// the head, with or without the per-head RMSNorm), and the scaled tables they read.
#include "cache_view.cuh"
#include "draft_kernels.h"

namespace tts {
namespace {

// ---------------------------------------------------------------------------
// Rows.  A head row is held by D/4 lanes, four entries each (one 16-byte load of f32, 8 bytes
// of bf16).  A pair's two entries sit in different lanes, at a distance that is any number up
// to D/2, so the normed row goes through a warp-private patch of shared memory and each lane
// reads its partners back from there (four neighbours of a vector's entries are a vector too
// unless rot_dim / 2 is not a multiple of four).  A warp takes U (one or six) heads of one row, all loads
// issued first; the row's (cos, sin) are loaded once and serve them all.  Bound by HBM on a
// prompt's rows, by launch latency on one decode step.
// ---------------------------------------------------------------------------
constexpr int kRopeWarps = 4;

template <typename T> struct Io;
template <> struct Io<float> {
  static __device__ __forceinline__ void load(const void* p, int64_t i, float (&x)[4]) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&x)[4]) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(x[0], x[1], x[2], x[3]);
  }
};
template <> struct Io<__nv_bfloat16> {
  static __device__ __forceinline__ void load(const void* p, int64_t i, float (&x)[4]) {
    const uint2 v = __ldcg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + i));
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xffff0000u);
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&x)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
};

template <typename InT, typename OutT, int D, int U>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_rows_kernel(const RopeRowsParams p) {
  constexpr int LPR = D / 4, HPW = 32 / LPR;   // lanes of a head, heads of a warp at once
  __shared__ float patch[kRopeWarps][32 * 4];
  grid_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lr = lane % LPR;
  const int n_heads = p.n_q_heads + p.n_kv_heads;
  const int64_t r = blockIdx.x;
  const int h0 = (blockIdx.y * kRopeWarps + warp) * (HPW * U) + lane / LPR;
  int pos = __ldcg(p.pos + r);
  float x[U][4];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * HPW;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[u][e] = 0.f;
    if (h < p.n_q_heads)
      Io<InT>::load(p.q, r * p.q_stride + static_cast<int64_t>(h) * D + lr * 4, x[u]);
    else if (h < n_heads)
      Io<InT>::load(p.k, r * p.k_stride + static_cast<int64_t>(h - p.n_q_heads) * D + lr * 4, x[u]);
  }
  // the norm's weights, of the kinds of head that the warp has (every warp of the grid reads the
  // same few lines)
  float4 gq = make_float4(1.f, 1.f, 1.f, 1.f), gk = gq;
  if (p.gamma_q != nullptr) {
    if (h0 < p.n_q_heads) gq = __ldcg(reinterpret_cast<const float4*>(p.gamma_q) + lr);
    if (h0 + (U - 1) * HPW >= p.n_q_heads && p.n_kv_heads > 0)
      gk = __ldcg(reinterpret_cast<const float4*>(p.gamma_k) + lr);
  }
  if (pos < 0 || pos >= p.max_pos) {
    if (h0 == 0 && lr == 0) set_err(p.err, TTS_EFLAG_POS_RANGE);
    pos = min(max(pos, 0), p.max_pos - 1);
  }
  // entry e: its partner's index, and its own and its partner's factors (1, 0 past rot_dim)
  const int half = p.rot_dim / 2;
  const bool by_vector = !p.interleaved && (half & 3) == 0;
  const float2* cs = p.cs + static_cast<int64_t>(pos) * half;
  int partner[4];
  float fc[4] = {1.f, 1.f, 1.f, 1.f}, fs[4] = {0.f, 0.f, 0.f, 0.f};
  if (by_vector) {
    const bool first = lr * 4 < half;
    partner[0] = lr * 4 < p.rot_dim ? (first ? lr * 4 + half : lr * 4 - half) : lr * 4;
    if (lr * 4 < p.rot_dim) {
      const float4* c4 = reinterpret_cast<const float4*>(cs + (first ? lr * 4 : lr * 4 - half));
      const float4 a = __ldcg(c4), b = __ldcg(c4 + 1);
      fc[0] = a.x; fc[1] = a.z; fc[2] = b.x; fc[3] = b.z;
      fs[0] = a.y; fs[1] = a.w; fs[2] = b.y; fs[3] = b.w;
      if (first) {
#pragma unroll
        for (int e = 0; e < 4; ++e) fs[e] = -fs[e];   // t_a c - t_b s, t_b c + t_a s
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = lr * 4 + e;
      partner[e] = i;
      if (i < p.rot_dim) {
        const bool first = p.interleaved ? (i & 1) == 0 : i < half;
        partner[e] = p.interleaved ? i ^ 1 : (first ? i + half : i - half);
        const float2 v = __ldcg(cs + (p.interleaved ? i >> 1 : (first ? i : i - half)));
        fc[e] = v.x;
        fs[e] = first ? -v.y : v.y;
      }
    }
  }
  float* mine = patch[warp] + (lane / LPR) * D;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * HPW;
    float t[4] = {x[u][0], x[u][1], x[u][2], x[u][3]};
    if (p.gamma_q != nullptr) {
      float ss = fmaf(t[0], t[0], fmaf(t[1], t[1], fmaf(t[2], t[2], t[3] * t[3])));
#pragma unroll
      for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
      const float rn = 1.0f / sqrtf(ss / static_cast<float>(D) + p.eps);
      const float4 gm = h < p.n_q_heads ? gq : gk;
      t[0] = t[0] * rn * gm.x;
      t[1] = t[1] * rn * gm.y;
      t[2] = t[2] * rn * gm.z;
      t[3] = t[3] * rn * gm.w;
    }
    // pairs of neighbours are a lane's own; others come from the patch
    float pt[4] = {t[1], t[0], t[3], t[2]};
    if (!p.interleaved) {
      __syncwarp();
      *reinterpret_cast<float4*>(mine + lr * 4) = make_float4(t[0], t[1], t[2], t[3]);
      __syncwarp();
      if (by_vector) {
        const float4 v = *reinterpret_cast<const float4*>(mine + partner[0]);
        pt[0] = v.x; pt[1] = v.y; pt[2] = v.z; pt[3] = v.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) pt[e] = mine[partner[e]];
      }
    }
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = lr * 4 + e < p.rot_dim ? fmaf(t[e], fc[e], pt[e] * fs[e]) : t[e];
    if (h < p.n_q_heads)
      Io<OutT>::store(p.q_out, r * p.q_out_stride + static_cast<int64_t>(h) * D + lr * 4, y);
    else if (h < n_heads)
      Io<OutT>::store(p.k_out, r * p.k_out_stride + static_cast<int64_t>(h - p.n_q_heads) * D + lr * 4, y);
  }
}

template <typename InT, typename OutT, int D, int U>
cudaError_t launch_rows(const RopeRowsParams& p, cudaStream_t s) {
  constexpr int per = 32 / (D / 4) * U * kRopeWarps;   // heads of a block
  const int gy = (p.n_q_heads + p.n_kv_heads + per - 1) / per;
  const dim3 grid(static_cast<unsigned>(p.rows), gy);
  return launch_pdl(rope_rows_kernel<InT, OutT, D, U>, grid, dim3(kRopeWarps * 32), 0, s, p);
}
template <typename InT, typename OutT, int D>
cudaError_t launch_rows_u(const RopeRowsParams& p, cudaStream_t s) {
  // six heads a warp (a row of 24 heads is then one block) once one each would give every SM
  // over 32 warps
  const int64_t warps = static_cast<int64_t>(p.rows) * (p.n_q_heads + p.n_kv_heads) / (32 / (D / 4));
  return warps > static_cast<int64_t>(p.n_sm) * 32 ? launch_rows<InT, OutT, D, 6>(p, s)
                                                   : launch_rows<InT, OutT, D, 1>(p, s);
}
template <typename InT, typename OutT>
cudaError_t launch_rows_d(const RopeRowsParams& p, cudaStream_t s) {
  return p.head_dim == 64 ? launch_rows_u<InT, OutT, 64>(p, s) : launch_rows_u<InT, OutT, 128>(p, s);
}

// ---------------------------------------------------------------------------
// Tables.  The frequencies and the angles need double, whose rate on this GPU is about a
// sixtieth of single, so a sine and cosine in double per entry would bound the table far above
// its bytes.  A block of kSpan positions from p0 takes them only of p0 f and of 2^k f, k < kBits
// (eleven per frequency for 1024 positions), and forms every entry by the angle-sum identities,
//   cos(x + y) = cos x cos y - sin x sin y,  sin(x + y) = sin x cos y + cos x sin y,
// in pairs of singles (a value and its remainder: about 48 bits): first the multiples
// j < kSide of f and p0 f + kSide j f, each a product over the bits of j, then the entry
// (p0 + kSide a + b) f as one product, rounded to f32 once.
// ---------------------------------------------------------------------------
constexpr int kBits = 10, kSide = 32, kSpan = kSide * kSide, kFreqs = 8, kTabThreads = 256;

struct Pair { float hi, lo; };
struct Turn { Pair c, s; };   // (cos, sin) of an angle
__device__ __forceinline__ Pair pair_of(double x) {
  const float h = static_cast<float>(x);
  return {h, static_cast<float>(x - static_cast<double>(h))};
}
__device__ __forceinline__ Pair negate(Pair a) { return {-a.hi, -a.lo}; }

// a b + c d to about 2^-46: a sum and the rest that its rounding leaves.
__device__ __forceinline__ Pair dot2(Pair a, Pair b, Pair c, Pair d) {
  // (explicit roundings: a contracted product would not be the p and q of the remainders)
  const float p = __fmul_rn(a.hi, b.hi), ep = __fmaf_rn(a.hi, b.hi, -p);
  const float q = __fmul_rn(c.hi, d.hi), eq = __fmaf_rn(c.hi, d.hi, -q);
  const float s = __fadd_rn(p, q), z = __fadd_rn(s, -p);
  // the rounding of p + q, exactly
  const float es = __fadd_rn(__fadd_rn(p, -__fadd_rn(s, -z)), __fadd_rn(q, -z));
  const float low = fmaf(a.hi, b.lo, fmaf(a.lo, b.hi, ep)) + fmaf(c.hi, d.lo, fmaf(c.lo, d.hi, eq));
  const float rest = __fadd_rn(es, low), hi = __fadd_rn(s, rest);
  return {hi, __fadd_rn(rest, -__fadd_rn(hi, -s))};
}
__device__ __forceinline__ Turn add_angles(const Turn& x, const Turn& y) {
  return {dot2(x.c, y.c, negate(x.s), y.s), dot2(x.s, y.c, x.c, y.s)};
}

__device__ double rope_frequency(const RopeTableParams& p, int i) {
  double base = p.base;
  const double d = p.rot_dim;
  if (p.s.kind == TTS_ROPE_BASE) base *= pow(p.s.factor, d / (d - 2.0));
  const double f = pow(base, -2.0 * i / d);
  if (p.s.kind == TTS_ROPE_LINEAR) return f / p.s.factor;
  if (p.s.kind == TTS_ROPE_PARTS) {
    const double turns = p.s.original_max_pos * f / 6.283185307179586476925;
    const double w = fmin(fmax((turns - p.s.low_rotations) / (p.s.high_rotations - p.s.low_rotations), 0.0), 1.0);
    return f * (w + (1.0 - w) / p.s.factor);
  }
  return f;
}

__global__ void __launch_bounds__(kTabThreads) rope_table_scaled_kernel(const RopeTableParams p) {
  __shared__ double freq[kFreqs];
  __shared__ Turn step[kBits + 1][kFreqs];            // 2^k f, and p0 f at the end
  __shared__ Turn far[kSide][kFreqs], near[kSide][kFreqs];
  grid_wait();
  grid_launch_dependents();
  const int half = p.rot_dim / 2, f0 = blockIdx.x * kFreqs;
  const int64_t p0 = static_cast<int64_t>(blockIdx.y) * kSpan;
  if (threadIdx.x < kFreqs && f0 + static_cast<int>(threadIdx.x) < half)
    freq[threadIdx.x] = rope_frequency(p, f0 + threadIdx.x);
  __syncthreads();
  const int f = threadIdx.x % kFreqs, j0 = threadIdx.x / kFreqs;   // j0 < kSide
  const bool live = f0 + f < half;
  if (live && j0 <= kBits) {
    double sn, cn;
    sincos(static_cast<double>(j0 < kBits ? int64_t{1} << j0 : p0) * freq[f], &sn, &cn);
    // the factor goes into the far side of every entry's product
    const double a = j0 < kBits ? 1.0 : p.s.attn_scale;
    step[j0][f] = {pair_of(cn * a), pair_of(sn * a)};
  }
  __syncthreads();
  if (live) {
    Turn x = {{1.f, 0.f}, {0.f, 0.f}}, y = step[kBits][f];
#pragma unroll
    for (int k = 0; k < kBits / 2; ++k)
      if ((j0 >> k) & 1) {
        x = add_angles(x, step[k][f]);
        y = add_angles(y, step[kBits / 2 + k][f]);
      }
    near[j0][f] = x;
    far[j0][f] = y;
  }
  __syncthreads();
  if (!live) return;
  // thread (j0, f): the entries p0 + kSide a + j0
  const Turn b = near[j0][f];
#pragma unroll 4
  for (int a = 0; a < kSide; ++a) {
    const int64_t pos = p0 + a * kSide + j0;
    if (pos >= p.max_pos) break;
    const Turn t = add_angles(far[a][f], b);
    p.cs[pos * half + f0 + f] = make_float2(t.c.hi, t.s.hi);
  }
}

}  // namespace

cudaError_t launch_rope_rows(const RopeRowsParams& p, cudaStream_t s) {
  if (p.in_bf16)
    return p.out_bf16 ? launch_rows_d<__nv_bfloat16, __nv_bfloat16>(p, s) : launch_rows_d<__nv_bfloat16, float>(p, s);
  return p.out_bf16 ? launch_rows_d<float, __nv_bfloat16>(p, s) : launch_rows_d<float, float>(p, s);
}

cudaError_t launch_rope_table_scaled(const RopeTableParams& p, cudaStream_t s) {
  const int64_t per = kSpan;
  const dim3 grid((p.rot_dim / 2 + kFreqs - 1) / kFreqs, static_cast<unsigned>((p.max_pos + per - 1) / per));
  return launch_pdl(rope_table_scaled_kernel, grid, dim3(kTabThreads), 0, s, p);
}

}  // namespace tts
