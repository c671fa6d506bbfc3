// Rotary positions: rows of q and k heads rotated (half or interleaved pairs, all or part of
// the head, with or without the per-head RMSNorm), and the scaled tables they read.
#include "cache_view.cuh"
#include "draft_kernels.h"

namespace tts {
namespace {

// ---------------------------------------------------------------------------
// Rows.  A head row is held by D/8 lanes, eight entries each.  In the half layout a pair's two
// entries sit in different lanes, at a distance that is any number up to D/2, so the normed row
// goes through a warp-private patch of shared memory and each lane reads its partners back from
// there (as vectors unless rot_dim / 2 is not a multiple of four).  A lane takes U (one or three)
// heads of one row, all loads issued first; the row's (cos, sin) are loaded once and serve them
// all.  8191 rows of 24 heads, f32 to bf16: 34.7 us (4.4 TB/s, 0.66 of the measured copy rate), bound
// by load latency and issue (0.61 of the slots); 32 rows: 2.1 us, a launch.
// ---------------------------------------------------------------------------
constexpr int kRopeWarps = 4;

// Eight entries of a lane.
template <typename T> struct Io;
template <> struct Io<float> {
  static __device__ __forceinline__ void load(const void* p, int64_t i, float (&x)[8]) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 v = __ldcg(q), w = __ldcg(q + 1);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w; x[4] = w.x; x[5] = w.y; x[6] = w.z; x[7] = w.w;
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&x)[8]) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(x[0], x[1], x[2], x[3]);
    q[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};
template <> struct Io<__nv_bfloat16> {
  static __device__ __forceinline__ void load(const void* p, int64_t i, float (&x)[8]) {
    unpack_bf16x8(__ldcg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i)), x);
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// a^(-1/2): the fast instruction and one Newton step (about one unit in the last place; 0 and
// infinity as they are).
__device__ __forceinline__ float inv_sqrt(float a) {
  const float r = rsqrtf(a);
  return a > 0.f && a < 3e38f ? r * fmaf(-0.5f * a * r, r, 1.5f) : r;
}

// Blocks of a many-row grid walk the rows, kRowBlocks a multiprocessor.  (The norm's weights are
// read once a block: read once a row, or once a warp, they are a few lines of L2 that the whole
// GPU asks for at once, and cost more than the rows.)
constexpr int kRowBlocks = 7;

template <typename InT, typename OutT, int D, int U>
__global__ void __launch_bounds__(kRopeWarps * 32, kRowBlocks) rope_rows_kernel(const RopeRowsParams p) {
  constexpr int LPR = D / 8, HPW = 32 / LPR;   // lanes of a head, heads of a warp at once
  __shared__ float patch[kRopeWarps][32 * 8];
  __shared__ float s_gamma[2][D];
  grid_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lr = lane % LPR;
  const int n_heads = p.n_q_heads + p.n_kv_heads;
  const int h0 = (blockIdx.y * kRopeWarps + warp) * (HPW * U) + lane / LPR;
  int64_t r = blockIdx.x;
  int pos = __ldcg(p.pos + r);
  if (p.gamma_q != nullptr) {
    if (threadIdx.x < D) {
      s_gamma[0][threadIdx.x] = __ldcg(p.gamma_q + threadIdx.x);
      if (p.n_kv_heads > 0) s_gamma[1][threadIdx.x] = __ldcg(p.gamma_k + threadIdx.x);
    }
    __syncthreads();
  }
  const int half = p.rot_dim / 2;
  const bool by_vector = !p.interleaved && (half & 3) == 0;
  float* mine = patch[warp] + (lane / LPR) * D;
#pragma unroll 1
  for (; r < p.rows; r += gridDim.x) {
    float x[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * HPW;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[u][e] = 0.f;
      if (h < p.n_q_heads)
        Io<InT>::load(p.q, r * p.q_stride + static_cast<int64_t>(h) * D + lr * 8, x[u]);
      else if (h < n_heads)
        Io<InT>::load(p.k, r * p.k_stride + static_cast<int64_t>(h - p.n_q_heads) * D + lr * 8, x[u]);
    }
    if (pos < 0 || pos >= p.max_pos) {
      if (h0 == 0 && lr == 0) set_err(p.err, TTS_EFLAG_POS_RANGE);
      pos = min(max(pos, 0), p.max_pos - 1);
    }
    // entry e: its partner's index, and its own and its partner's factors (1, 0 past rot_dim)
    const float2* cs = p.cs + static_cast<int64_t>(pos) * half;
    if (r + gridDim.x < p.rows) pos = __ldcg(p.pos + r + gridDim.x);   // the next row's
    int partner[8];
    float fc[8], fs[8];
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      const int i0 = lr * 8 + j;
      if (by_vector) {
        // four neighbours turn alike: their partners and factors are vectors too
        const bool first = i0 < half, turns = i0 < p.rot_dim;
        partner[j] = !turns ? i0 : first ? i0 + half : i0 - half;
        float4 a = make_float4(1.f, 0.f, 1.f, 0.f), b = a;
        if (turns) {
          const float4* c4 = reinterpret_cast<const float4*>(cs + (first ? i0 : i0 - half));
          a = __ldcg(c4);
          b = __ldcg(c4 + 1);
        }
        const float sign = first ? -1.f : 1.f;   // t_a c - t_b s, t_b c + t_a s
        fc[j] = a.x; fc[j + 1] = a.z; fc[j + 2] = b.x; fc[j + 3] = b.z;
        fs[j] = a.y * sign; fs[j + 1] = a.w * sign; fs[j + 2] = b.y * sign; fs[j + 3] = b.w * sign;
      } else {
#pragma unroll
        for (int e = j; e < j + 4; ++e) {
          const int i = lr * 8 + e;
          const bool first = p.interleaved ? (i & 1) == 0 : i < half;
          partner[e] = i;
          fc[e] = 1.f;
          fs[e] = 0.f;
          if (i < p.rot_dim) {
            partner[e] = p.interleaved ? i ^ 1 : (first ? i + half : i - half);
            const float2 v = __ldcg(cs + (p.interleaved ? i >> 1 : (first ? i : i - half)));
            fc[e] = v.x;
            fs[e] = first ? -v.y : v.y;
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * HPW;
      float t[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = x[u][e];
      if (p.gamma_q != nullptr) {
        const float* gamma = s_gamma[h < p.n_q_heads ? 0 : 1];
        const float4 ga = *reinterpret_cast<const float4*>(gamma + 8 * lr), gb = *reinterpret_cast<const float4*>(gamma + 8 * lr + 4);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(t[e], t[e], ss);
#pragma unroll
        for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
        const float rn = inv_sqrt(ss * (1.0f / D) + p.eps);
        const float gm[8] = {ga.x, ga.y, ga.z, ga.w, gb.x, gb.y, gb.z, gb.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] *= rn * gm[e];
      }
      // pairs of neighbours are a lane's own; others come from the patch
      float pt[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) pt[e] = t[e ^ 1];
      if (!p.interleaved) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; j += 4)
          *reinterpret_cast<float4*>(mine + lr * 8 + j) = make_float4(t[j], t[j + 1], t[j + 2], t[j + 3]);
        __syncwarp();
        if (by_vector) {
#pragma unroll
          for (int j = 0; j < 8; j += 4) {
            const float4 v = *reinterpret_cast<const float4*>(mine + partner[j]);
            pt[j] = v.x; pt[j + 1] = v.y; pt[j + 2] = v.z; pt[j + 3] = v.w;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) pt[e] = mine[partner[e]];
        }
      }
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = lr * 8 + e < p.rot_dim ? fmaf(t[e], fc[e], pt[e] * fs[e]) : t[e];
      if (h < p.n_q_heads)
        Io<OutT>::store(p.q_out, r * p.q_out_stride + static_cast<int64_t>(h) * D + lr * 8, y);
      else if (h < n_heads)
        Io<OutT>::store(p.k_out, r * p.k_out_stride + static_cast<int64_t>(h - p.n_q_heads) * D + lr * 8, y);
    }
  }
}

template <typename InT, typename OutT, int D, int U>
cudaError_t launch_rows(const RopeRowsParams& p, cudaStream_t s) {
  constexpr int per = 32 / (D / 8) * U * kRopeWarps;   // heads of a block
  const int gy = (p.n_q_heads + p.n_kv_heads + per - 1) / per;
  const int64_t most = gy > kRowBlocks * p.n_sm ? 1 : kRowBlocks * p.n_sm / gy;
  const dim3 grid(static_cast<unsigned>(p.rows < most ? p.rows : most), gy);
  return launch_pdl(rope_rows_kernel<InT, OutT, D, U>, grid, dim3(kRopeWarps * 32), 0, s, p);
}
template <typename InT, typename OutT, int D>
cudaError_t launch_rows_u(const RopeRowsParams& p, cudaStream_t s) {
  // three heads a lane (at head_dim 128 a row of 24 heads is then one block) once one each would
  // give every SM over 16 warps
  const int64_t warps = static_cast<int64_t>(p.rows) * (p.n_q_heads + p.n_kv_heads) / (32 / (D / 8));
  return warps > static_cast<int64_t>(p.n_sm) * 16 ? launch_rows<InT, OutT, D, 3>(p, s)
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
// (p0 + kSide a + b) f as one product, rounded to f32 once.  32768 x 64: 13.8 us (21 with 64
// angles in double a block and frequency; its bytes need 2.5), mostly latency of pow and sincos.
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
