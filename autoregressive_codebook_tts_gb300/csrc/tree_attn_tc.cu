// Attention of a tree of drafted tokens over a bf16 or 8-bit cache, on the 5th-generation
// tensor cores (bf16 queries).
//
// An item's query rows (nodes times the q heads of the kv head) are the MMA's M = 128, the
// 128 cache rows of a tile its N.  With 32 or 64 rows to fill, the rows are there F = 4 or 2
// times over: replica f of a row owns columns [f 128 / F, (f + 1) 128 / F) of every tile and
// keeps its own softmax statistics and output row, so a thread has 128 / F scores a tile and
// no two threads ever exchange anything inside the loop.  Two softmax warpgroups take even
// and odd tiles, each with its own scores, statistics and output in tensor memory; so a row
// ends as 2 F partial rows, which meet once per item in shared memory.
//
//   S = Q K^T          exact products, f32 sums.  bf16 caches: bf16 operands.  8-bit caches: f16,
//                      which holds every code, and a bf16 row of q once it is scaled by a power
//                      of two; the K row's scale multiplies S.
//   P = 2^(S c - m)    f32, rounded to bf16 (8-bit caches: times V's row scale, to f16 in a unit
//                      that follows the row's largest such product) and written over S in tensor
//                      memory as the A operand of the second product
//   O += P V           V as the MN-major operand.  The maximum in use moves only when a row's
//                      grows by more than 2^8; then O is rescaled in tensor memory.
//
// Two loader warps (K, V) stream the cache with the TMA engine: a bf16 tile as tensor-map boxes
// (the whole tile, or one box per page and 64 columns) that land in the 128-byte swizzled layout
// of the MMA; an 8-bit tile as plain bulk copies into a staging tile, which four warps widen to
// f16 in the operand layout (f16 and not bf16: 1.4 against 2.5 operations an entry).  In tiles
// with node rows, V rows past the window are zeroed before their product (whatever a page holds
// there).  One warp issues both products of either group, whichever has its operands first.
//
// Traced before the one-pass softmax (cycles of one CTA's steady state, head_dim 128): a bf16 tile
// every 2120 (64 KB: 58 GB/s an SM, the HBM's share being 44) with few query rows; an int8 tile every 2650,
// set by the chain widening (650) - scores (650) - weights (1000) - output (600) of each group;
// with 128 rows the weights of a tile (4450: 128 a thread, traced after it) set 3650.  An item's end costs
// 3000 to 12000 more (query rows, partial rows, their merge), which the cut counts as two tiles, or
// as four and a half with 128 rows.  All roles' loops share the instruction cache: the step
// that rolled them (with one arrival a warp and elected issue) took int8 from 137 to 98 us.
// 32 streams of 1500..4000 rows, one node: bf16 66 us (5.4 TB/s, 0.81 of the measured copy rate),
// int8 69 us, e4m3 79 us; 63 nodes: bf16 95 us, int8 133 us, e4m3 137 us.
//
// The window is cut over one CTA per SM by cost (tree_plan.cuh).  Non-finite V entries of node
// rows are handled as in tree_attn.cu, those of committed rows behind the output passes.  Every wait is bounded; on expiry TTS_EFLAG_TIMEOUT is
// set and the CTA winds down.
#include <mutex>
#include <type_traits>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "tree_plan.cuh"

namespace tts {
namespace {

constexpr int kM = 128, kN = 128;
constexpr int kSmxThreads = 256, kWidenThreads = 128;
constexpr int kLoadWarp = 8, kMmaWarp = 10, kWidenWarp = 11;   // (a loader for K, one for V)
constexpr int kTmemCols = 512;            // S (P over it) 2 x 128, O 2 x 128

template <int D, typename KvT>
struct TcCfg {
  static constexpr bool k8 = CacheElem<KvT>::kScaled;
  static constexpr int kThreads = k8 ? 480 : 352;
  static constexpr int kTileBytes = kN * D * 2;                 // an operand tile
  static constexpr int kStages = k8 ? 2 : (D == 128 ? 3 : 5);   // operand tiles of K, and of V
  static constexpr int kRawBytes = k8 ? kN * D : 0;             // a staged 8-bit tile (K or V)
  static constexpr int kRaw = 2;                                // staged tiles of K, and of V
  static constexpr int kQBytes = 32768;                         // Q, and the epilogue's 256 x 32 f32
  static constexpr int kOffK = kQBytes, kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffRawK = kOffV + kStages * kTileBytes, kOffRawV = kOffRawK + kRaw * kRawBytes;
  static constexpr int kOffScale = kOffRawV + kRaw * kRawBytes; // [2][K, V][128] f32: scales of a tile's rows
  static constexpr int kOffQs = kOffScale + (k8 ? 2048 : 0);    // [128] f32: the power of two q was divided by
  static constexpr int kOffBar = kOffQs + (k8 ? 512 : 0);
  static constexpr int kOffNf = kOffBar + 320;                  // [D] f32, bf16: a column's non-finite V entries
  static constexpr size_t kSmem = kOffNf + (k8 ? 0 : D * 4);
};

__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFF) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFF) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);   // 128-byte swizzle
}

// Byte offset of 16-byte unit u of row r of a 128-row operand tile: chunks of 64 columns, 128
// bytes a row, unit u of a chunk's row at u ^ r % 8.
__device__ __forceinline__ uint32_t unit_off(int r, int u) {
  return static_cast<uint32_t>((u >> 3) * (kN * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// The products and their commits are issued by one elected lane of a converged warp, so every
// operand is warp-uniform (the instructions take uniform registers).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(smem_u32(bar)) : "memory");
}
// One arrival for a warp, after what all its lanes did before.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// A bounded wait of a converged warp, its outcome common to the lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(kFull, mbar_wait(bar, parity));
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr) : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      ::"r"(taddr), "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
        "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
        "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
        "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
        "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
        "r"(__float_as_uint(v[15])), "r"(__float_as_uint(v[16])), "r"(__float_as_uint(v[17])),
        "r"(__float_as_uint(v[18])), "r"(__float_as_uint(v[19])), "r"(__float_as_uint(v[20])),
        "r"(__float_as_uint(v[21])), "r"(__float_as_uint(v[22])), "r"(__float_as_uint(v[23])),
        "r"(__float_as_uint(v[24])), "r"(__float_as_uint(v[25])), "r"(__float_as_uint(v[26])),
        "r"(__float_as_uint(v[27])), "r"(__float_as_uint(v[28])), "r"(__float_as_uint(v[29])),
        "r"(__float_as_uint(v[30])), "r"(__float_as_uint(v[31]))
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr) : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A box of a tensor map at (column 0, row, 64-column chunk) into shared memory.
__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, int row, int chunk, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(chunk), "r"(smem_u32(bar)),
        "l"(policy)
      : "memory");
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds128a(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// Named barrier over the softmax threads, and the same with the AND of every thread's v.
__device__ __forceinline__ void smx_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool smx_sync_and(bool v) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\tsetp.ne.u32 pi, %1, 0;\n\t"
      "bar.red.and.pred po, 1, 256, pi;\n\tselp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(out) : "r"(static_cast<uint32_t>(v)) : "memory");
  return out != 0;
}

// 16 codes as 16 f16 values (two 16-byte units), exactly.  int8: with 128 added, a code is the low
// byte of the f16 number 1024 + code + 128.
template <typename KvT>
__device__ __forceinline__ void widen16(const uint4 v, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<KvT, CodeI8>::value) {
      const uint32_t u = w[i] ^ 0x80808080u, off = 0x64806480u;   // 1152
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t x = __byte_perm(u, 0x64646464u, k == 0 ? 0x4140 : 0x4342);
        const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&off));
        o[2 * i + k] = *reinterpret_cast<const uint32_t*>(&r);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i] >> (16 * k)), __NV_E4M3);
        o[2 * i + k] = static_cast<uint32_t>(r.x) | (static_cast<uint32_t>(r.y) << 16);
      }
    }
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// Replaces the non-finite ones of eight 16-bit values by 0 (kExp: the exponent bits of their
// type); whether there were any.
template <uint32_t kExp>
__device__ __forceinline__ bool clear_nonfinite(uint4& v) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w}, hit = 0;
  // (all exponent bits set: one more at their lowest place carries into the sign's)
  constexpr uint32_t both = kExp | (kExp << 16), one = both & ~(both << 1);
#pragma unroll
  for (int i = 0; i < 4; ++i) hit |= (w[i] & both) + one;
  if ((hit & 0x80008000u) == 0) return false;
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & kExp) == kExp) {
      any = true;
      w[i] &= 0xffff0000u;
    }
    if ((w[i] & (kExp << 16)) == (kExp << 16)) {
      any = true;
      w[i] &= 0x0000ffffu;
    }
  }
  v = make_uint4(w[0], w[1], w[2], w[3]);
  return any;
}

// Every tile of a CTA's pieces, in order.
struct TileWalk {
  PieceWalk walk;
  Piece it;
  int tile, piece;
  bool have;
  __device__ __forceinline__ void init(const TreeParams& p, int cta) {
    walk.init(p, cta);
    piece = 0;
    have = walk.get(p, it);
    tile = it.t0;
  }
  __device__ __forceinline__ void next(const TreeParams& p) {
    if (++tile >= it.t1) {
      have = walk.get(p, it);
      tile = it.t0;
      ++piece;
    }
  }
};

// Which of 32 columns a row sees, the first at node offset off (below 0: committed rows).
__device__ __forceinline__ uint32_t visible32(int off, uint64_t see) {
  if (off >= 64) return 0u;
  if (off >= 0) return static_cast<uint32_t>(see >> off);
  if (off > -32) return static_cast<uint32_t>(see << -off) | ((1u << -off) - 1u);
  return ~0u;
}

// 32 scores of a row from tensor memory: times the columns' K scales (8-bit), -inf where the row
// does not see the column.
template <bool k8>
__device__ __forceinline__ void load_scores(uint32_t taddr, const float* ksc, bool masked, uint32_t vis, float (&s)[32]) {
  tmem_ld32(taddr, s);
  if constexpr (k8) {
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      const float4 k = *reinterpret_cast<const float4*>(ksc + e);
      const float2 a = __fmul2_rn(make_float2(s[e], s[e + 1]), make_float2(k.x, k.y));
      const float2 b = __fmul2_rn(make_float2(s[e + 2], s[e + 3]), make_float2(k.z, k.w));
      s[e] = a.x; s[e + 1] = a.y; s[e + 2] = b.x; s[e + 3] = b.y;
    }
  }
  if (masked) {
#pragma unroll
    for (int e = 0; e < 32; ++e) s[e] = (vis >> e) & 1u ? s[e] : -INFINITY;
  }
}

__device__ __forceinline__ float max32(const float (&s)[32]) {
  float z[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) z[e] = fmaxf(s[e], s[e + 16]);
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1)
#pragma unroll
    for (int e = 0; e < o; ++e) z[e] = fmaxf(z[e], z[e + o]);
  return z[0];
}

// The weights 2^(s c - ms) of 32 columns, packed to 16 bits (8-bit caches: f16, times the
// columns' V scales and g; else bf16), and their unrounded sum (without the scales).  `top`
// (8-bit): the largest magnitude packed; infinity when one does not fit.
template <bool k8>
__device__ __forceinline__ float weights(const float (&s)[32], const float* vsc, float g, float c, float ms,
                                         uint32_t (&pk)[16], float& top) {
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  const float2 neg = make_float2(-ms, -ms), c2 = make_float2(c, c), g2 = make_float2(g, g);
  __half2 t2[2] = {__half2half2(__ushort_as_half(0)), __half2half2(__ushort_as_half(0))};
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    float2 a = __ffma2_rn(make_float2(s[e], s[e + 1]), c2, neg);
    float2 b = __ffma2_rn(make_float2(s[e + 2], s[e + 3]), c2, neg);
    a.x = ex2(a.x); a.y = ex2(a.y); b.x = ex2(b.x); b.y = ex2(b.y);
    sum[0] = __fadd2_rn(sum[0], a);
    sum[1] = __fadd2_rn(sum[1], b);
    if constexpr (k8) {
      // (weight times scale first: a weight of 0 stays 0 whatever finite scale it meets)
      const float4 v = *reinterpret_cast<const float4*>(vsc + e);
      a = __fmul2_rn(__fmul2_rn(a, make_float2(v.x, v.y)), g2);
      b = __fmul2_rn(__fmul2_rn(b, make_float2(v.z, v.w)), g2);
      const __half2 x = __floats2half2_rn(a.x, a.y), y = __floats2half2_rn(b.x, b.y);
      t2[0] = __hmax2(t2[0], __habs2(x));
      t2[1] = __hmax2(t2[1], __habs2(y));
      pk[e / 2] = *reinterpret_cast<const uint32_t*>(&x);
      pk[e / 2 + 1] = *reinterpret_cast<const uint32_t*>(&y);
    } else {
      const __nv_bfloat162 x = __floats2bfloat162_rn(a.x, a.y), y = __floats2bfloat162_rn(b.x, b.y);
      pk[e / 2] = *reinterpret_cast<const uint32_t*>(&x);
      pk[e / 2 + 1] = *reinterpret_cast<const uint32_t*>(&y);
    }
  }
  if constexpr (k8) {
    const float2 t = __half22float2(__hmax2(t2[0], t2[1]));
    top = fmaxf(t.x, t.y);
  }
  const float2 t = __fadd2_rn(sum[0], sum[1]);
  return t.x + t.y;
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// The same weights times V scales once more, when the unit 2^(ve - 127) no longer suits them: the
// largest product so far (`top` units, before these 32) or of these is to be 2^6 to 2^7 units.
// Returns the power of two that what was summed in the old unit is to be multiplied by.
__device__ __forceinline__ int weights_in_new_unit(const float (&s)[32], const float* vsc, float c, float ms, int& ve,
                                                   float& top, uint32_t (&pk)[16]) {
  // 2^9 down, so that no weight (up to 2^8) times a finite scale overflows; what is not finite does
  // not choose the unit
  float x[32], most = 0.f;
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    x[e] = ex2(fmaf(s[e], c, -ms)) * pow2(-9) * vsc[e];
    const float a = fabsf(x[e]);
    most = fmaxf(most, a < INFINITY ? a : 0.f);
  }
  const auto exponent = [](float a) { return static_cast<int>(__float_as_uint(a) >> 23) - 127; };
  const int old = ve;
  int e = -1000;
  if (top > 0.f) e = exponent(top) + ve - 127;
  if (most > 0.f) e = max(e, exponent(most) + 9);
  const int at = e + 127 - ve;   // the exponent of the largest in units
  if (e > -1000 && (at < 0 || at > 14)) ve = min(max(e + 121, 10), 253);
  const int up = old - ve;
  const float g = pow2(136 - ve);
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const __half2 h = __floats2half2_rn(x[2 * k] * g, x[2 * k + 1] * g);
    pk[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  top = fmaxf(top * pow2(up / 2) * pow2(up - up / 2), most * g);
  return up;
}

// A packed pair of weights times a and b (rounded once more: only weights of a tile whose maximum
// or unit moved after they were written).
template <bool k8>
__device__ __forceinline__ uint32_t scale_pair(uint32_t w, float a, float b) {
  if constexpr (k8) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w));
    const __half2 y = __floats2half2_rn(x.x * a * b, x.y * a * b);
    return *reinterpret_cast<const uint32_t*>(&y);
  } else {
    const __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(w << 16) * a, __uint_as_float(w & 0xffff0000u) * a);
    (void)b;
    return *reinterpret_cast<const uint32_t*>(&y);
  }
}

// 2^(m - M) of a partial row; one that saw nothing has weight 0, one that only saw NaN scores
// (which no maximum holds) passes its NaN on.
__device__ __forceinline__ float partial_weight(float m, float l, float M) {
  return m == -INFINITY ? (l != l ? 1.f : 0.f) : ex2(m - M);
}

// The non-finite ones among entries [col, col + 4) of the V rows of the nodes in `bits`, added up.
template <typename KvT, int D>
__device__ __forceinline__ float4 bad_v_sum(const CacheView& c, int b, int g, int past, unsigned long long bits, int col) {
  float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  while (bits != 0) {
    const int u = __ffsll(static_cast<long long>(bits)) - 1;
    bits &= bits - 1;
    const int pos = past + u, page = c.paged ? max(cache_page(c, b, pos), 0) : 0;
    const int64_t row = cache_row(c, b, g, pos, page);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float x;
      if constexpr (CacheElem<KvT>::kScaled) {
        const uint32_t code = static_cast<const uint8_t*>(c.v)[row * D + col + e];
        x = (std::is_same<KvT, CodeI8>::value ? I8Code::value(code) : E4m3Code::value(code)) * c.v_scale[row];
      } else
        x = static_cast<float>(static_cast<const __nv_bfloat16*>(c.v)[row * D + col + e]);
      if ((__float_as_uint(x) & 0x7f800000u) == 0x7f800000u) a[e] += x;
    }
  }
  return make_float4(a[0], a[1], a[2], a[3]);
}

// Adds up the non-finite V entries of the piece's committed rows, by column, into nf [D] (zeros
// before): by the softmax threads, 16 bytes of a row each.
template <int D>
__device__ __forceinline__ void nonfinite_columns(const TreeParams& p, const Piece& it, int tid, float* nf) {
  constexpr int UR = D / 8, STEP = kSmxThreads / UR;
  const CacheView& c = p.cache;
  const int u = tid % UR, end = min(it.t1 * kN, it.w.past);
  float sum[8] = {};
#pragma unroll 4
  for (int j = it.t0 * kN + tid / UR; j < end; j += STEP) {
    const int page = c.paged ? max(cache_page(c, it.b, j), 0) : 0;
    const int64_t row = cache_row(c, it.b, it.g, j, page);
    float x[8];
    unpack_bf16x8(__ldcg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(c.v) + row * D) + u), x);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if ((__float_as_uint(x[e]) & 0x7f800000u) == 0x7f800000u) sum[e] += x[e];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (sum[e] != 0.f) atomicAdd(nf + u * 8 + e, sum[e]);   // (infinities and NaN: in any order)
}

// One tile of K or V into `dst`, by a whole warp: bf16 in the operand layout (boxes of the
// tensor map), 8-bit as it lies (bulk copies).  Rows past the window are not asked for, but for
// the rest of a box.  `page` is the lane's entry of the tile's pages (lane pages apart).
template <int D, typename KvT>
__device__ __forceinline__ void load_tile(const TreeParams& p, const CUtensorMap* map, const unsigned char* base,
                                          const Piece& it, int r0, int lane, unsigned char* dst, uint64_t* bar,
                                          uint64_t policy) {
  constexpr bool k8 = CacheElem<KvT>::kScaled;
  const CacheView& c = p.cache;
  const int n = min(kN, it.w.past + it.w.nodes - r0);   // rows of the window in the tile
  const int ps = 1 << c.page_shift;
  if (!c.paged || ps >= kN) {
    if (lane == 0) {
      int page = 0;
      if (c.paged) {
        page = cache_page(c, it.b, r0);
        if (page < 0) {
          set_err(p.err, TTS_EFLAG_PAGE);
          page = 0;
        }
      }
      const int64_t row = cache_row(c, it.b, it.g, r0, page);
      if constexpr (k8) {
        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(n * D));
        bulk_g2s(dst, base + row * D, static_cast<uint32_t>(n * D), bar, policy);
      } else {
        mbar_arrive_expect_tx(bar, kN * D * 2);
        tma_box(dst, map, static_cast<int>(row), 0, bar, policy);
      }
    }
    return;
  }
  const int pages = (n + ps - 1) >> c.page_shift;
  if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>((k8 ? n : pages << c.page_shift) * D * (k8 ? 1 : 2)));
  __syncwarp();
  for (int i = lane; i < pages; i += 32) {
    const int pos = r0 + (i << c.page_shift);
    int page = cache_page(c, it.b, pos);
    if (page < 0) {
      set_err(p.err, TTS_EFLAG_PAGE);
      page = 0;
    }
    const int64_t row = cache_row(c, it.b, it.g, pos, page);
    if constexpr (k8) {
      const int rows = min(ps, n - (i << c.page_shift));
      bulk_g2s(dst + (i << c.page_shift) * D, base + row * D, static_cast<uint32_t>(rows * D), bar, policy);
    } else {
#pragma unroll
      for (int ch = 0; ch < D / 64; ++ch)
        tma_box(dst + ch * (kN * 128) + (i << c.page_shift) * 128, map, static_cast<int>(row), ch, bar, policy);
    }
  }
}

// 128 x D codes of a staged tile to f16 in the operand layout, by the widening threads: four
// 16-code vectors of a thread at a time.  Which thread takes which vector: a phase's eight lanes
// read from every bank once, and what they write lies in eight different bank groups (the even
// units of an even row and the odd places they take in an odd one).
template <int D, typename KvT>
__device__ __forceinline__ void widen_tile(const unsigned char* raw, unsigned char* dst, int wt) {
  constexpr int UR = D / 16, STEP = kWidenThreads / UR, NR = kN / STEP, BATCH = 4;
  const int half = (wt >> 2) & 1;
  const int u = D == 128 ? half * 4 + (wt & 3) : wt & 3;
  const int row0 = D == 128 ? (wt >> 4) * 2 + (half ^ ((wt >> 3) & 1)) : wt >> 2;
  const unsigned char* src = raw + row0 * D + u * 16;
  // (rows are STEP, a multiple of eight, apart: the swizzle is the same for all of them)
  unsigned char* lo_at = dst + unit_off(row0, 2 * u);
  unsigned char* hi_at = dst + unit_off(row0, 2 * u + 1);
  // (rolled: the roles' loops together have to stay in the instruction cache)
#pragma unroll 1
  for (int i0 = 0; i0 < NR; i0 += BATCH) {
    uint4 x[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) x[i] = *reinterpret_cast<const uint4*>(src + (i0 + i) * (STEP * D));
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      uint4 lo, hi;
      widen16<KvT>(x[i], lo, hi);
      *reinterpret_cast<uint4*>(lo_at + (i0 + i) * (STEP * 128)) = lo;
      *reinterpret_cast<uint4*>(hi_at + (i0 + i) * (STEP * 128)) = hi;
    }
  }
}

template <int D, typename KvT, int F>
__global__ void __launch_bounds__(TcCfg<D, KvT>::kThreads, 1)
    tree_attn_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const TreeParams p) {
  using C = TcCfg<D, KvT>;
  constexpr bool k8 = C::k8;
  constexpr int NS = C::kStages;
  constexpr int RP = kM / F;        // query rows of an item (padded)
  constexpr int W = kN / F;         // columns a replica owns
  constexpr int UR = D / 8;         // 16-byte units of a bf16 row
  extern __shared__ __align__(1024) unsigned char smem[];
  float* stage = reinterpret_cast<float*>(smem);                          // epilogue: [256][32]
  float* s_scale = reinterpret_cast<float*>(smem + C::kOffScale);         // [2][2][128]
  float* s_qs = reinterpret_cast<float*>(smem + C::kOffQs);               // [128]
  float* s_nf = reinterpret_cast<float*>(smem + C::kOffNf);               // [D]
  uint64_t* fullK = reinterpret_cast<uint64_t*>(smem + C::kOffBar);       // [NS] operand tile written
  uint64_t* emptyK = fullK + NS;                                          // [NS] its product done
  uint64_t* fullV = emptyK + NS;
  uint64_t* emptyV = fullV + NS;
  uint64_t* rawK = emptyV + NS;                                           // [2] staged 8-bit tile landed
  uint64_t* rawKe = rawK + 2;                                             // [2] and widened
  uint64_t* rawV = rawKe + 2;
  uint64_t* rawVe = rawV + 2;
  uint64_t* qready = rawVe + 2;                                           // the piece's query rows written, O free
  uint64_t* sready = qready + 1;                                          // [2] S of the group's tile (and its scales)
  uint64_t* pready = sready + 2;                                          // [2] P written, O rescaled
  uint64_t* odone = pready + 2;                                           // [2] the group's last product of a piece
  uint64_t* scfree = odone + 2;                                           // [2] scales of the slot's tile used
  uint64_t* drained = scfree + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drained + 1);
  unsigned long long* s_bad = reinterpret_cast<unsigned long long*>(drained + 2);   // node rows with non-finite V
  static_assert((4 * NS + 8 + 1 + 6 + 2 + 2 + 1) * 8 <= 320, "barrier area");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&fullK[s], k8 ? kWidenThreads / 32 : 1);   // (arrivals are one a warp)
      mbar_init(&emptyK[s], 1);
      mbar_init(&fullV[s], k8 ? kWidenThreads / 32 : 1);
      mbar_init(&emptyV[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&rawK[i], 1);
      mbar_init(&rawKe[i], kWidenThreads / 32);
      mbar_init(&rawV[i], 1);
      mbar_init(&rawVe[i], kWidenThreads / 32);
    }
    mbar_init(qready, kSmxThreads / 32);
    for (int i = 0; i < 2; ++i) {
      // the products' commit, and the issuer's own arrival, which passes on what it has seen
      // of the widening threads' plain stores (the scales)
      mbar_init(&sready[i], 2);
      mbar_init(&pready[i], 4);
      mbar_init(&odone[i], 1);
      mbar_init(&scfree[i], 4);
    }
    mbar_init(drained, 1);
    *s_bad = 0;
    mbar_init_fence();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_u32(s_tmem)), "n"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const uint32_t tO = tmem + 2 * kN;
  grid_wait();
  grid_launch_dependents();

  if (warp == kLoadWarp || warp == kLoadWarp + 1) {
    // ----------------------------------------------------------------- loaders
    // K and V stream side by side: a K tile is free once its scores are done, a V tile one
    // softmax later
    const bool is_v = warp != kLoadWarp;
    constexpr int NL = k8 ? C::kRaw : NS;   // tiles of the ring that they fill
    constexpr int bytes = k8 ? C::kRawBytes : C::kTileBytes;
    unsigned char* ring = smem + (k8 ? (is_v ? C::kOffRawV : C::kOffRawK) : (is_v ? C::kOffV : C::kOffK));
    uint64_t* full = k8 ? (is_v ? rawV : rawK) : (is_v ? fullV : fullK);
    uint64_t* empty = k8 ? (is_v ? rawVe : rawKe) : (is_v ? emptyV : emptyK);
    const unsigned char* cache = static_cast<const unsigned char*>(is_v ? p.cache.v : p.cache.k);
    const CUtensorMap* map = is_v ? &vmap : &kmap;
    const uint64_t policy = l2_evict_first_policy();
    TileWalk w;
    w.init(p, blockIdx.x);
    bool ok = true;
    int n = 0;
    for (; w.have; w.next(p)) {
      const int s = n % NL;
      if (n >= NL && !warp_wait(&empty[s], static_cast<uint32_t>(n / NL - 1) & 1u)) {
        ok = false;
        break;
      }
      load_tile<D, KvT>(p, map, cache, w.it, w.tile * kN, lane, ring + s * bytes, &full[s], policy);
      ++n;
    }
    if (!ok && lane == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
    // every copy still in flight lands before the CTA ends (earlier ones were consumed)
    for (int t = max(0, n - NL); t < n; ++t) mbar_wait(&full[t % NL], static_cast<uint32_t>(t / NL) & 1u);
  } else if (k8 && warp >= kWidenWarp) {
    // ----------------------------------------------------------------- widening
    if constexpr (k8) {
      const int wt = tid - kWidenWarp * 32;
      const CacheView& c = p.cache;
      TileWalk w;
      w.init(p, blockIdx.x);
      // the scales of row wt of the next tile, 0 past the window
      float ks = 0.f, vs = 0.f;
      bool node = false;
      auto scales = [&]() {
        const int pos = w.tile * kN + wt;
        ks = vs = 0.f;
        node = false;
        if (w.have && pos < w.it.w.past + w.it.w.nodes) {
          const int page = c.paged ? max(cache_page(c, w.it.b, pos), 0) : 0;
          const int64_t row = cache_row(c, w.it.b, w.it.g, pos, page);
          ks = __ldcg(c.k_scale + row);
          vs = __ldcg(c.v_scale + row);
          node = pos >= w.it.w.past;
        }
      };
      scales();
      bool ok = true;
      for (int t = 0; w.have; ++t) {
        const int s = t & 1;
        const uint32_t ph = static_cast<uint32_t>(t >> 1) & 1u;
        // a node row's non-finite V scale may not meet the weight 0 of the rows that do not see it
        // (the epilogue adds it to those that do)
        const float k = ks, v = node && (__float_as_uint(vs) & 0x7f800000u) == 0x7f800000u ? 0.f : vs;
        w.next(p);
        scales();   // in flight while this tile is widened
        // K's operand tile is free once the scores of tile t - 2 are done, the scales' slot once its
        // weights are, V's operand tile once its product is
        if ((t >= 2 && (!warp_wait(&emptyK[s], ph ^ 1u) || !warp_wait(&scfree[s], ph ^ 1u))) || !warp_wait(&rawK[s], ph)) {
          ok = false;
          break;
        }
        s_scale[s * 256 + wt] = k;
        s_scale[s * 256 + 128 + wt] = v;
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {   // K, then V
          if (x == 1 && (!warp_wait(&rawV[s], ph) || (t >= 2 && !warp_wait(&emptyV[s], ph ^ 1u)))) {
            ok = false;
            break;
          }
          widen_tile<D, KvT>(smem + (x ? C::kOffRawV : C::kOffRawK) + s * C::kRawBytes,
                             smem + (x ? C::kOffV : C::kOffK) + s * C::kTileBytes, wt);
          fence_async_smem();
          warp_arrive(x ? &fullV[s] : &fullK[s]);
          warp_arrive(x ? &rawVe[s] : &rawKe[s]);
        }
        if (!ok) break;
      }
      if (!ok && lane == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
    }
  } else if (warp == kMmaWarp) {
    // -------------------------------------------------------------- MMA issuer
    PieceWalk walk;
    walk.init(p, blockIdx.x);
    {
      // kind::f16, f32 accumulator, A and B bf16 (over 8-bit caches f16), M = 128; S: N = 128, B (K)
      // K-major; O: N = D, B (V) MN-major (bit 16)
      constexpr uint32_t type = k8 ? 0u : 1u;
      constexpr uint32_t base = (1u << 4) | (type << 7) | (type << 10) | ((kM >> 4) << 24);
      constexpr uint32_t idS = base | ((kN >> 3) << 17), idO = base | (1u << 16) | ((D >> 3) << 17);
      const uint64_t qd = smem_desc(smem_u32(smem), 16, 1024);
      const uint64_t kd0 = smem_desc(smem_u32(smem + C::kOffK), 16, 1024);
      const uint64_t vd0 = smem_desc(smem_u32(smem + C::kOffV), kN * 128, 1024);
      int ks = 0, vs = 0;                 // next K and V operand tiles
      uint32_t kph = 0, vph = 0, pph[2] = {0, 0};
      bool ok = true;
      auto issue_s = [&](int wg) {
        tc_fence_after();
        const uint64_t kd = kd0 + static_cast<uint64_t>(ks * (C::kTileBytes >> 4));
        const uint32_t d = tmem + wg * kN;
        // (rolled, as all loops here: see widen_tile)
#pragma unroll 1
        for (int j = 0; j < D / 16; ++j) {
          const uint32_t o = (j >> 2) * (kN * 128 >> 4) + (j & 3) * 2;
          mma_ss(d, qd + o, kd + o, idS, j);
        }
        mma_commit(&sready[wg]);
        mma_commit(&emptyK[ks]);
        warp_arrive(&sready[wg]);
        if (++ks == NS) {
          ks = 0;
          kph ^= 1u;
        }
      };
      auto issue_pv = [&](int i, bool last) {
        const int wg = i & 1;
        pph[wg] ^= 1u;
        tc_fence_after();
        const uint64_t vd = vd0 + static_cast<uint64_t>(vs * (C::kTileBytes >> 4));
        const uint32_t a = tmem + wg * kN, d = tO + wg * D;
#pragma unroll 1
        for (int j = 0; j < kN / 16; ++j) mma_ts(d, a + j * 8, vd + j * (2048 >> 4), idO, i > 1 ? 1 : j);
        mma_commit(&emptyV[vs]);
        if (last) mma_commit(&odone[wg]);
        if (++vs == NS) {
          vs = 0;
          vph ^= 1u;
        }
      };
      auto ready = [&](uint64_t* bar, uint32_t parity) { return __all_sync(kFull, mbar_try_wait(bar, parity)); };
      Piece it;
      for (uint32_t piece = 0; ok && walk.get(p, it); ++piece) {
        const int n = it.t1 - it.t0;
        ok = warp_wait(qready, piece & 1u);
        // tile ns's scores go out once K is there and the product that read its tensor memory has
        // been issued, tile np's product once P and V are: whichever is ready first
        int ns = 0, np = 0;
        long long start = clock64();
        while (ok && np < n) {
          if (ns < n && ns < np + 2 && ready(&fullK[ks], kph)) {
            issue_s(ns & 1);
            ++ns;
            start = clock64();
          } else if (np < ns && ready(&pready[np & 1], pph[np & 1]) && ready(&fullV[vs], vph)) {
            issue_pv(np, np + 2 >= n);
            ++np;
            start = clock64();
          } else {
            ok = __all_sync(kFull, clock64() - start <= kWaitLimitCycles);
          }
        }
      }
      // no product is in flight when the CTA gives its tensor memory back
      mma_commit(drained);
      if (!warp_wait(drained, 0)) ok = false;
      if (!ok && lane == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
    }
  } else {
    // ---------------------------------------------------------- softmax warps
    const int wg = warp >> 2;
    const int r = (warp & 3) * 32 + lane;        // row of the MMA = TMEM lane
    const int f = r / RP, rr = r % RP;           // replica (uniform in a warp), query row
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + wg * kN + lane_base, tOw = tO + wg * D + lane_base;
    // a negative scale turns q round; a scale of 0 (equal weights) may not meet -inf scores
    const float c = fmaxf(fabsf(p.scale_log2), 1e-30f);
    const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    const int gs = p.group >> 1;   // log2 of the group (1, 2 or 4)
    PieceWalk walk;
    walk.init(p, blockIdx.x);
    if (blockIdx.x == 0 && p.err != nullptr) {
      bool any = false;
      for (int b = tid; b < p.cache.B; b += kSmxThreads) {
        bool bad;
        tree_window(p, b, &bad);
        any = any || bad;
      }
      if (any) set_err(p.err, TTS_EFLAG_NVALID);
    }
    uint32_t sph = 0, oph = 0;
    int taken = 0;   // tiles of the pieces before
    bool ok = true;
    // a piece's query rows, loaded while the piece before is finished: 16-byte units
    // tid, tid + 256, ... of its RP rows; rows without a node are 0
    constexpr int QU = RP * UR / kSmxThreads;
    uint4 qv[QU];
    auto load_q = [&](const Piece& x) {
#pragma unroll
      for (int k = 0; k < QU; ++k) {
        const int i = tid + k * kSmxThreads, row = i / UR, u = i % UR, q = x.rb * RP + row, t = q >> gs,
                  h = q & (p.group - 1);
        qv[k] = make_uint4(0, 0, 0, 0);
        if (t < x.w.nodes)
          qv[k] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                        (static_cast<int64_t>(x.b) * p.T + t) * p.q_stride +
                                                        (x.g * p.group + h) * D) + u);
      }
    };
    Piece it, next;
    bool have = walk.get(p, next);
    if (have) load_q(next);
    while (have) {
      it = next;
      const int first = it.rb * RP;   // of the stream and kv head's query rows
      // each query row F times; over 8-bit caches as f16, times the power of two that takes its
      // largest entry to [2^14, 2^15) (bf16's eight bits are exact there down to 2^-28 of that)
#pragma unroll
      for (int k = 0; k < QU; ++k) {
        const int i = tid + k * kSmxThreads, row = i / UR, u = i % UR;
        uint4 v = make_uint4(qv[k].x ^ flip, qv[k].y ^ flip, qv[k].z ^ flip, qv[k].w ^ flip);
        if constexpr (k8) {
          uint32_t w[4] = {v.x, v.y, v.z, v.w}, top = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
#pragma unroll
          for (int o = UR / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
          const int up = min(141 - static_cast<int>(top >> 7), 126);   // (at least -114)
          const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __half2 h = __floats2half2_rn(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xffff0000u) * f);
            w[e] = *reinterpret_cast<const uint32_t*>(&h);
          }
          v = make_uint4(w[0], w[1], w[2], w[3]);
          if (u == 0) s_qs[row] = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
        }
#pragma unroll
        for (int x = 0; x < F; ++x) *reinterpret_cast<uint4*>(smem + unit_off(x * RP + row, u)) = v;
      }
      fence_async_smem();
      tc_fence_before();
      warp_arrive(qready);
      const int node = (first + rr) >> gs;
      const uint64_t see = node < it.w.nodes ? seen_nodes(p, it.b, node, it.w.nodes) : 0ull;
      const int n = it.t1 - it.t0;
      // the V scale of node tid, where the piece holds its row
      float node_scale = 0.f;
      if (k8 && tid < it.w.nodes && it.w.past + tid >= it.t0 * kN && it.w.past + tid < it.t1 * kN) {
        const CacheView& cv = p.cache;
        const int pos = it.w.past + tid, page = cv.paged ? max(cache_page(cv, it.b, pos), 0) : 0;
        node_scale = __ldcg(cv.v_scale + cache_row(cv, it.b, it.g, pos, page));
      }
      float m = -INFINITY, l = 0.f;
      // (8-bit) P and O are in units of 2^(ve - 127), at first 2^-12: rows of deviation 1 have V scales
      // of about 2^-5 (int8) and 2^-7 (e4m3); `top`: the largest product so far, in that unit
      int ve = 115;
      float top = 0.f;
      for (int i = wg; ok && i < n; i += 2) {
        const int base = (it.t0 + i) * kN + f * W;   // position of this thread's first column
        const bool masked = (it.t0 + i) * kN + kN > it.w.past;
        if (!warp_wait(&sready[wg], sph)) {
          ok = false;
          break;
        }
        sph ^= 1u;
        tc_fence_after();
        // the scales of this thread's columns (8-bit): the slot is the operand stage of the tile
        const int slot = (taken + i) & 1;
        const float* ksc = s_scale + (slot * 256 + f * W);
        const float* vsc = ksc + 128;
        const int off = base - it.w.past, node_row = off - f * W + r;   // (of row r of the tile)
        // (kept off 0: scores of -inf times it)
        const float cr = k8 ? fmaxf(c * s_qs[rr], 1e-37f) : c;
        // chunks of 32 columns, P over S (a chunk's 16 packed columns lie below every S column
        // still to be read).  A chunk that moves the maximum or the unit rescales O and the chunks
        // before it.
#pragma unroll 1
        for (int cc = 0; cc < W / 32; ++cc) {
          float sv[32];
          const uint32_t vis = masked ? visible32(off + 32 * cc, see) : ~0u;
          load_scores<k8>(tS + f * W + 32 * cc, ksc + 32 * cc, masked, vis, sv);
          float mx = max32(sv);
          if (mx > -INFINITY) mx *= cr;
          const bool move = mx > m + 8.0f;
          const float alpha = move && m > -INFINITY ? ex2(m - mx) : 1.0f;
          if (move) {
            l *= alpha;
            m = mx;
          }
          const float ms = m == -INFINITY ? 0.f : m;
          uint32_t pk[16];
          float now = 0.f;
          l += weights<k8>(sv, vsc + 32 * cc, pow2(127 - ve), cr, ms, pk, now);
          int up = 0;   // O's unit changes by 2^-up
          if constexpr (k8) {
            // The unit follows the largest product of weight and V scale of what this row sees: the
            // largest so far stays between 1 and f16's 65504 of it, so that products are lost
            // (rounded to 0) only below 2^-25 of that, and mostly below 2^-31.  Rows that are not
            // seen, or of no weight, do not matter whatever their scale.
            top *= alpha;
            const bool off_unit = !(now < INFINITY) || (fmaxf(top, now) < 1.0f && mx > -INFINITY);
            if (__any_sync(kFull, off_unit)) {
              load_scores<k8>(tS + f * W + 32 * cc, ksc + 32 * cc, masked, vis, sv);
              if (off_unit) up = weights_in_new_unit(sv, vsc + 32 * cc, cr, ms, ve, top, pk);
            }
            if (!off_unit) top = fmaxf(top, now);
          }
          if (__any_sync(kFull, alpha != 1.0f || up != 0)) {
            const float a = alpha * pow2(up / 2), b = pow2(up - up / 2);
            if (i > 1) {
              // O is complete up to the group's tile before: its product was issued before S
#pragma unroll 1
              for (int k = 0; k < D / 32; ++k) {
                float o[32];
                tmem_ld32(tOw + 32 * k, o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = k8 ? o[e] * a * b : o[e] * a;
                tmem_st32(tOw + 32 * k, o);
              }
            }
            if (cc > 0) {
              tmem_wait_st();
#pragma unroll 1
              for (int k = 0; k < cc; ++k) {
                uint32_t old[16];
                tmem_ld16(tS + f * (W / 2) + 16 * k, old);
#pragma unroll
                for (int e = 0; e < 16; ++e) old[e] = scale_pair<k8>(old[e], a, b);
                tmem_st16(tS + f * (W / 2) + 16 * k, old);
              }
            }
          }
          tmem_st16(tS + f * (W / 2) + 16 * cc, pk);
        }
        if constexpr (k8) warp_arrive(&scfree[slot]);
        if (F > 1) {
          // the columns of the other replicas
          const uint32_t zero[16] = {};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k / (4 / F) != f) tmem_st16(tS + 16 * k, zero);
        }
        tmem_wait_st();
        if constexpr (!std::is_same<KvT, CodeI8>::value) {
          // V's node rows: non-finite entries are noted and cleared, rows past the window (which
          // the copies left as they were, or filled from the page) zeroed.  Widened int8 is
          // finite whatever the staging tile held.
          if (masked) {
            const int s = (taken + i) % NS;
            if (!warp_wait(&fullV[s], static_cast<uint32_t>((taken + i) / NS) & 1u)) {
              ok = false;
              break;
            }
            if (node_row >= 0) {
              unsigned char* vt = smem + C::kOffV + s * C::kTileBytes;
              bool any = false;
              if (node_row >= it.w.nodes) {
#pragma unroll 4
                for (int u = 0; u < UR; ++u) *reinterpret_cast<uint4*>(vt + unit_off(r, u)) = make_uint4(0, 0, 0, 0);
              } else {
#pragma unroll 1
                for (int u0 = 0; u0 < UR; u0 += 4) {
                  uint4 x[4];
#pragma unroll
                  for (int u = 0; u < 4; ++u) x[u] = *reinterpret_cast<const uint4*>(vt + unit_off(r, u0 + u));
#pragma unroll
                  for (int u = 0; u < 4; ++u)
                    if (clear_nonfinite<k8 ? 0x7c00u : 0x7f80u>(x[u])) {
                      any = true;
                      *reinterpret_cast<uint4*>(vt + unit_off(r, u0 + u)) = x[u];
                    }
                }
              }
              if (any) atomicOr(s_bad, 1ull << node_row);
            }
            fence_async_smem();
          }
        }
        tc_fence_before();
        warp_arrive(&pready[wg]);
      }
      taken += n;
      have = walk.get(p, next);
      if (have) load_q(next);
      // ------------------------------------------------------------- epilogue
      const bool had = wg < n;
      if (ok && had) {
        ok = warp_wait(&odone[wg], oph);
        oph ^= 1u;
      }
      if (k8 && (__float_as_uint(node_scale) & 0x7f800000u) == 0x7f800000u) atomicOr(s_bad, 1ull << tid);
      ok = smx_sync_and(ok);   // every product of the piece is done: the query rows are free
      if (!ok) break;
      tc_fence_after();
      float2* s_ml = reinterpret_cast<float2*>(stage);
      s_ml[wg * kM + r] = had ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
      smx_sync();
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int x = 0; x < 2 * F; ++x) M = fmaxf(M, s_ml[(x & 1) * kM + (x >> 1) * RP + rr].x);
#pragma unroll
      for (int x = 0; x < 2 * F; ++x) {
        const float2 ml = s_ml[(x & 1) * kM + (x >> 1) * RP + rr];
        L = fmaf(ml.y, partial_weight(ml.x, ml.y, M), L);
      }
      const bool complete = it.complete();
      const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + it.slot();
      float wt = had ? partial_weight(m, l, M) : 0.f;
      if (k8) wt *= __uint_as_float(static_cast<uint32_t>(ve) << 23);   // O's unit
      if (complete) {
        // nothing seen: 0; only scores of -inf: NaN, as the formula's 0 / 0
        wt *= L == 0.f ? (it.w.past > 0 || see != 0 ? __uint_as_float(0x7fc00000u) : 0.f) : 1.f / L;
      } else if (tid < RP) {
        p.ml[slot * RP + rr] = make_float2(M, L);
      }
      const unsigned long long bad_v = *s_bad;
      smx_sync();   // the statistics are read; everyone has the noted rows
      if (tid == 0) *s_bad = 0;
      // the item's rows, in passes of 32 columns, or of 64 or 128 where few enough rows leave the
      // room: partial row x of row rr at slot x * (RP >> wide) + rr, its 16-byte units turned by rr
      const int rows = min(RP, it.w.nodes * p.group - first);
      const int wide = rows * 4 <= RP && D == 128 ? 2 : rows * 2 <= RP ? 1 : 0;
      const int per = RP >> wide, units = 8 << wide;
      bool fine = true;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32 << wide) {
        float* mine = stage + ((wg * F + f) * per + rr) * (32 << wide);
#pragma unroll 1
        for (int k = 0; k < 1 << wide; ++k) {
          float o[32];
          if (had) tmem_ld32(tOw + c0 + 32 * k, o);
          if (rr < rows) {
#pragma unroll
            for (int u = 0; u < 8; ++u)
              *reinterpret_cast<float4*>(mine + ((8 * k + (u ^ (rr & 7))) << 2)) =
                  had ? make_float4(o[4 * u] * wt, o[4 * u + 1] * wt, o[4 * u + 2] * wt, o[4 * u + 3] * wt)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
        smx_sync();
#pragma unroll 1
        for (int i = tid; i < rows * units; i += kSmxThreads) {
          const int row = i >> (3 + wide), u = i & (units - 1), t = (first + row) >> gs, h = (first + row) & (p.group - 1);
          const float* src = stage + row * (32 << wide) + ((u ^ (row & 7)) << 2);
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int x = 0; x < 2 * F; ++x) {
            const float4 v = *reinterpret_cast<const float4*>(src + x * per * (32 << wide));
            a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
          }
          if (!k8) fine = fine && fmaf(a.x, 0.f, fmaf(a.y, 0.f, fmaf(a.z, 0.f, a.w * 0.f))) == 0.f;
          const int col = c0 + 4 * u;
          if (bad_v != 0) {
            const float4 x = bad_v_sum<KvT, D>(p.cache, it.b, it.g, it.w.past, bad_v & seen_nodes(p, it.b, t, it.w.nodes), col);
            a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
          }
          if (complete)
            store_tree_row4(p, it.b, t, it.g * p.group + h, D, col, a, 1.f);
          else
            *reinterpret_cast<float4*>(p.part + (slot * RP + row) * D + col) = a;
        }
        smx_sync();
      }
      // A committed row's infinite V entry leaves NaN in the replicas that hold weights of 0 for it.
      // bf16: where an output row is not finite, the piece's rows are looked through and such a
      // column becomes the sum of its infinities and NaN, whose weights are above 0.  (Columns of
      // other causes stay; 8-bit V operands are finite, or NaN.)
      if constexpr (!k8) {
        if (__builtin_expect(!smx_sync_and(fine), false)) {
          float* s_row = stage;   // [256]: whether the weights of this thread's row are NaN
          s_row[tid] = had && (l != l || wt != wt) ? 1.f : 0.f;
          if (tid < D) s_nf[tid] = 0.f;
          smx_sync();
          nonfinite_columns<D>(p, it, tid, s_nf);
          smx_sync();
#pragma unroll 1
          for (int i = tid; i < rows * D; i += kSmxThreads) {
            const int row = i / D, col = i % D, t = (first + row) >> gs, h = (first + row) & (p.group - 1);
            float a = s_nf[col];
            if (a == 0.f) continue;
            float nan = 0.f;
            for (int x = 0; x < 2 * F; ++x) nan += s_row[(x & 1) * kM + (x >> 1) * RP + row];
            if (nan != 0.f) a = __uint_as_float(0x7fc00000u);
            if (bad_v != 0) {
              const float4 x = bad_v_sum<KvT, D>(p.cache, it.b, it.g, it.w.past, bad_v & seen_nodes(p, it.b, t, it.w.nodes), col & ~3);
              a += (col & 3) == 0 ? x.x : (col & 3) == 1 ? x.y : (col & 3) == 2 ? x.z : x.w;
            }
            if (complete) {
              const int64_t at = ((static_cast<int64_t>(it.b) * p.T + t) * p.n_q_heads + it.g * p.group + h) * D + col;
              static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(a);
            } else {
              p.part[(slot * RP + row) * D + col] = a;
            }
          }
          smx_sync();
        }
      }
    }
    if (!ok && lane == 0) set_err(p.err, TTS_EFLAG_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static std::mutex mtx;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::lock_guard<std::mutex> lock(mtx);
  if (fn == nullptr) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    else
      cudaGetLastError();
  }
  return fn;
}

template <int D, typename KvT, int F>
cudaError_t launch_t(const TreeParams& p, cudaStream_t s) {
  auto kern = tree_attn_tc_kernel<D, KvT, F>;
  constexpr size_t smem = TcCfg<D, KvT>::kSmem;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  CUtensorMap maps[2] = {};
  if (!TcCfg<D, KvT>::k8) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    if (enc == nullptr) return cudaErrorNotSupported;
    // the cache as [chunks of 64 columns][rows][64]; a box is a tile, or a page's 64 columns
    const CacheView& c = p.cache;
    const int ps = 1 << c.page_shift;
    const bool whole = !c.paged || ps >= kN;
    const uint64_t rows = c.paged ? static_cast<uint64_t>(c.n_pages) * c.n_kv_heads * ps
                                  : static_cast<uint64_t>(c.B) * c.n_kv_heads * c.capacity;
    cuuint64_t dims[3] = {64, rows, D / 64};
    cuuint64_t strides[2] = {D * 2, 128};
    cuuint32_t box[3] = {64, static_cast<cuuint32_t>(whole ? kN : ps), static_cast<cuuint32_t>(whole ? D / 64 : 1)};
    cuuint32_t estr[3] = {1, 1, 1};
    for (int i = 0; i < 2; ++i)
      if (enc(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, i == 0 ? c.k : c.v, dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
  }
  return launch_pdl(kern, dim3(p.n_cta), dim3(TcCfg<D, KvT>::kThreads), smem, s, maps[0], maps[1], p);
}
template <int D, typename KvT>
cudaError_t launch_f(const TreeParams& p, cudaStream_t s) {
  switch (p.rows) {
    case 32: return launch_t<D, KvT, 4>(p, s);
    case 64: return launch_t<D, KvT, 2>(p, s);
    case 128: return launch_t<D, KvT, 1>(p, s);
    default: return cudaErrorInvalidValue;
  }
}
template <int D>
cudaError_t launch_kv(const TreeParams& p, int kv_dtype, cudaStream_t s) {
  switch (kv_dtype) {
    case TTS_BF16: return launch_f<D, __nv_bfloat16>(p, s);
    case TTS_I8: return launch_f<D, CodeI8>(p, s);
    case TTS_E4M3: return launch_f<D, CodeE4m3>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

bool tree_attn_tc_supported(const tts_kv_desc* d) {
  if (d->kv_dtype == TTS_I8 || d->kv_dtype == TTS_E4M3) return true;
  // tensor-map boxes: whole swizzle groups of eight rows, 32-bit row coordinates
  const int64_t rows = d->paged ? static_cast<int64_t>(d->n_pages) * d->n_kv_heads * d->page_size
                                : static_cast<int64_t>(d->B) * d->n_kv_heads * d->capacity;
  return d->kv_dtype == TTS_BF16 && (!d->paged || d->page_size >= 8) && rows < (int64_t{1} << 31) - kN;
}

cudaError_t launch_tree_attn_tc(const TreeParams& p, int kv_dtype, int head_dim, cudaStream_t s) {
  return head_dim == 64 ? launch_kv<64>(p, kv_dtype, s) : launch_kv<128>(p, kv_dtype, s);
}

}  // namespace tts
