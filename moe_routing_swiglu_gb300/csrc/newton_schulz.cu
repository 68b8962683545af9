// Orthogonalised updates by Newton-Schulz products, on the tensor cores.
//
// For each matrix G [r, c] of a batch (s = min(r, c) the short, l the long side):
//   X = G / (|G|_F + eps), then per step, with A = X X^T (X^T X where r > c)
//   and a, b, c = 3.4445, -4.7750, 2.0315:
//   X <- B X (X B),  B = a I + b A + c A A
// which moves every singular value of X from (0, 1] towards the interval
// [0.7, 1.21] and keeps its singular vectors. Grouped products:
//   GRAM   A, and any other product of polynomials in A (symmetric: the tiles
//          on and above the diagonal are computed, each also stored mirrored)
//   POLY   B = a I + b A + c A A, the first two terms in the epilogue
//          (symmetric too)
//   APPLY  X' = B X, or X B; FINAL the last one, whose epilogue writes the
//          result (16-bit, or the weights' update) instead of X'
// Two steps go together where that is less work: X'' = (B1 B) X with B1 from
// X' X'^T = B A B, so that X' itself is never computed.
//
// Precision. The map multiplies small singular values by 3.4 a step, 485 in
// five, and with them every rounding error made before; in 16-bit operands that
// shows along the weak directions. Operands are pairs of FP16 instead, v = hi +
// lo, lo the FP16 of v - hi, and a product is hi hi + hi lo + lo hi: 22 bits,
// for three MMAs. FP16 rather than BF16 pairs (16 bits) because every value here
// is bounded: |X| <= 1.21 (its largest singular value: the quintic maps [0,
// 1.21] into itself), |A| <= 1.47, |B| <= 3.45, |B1 B| <= 11.9. Stored times 2^14
// (X, A), 2^13 (B) or 2^12 (B1 B) they stay under FP16's 65504, and lo of an
// entry as small as 2^-14 is still a normal FP16. What is left is the FP32
// accumulators' truncation: 1e-6 (2-norm, of the result) for sides of 64, 3e-5
// to 1e-4 for 768 x 2048 to 2048 x 1408, 3e-4 for 4096 x 14336 with few strong
// directions, against 1.7e-3 of a BF16 and 2.1e-4 of an F16 result's rounding.
//
// Structure: a persistent pair of CTAs on two SMs (cta_group::2) per tile of
// 256 x 256, K in blocks of 64. Each CTA brings 128 rows of P and half of Q's
// columns, hi and lo, 64 KB a k-block for 1536 cycles of MMAs; one CTA alone
// with 128 x 256 tiles needs 96 KB, all that an SM takes in from L2 in that
// time. Warp 0 issues the TMA copies, warp 1 of the first CTA the MMAs, warps
// 2..9 drain TMEM, whose two 256-column accumulators let one tile's epilogue
// run under the next one's MMAs. Operands along their rows (K contiguous) are
// K-major tiles, X as a right-hand side and X^T X read X as it is stored,
// MN-major. Waits are bounded; one that runs out records a code and the CTA
// winds down.
//
// Bound by the power limit at the large sizes: 2 x 14336 x 4096 takes 8.5 ms on
// zeros and 11.1 ms on random values, for which the clock falls, 1.6 to 1.7
// PFLOP/s of MMAs; 128 x 768 x 2048 5.4 ms (4.3 on zeros), of which 4.2 at that
// rate. A few small matrices are bound by the 22 launches, 7 us each from one's
// last store to the next one's; where the short side is at most 128 they have a kernel of their
// own, which takes all steps in one launch.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "moe_common.cuh"
#include "moe_internal.h"
#include "ring_drain.h"
#include "round_sums.h"

namespace moe {
namespace {

constexpr float NS_A = 3.4445f, NS_B = -4.7750f, NS_C = 2.0315f;
__host__ __device__ constexpr float pow2(int e) { return e == 0 ? 1.0f : e > 0 ? 2.0f * pow2(e - 1) : 0.5f * pow2(e + 1); }
constexpr int X_EXP = 14, A_EXP = 14, B_EXP = 13, BB_EXP = 12;   // stored = value * 2^EXP

// ---------------------------------------------------------------- norm, momentum, first X

constexpr int PRE_THREADS = 256;
constexpr int PRE_GROUP = 4;         // groups of 8 elements that a thread loads together
constexpr int MAX_CHUNKS = 256;      // partial sums per matrix
constexpr int64_t MIN_CHUNK = PRE_THREADS * PRE_GROUP * 8;
constexpr int64_t PRE_BLOCKS = 1216; // blocks that a batch is cut into, at least, where its size allows it: 8 per SM

// Elements of a matrix that one block adds the squares of.
inline int64_t chunk_elems(int64_t E, int64_t n) {
  const int64_t least = (n + MAX_CHUNKS - 1) / MAX_CHUNKS, fair = E * n / PRE_BLOCKS;
  return (std::max(std::max(least, fair), MIN_CHUNK) + MIN_CHUNK - 1) / MIN_CHUNK * MIN_CHUNK;
}
inline int64_t chunk_count(int64_t E, int64_t n) { return (n + chunk_elems(E, n) - 1) / chunk_elems(E, n); }

template <typename T>
struct alignas(16) Eight {
  T e[8];
};
template <typename T>
__device__ __forceinline__ void load8(const T* p, Eight<T>& x) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(x) / 16); ++i)
    reinterpret_cast<uint4*>(&x)[i] = reinterpret_cast<const uint4*>(p)[i];
}
// The first n of 8 elements one by one, zeros for the others.
template <typename T>
__device__ __forceinline__ void load_some(const T* p, int n, Eight<T>& x) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x.e[i] = i < n ? p[i] : from_f32<T>(0.0f);
}

// Sums of squares that FP32 cannot hold: values above 2^40 and below 2^-40 are
// squared times 2^-180 and 2^180, in sums of their own.
struct Squares {
  float mid, big, small;
  __device__ void add(float v) {
    const float a = fabsf(v);
    if (a > 0x1p40f) {
      const float s = a * 0x1p-90f;
      big = fmaf(s, s, big);
    } else if (a < 0x1p-40f) {
      const float s = a * 0x1p90f;
      small = fmaf(s, s, small);
    } else {
      mid = fmaf(v, v, mid);   // NaN too
    }
  }
  __device__ double total() const { return mid + big * 0x1p180 + small * 0x1p-180; }
};

struct PreArgs {
  const void* g;       // [E, r, c]
  float* m;            // momentum [E, r, c] or NULL
  double* partial;     // [E, chunks]
  __half* hi;          // X [E, r, pitch]
  __half* lo;
  int64_t n, chunk;    // elements of a matrix, of a chunk
  int64_t pitch;
  int r, c, chunks, nesterov, vec;
  float mu, eps;
};

// u of the momentum step: what is orthogonalised.
__device__ __forceinline__ float update_of(const PreArgs& a, float g, float m) {
  return a.nesterov ? fmaf(a.mu, m, g) : m;
}

template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(FULL_MASK, v, off);
  return v;
}

// partial[e][chunk]: the sum of squares of the chunk's u; updates the momentum.
// A thread's squares are added in FP32, 32 of a round, 16 rounds, then a warp's: 53
// roundings, which leave a norm off by fewer than 2^-19 of it. The rest is FP64, as
// are rounds whose sum FP32 does not hold.
template <typename T, bool MOMENTUM>
__global__ void __launch_bounds__(PRE_THREADS) squares_kernel(const PreArgs a) {
  __shared__ double sm[PRE_THREADS / 32];
  grid_dependency_wait();
  launch_dependents();
  const T* gp = static_cast<const T*>(a.g) + blockIdx.y * a.n;
  float* mp = MOMENTUM ? a.m + blockIdx.y * a.n : nullptr;
  const int64_t lo = blockIdx.x * a.chunk, hi = min(lo + a.chunk, a.n);
  constexpr int ROUND = PRE_THREADS * 8 * PRE_GROUP;
  RoundSums total;
  for (int64_t i0 = lo; i0 < hi; i0 += ROUND) {
    const int64_t at = i0 + static_cast<int64_t>(threadIdx.x) * 8;
    const bool whole = a.vec && i0 + ROUND <= hi;
    Eight<T> g[PRE_GROUP];
    Eight<float> m[PRE_GROUP];
    int n[PRE_GROUP];
    if (whole) {
#pragma unroll
      for (int k = 0; k < PRE_GROUP; ++k) {
        load8<T>(gp + at + k * PRE_THREADS * 8, g[k]);
        if (MOMENTUM) load8<float>(mp + at + k * PRE_THREADS * 8, m[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < PRE_GROUP; ++k) {
        const int64_t i = at + k * PRE_THREADS * 8;
        n[k] = static_cast<int>(max(min(hi - i, int64_t{8}), int64_t{0}));
        load_some<T>(gp + i, n[k], g[k]);
        if (MOMENTUM) load_some<float>(mp + i, n[k], m[k]);
      }
    }
    float sum = 0.0f;
    Eight<float> u[PRE_GROUP];
#pragma unroll
    for (int k = 0; k < PRE_GROUP; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[k].e[j] = to_f32(g[k].e[j]);
        if (MOMENTUM) {
          m[k].e[j] = fmaf(a.mu, m[k].e[j], u[k].e[j]);
          u[k].e[j] = update_of(a, u[k].e[j], m[k].e[j]);
        }
        sum = fmaf(u[k].e[j], u[k].e[j], sum);
      }
    if (MOMENTUM) {
#pragma unroll
      for (int k = 0; k < PRE_GROUP; ++k) {
        float* p = mp + at + k * PRE_THREADS * 8;
        if (whole) {
          reinterpret_cast<uint4*>(p)[0] = reinterpret_cast<const uint4*>(&m[k])[0];
          reinterpret_cast<uint4*>(p)[1] = reinterpret_cast<const uint4*>(&m[k])[1];
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < n[k]) p[j] = m[k].e[j];
        }
      }
    }
    // 32 squares that each lose at most 2^-150 do not show in a sum of 2^-60; 2^80 leaves room for the other rounds.
    if (sum >= 0x1p-60f && sum <= 0x1p80f) {
      total.add(sum);
    } else {
      Squares s{0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < PRE_GROUP; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) s.add(u[k].e[j]);
      total.far += s.total();
    }
  }
  const float near = warp_sum(total.near);
  double far = total.far;
  if (__any_sync(FULL_MASK, far != 0.0)) far = warp_sum(far);   // NaN != 0 too
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = near + far;
  __syncthreads();
  if (threadIdx.x == 0) {
    double sum = 0.0;
    for (int w = 0; w < PRE_THREADS / 32; ++w) sum += sm[w];
    a.partial[static_cast<int64_t>(blockIdx.y) * a.chunks + blockIdx.x] = sum;
  }
}

__device__ __forceinline__ void split_half(float v, __half* hi, __half* lo) {
  *hi = __float2half_rn(v);
  *lo = __float2half_rn(v - __half2float(*hi));
}
__device__ __forceinline__ void split_half2(float x, float y, uint32_t* hi, uint32_t* lo) {
  const __half2 p = __floats2half2_rn(x, y);
  const float2 f = __half22float2(p);
  *hi = *reinterpret_cast<const uint32_t*>(&p);
  *lo = pack2<__half>(x - f.x, y - f.y);
}

__device__ __forceinline__ float power2(int e) { return __int_as_float((e + 127) << 23); }   // -126 .. 127

// 2^14 / (sqrt(sum) + eps) as two FP32 factors, both far from FP32's ends: with
// sum = m 4^k and eps = f 2^j over the larger power p of k and j, 2^(14 - p) /
// (sqrt(m) 2^(k - p) + f 2^(j - p)). NaN where the sum is not finite: a matrix
// with a NaN or an infinity becomes NaN as a whole.
__device__ __forceinline__ float2 scale_of(double sum, float eps) {
  if (!(sum <= 0x1p1000)) return make_float2(__int_as_float(0x7FC00000), 1.0f);
  int j, k = -600;
  const float f = frexpf(eps, &j);
  float root = 0.0f;
  if (sum > 0x1p-1000) {
    const int ex = ((__double2hiint(sum) >> 20) & 0x7FF) - 1022;   // sum = m 2^ex, m in [1/2, 1)
    k = (ex + (ex & 1)) / 2;
    root = sqrtf(static_cast<float>(sum * __hiloint2double((1023 - 2 * k) << 20, 0)));
  }
  const int p = max(j, k);
  const float t = (k - p > -100 ? root * power2(k - p) : 0.0f) + (j - p > -100 ? f * power2(j - p) : 0.0f);
  const int e = 14 - p, h = e / 2;
  return make_float2(power2(e - h) / t, power2(h));
}

// X = u / (norm + eps), as FP16 pairs.
template <typename T, bool MOMENTUM>
__global__ void __launch_bounds__(PRE_THREADS) first_x_kernel(const PreArgs a) {
  __shared__ float2 factors;
  grid_dependency_wait();
  launch_dependents();
  const int64_t e = blockIdx.y;
  if (threadIdx.x < 32) {
    double sum = 0.0;
    for (int i = threadIdx.x; i < a.chunks; i += 32) sum += a.partial[e * a.chunks + i];
    sum = warp_sum(sum);
    if (threadIdx.x == 0) factors = scale_of(sum, a.eps);
  }
  __syncthreads();
  const float s1 = factors.x, s2 = factors.y;
  const T* gp = static_cast<const T*>(a.g) + e * a.n;
  const float* mp = MOMENTUM ? a.m + e * a.n : nullptr;
  __half* hi = a.hi + e * a.r * a.pitch;
  __half* lo = a.lo + e * a.r * a.pitch;
  const uint32_t per_row = static_cast<uint32_t>(a.pitch / 8), groups = per_row * a.r;
  const bool flat = a.vec && a.c % 8 == 0;   // rows without padding: group i is elements 8 i ..
  const uint32_t step = gridDim.x * PRE_THREADS;
  for (uint32_t i0 = blockIdx.x * PRE_THREADS + threadIdx.x; i0 < groups; i0 += PRE_GROUP * step) {
    Eight<T> g[PRE_GROUP];
    Eight<float> m[PRE_GROUP];
    if (flat && i0 + (PRE_GROUP - 1) * step < groups) {
#pragma unroll
      for (int k = 0; k < PRE_GROUP; ++k) {
        const int64_t at = static_cast<int64_t>(i0 + k * step) * 8;
        load8<T>(gp + at, g[k]);
        if (MOMENTUM) load8<float>(mp + at, m[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < PRE_GROUP; ++k) {
        const uint32_t i = i0 + k * step;
        if (i >= groups) continue;
        const uint32_t row = i / per_row, col = (i - row * per_row) * 8;
        const int64_t at = static_cast<int64_t>(row) * a.c + col;
        load_some<T>(gp + at, min(a.c - static_cast<int>(col), 8), g[k]);
        if (MOMENTUM) load_some<float>(mp + at, min(a.c - static_cast<int>(col), 8), m[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < PRE_GROUP; ++k) {
      const uint32_t i = i0 + k * step;
      if (i >= groups) continue;
      float u[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[j] = to_f32(g[k].e[j]);
        if (MOMENTUM) u[j] = update_of(a, u[j], m[k].e[j]);
        u[j] = u[j] * s1 * s2;
      }
      uint32_t h[4], l[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) split_half2(u[2 * j], u[2 * j + 1], &h[j], &l[j]);
      reinterpret_cast<uint4*>(hi)[i] = make_uint4(h[0], h[1], h[2], h[3]);
      reinterpret_cast<uint4*>(lo)[i] = make_uint4(l[0], l[1], l[2], l[3]);
    }
  }
}

// ---------------------------------------------------------------- the products

enum NsMode { GRAM = 0, POLY = 1, APPLY = 2, FINAL = 3, GRAM_PART = 4 };

constexpr int TILE = 256, BM = 128, BK = 64, UMMA_K = 16;
constexpr int BOX = 64 * 128;                        // 64 x 64 elements, or 64 rows of 128 bytes
constexpr int OP_BYTES = BM * BK * 2;                // a block's half of an operand: 128 rows, or columns
constexpr int STAGE_BYTES = 4 * OP_BYTES;            // hi and lo of both operands
constexpr int STAGES = 3;
constexpr uint32_t TMEM_COLS = 512;
constexpr int NUM_EPI_WARPS = 8;
constexpr int NUM_THREADS = 32 * (2 + NUM_EPI_WARPS);
constexpr uint64_t WAIT_LIMIT_NS = 1000000000ull;
constexpr int STAGING_BYTES = 32 * 32 * 4;           // per epilogue warp: 32 x 32 FP32, or FP16 hi and lo
constexpr int SMEM_STAGING = STAGES * STAGE_BYTES;
constexpr int SMEM_BAR = SMEM_STAGING + NUM_EPI_WARPS * STAGING_BYTES;
constexpr int NUM_BARS = 2 * STAGES + 5;
constexpr int SMEM_MISC = SMEM_BAR + 8 * NUM_BARS;   // TMEM address, abort flag, stages issued
constexpr int SMEM_BYTES = 1024 + SMEM_MISC + 16;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");

constexpr uint32_t ST_PRODUCER_EMPTY = 0x41;
constexpr uint32_t ST_MMA_FULL = 0x42;
constexpr uint32_t ST_MMA_TMEM_EMPTY = 0x43;
constexpr uint32_t ST_EPI_TMEM_FULL = 0x44;
constexpr uint32_t ST_MMA_DRAIN = 0x45;
constexpr uint32_t ST_PRODUCER_DRAIN = 0x46;

// A block pair's instructions (cta_group::2): block 0 of the pair issues one
// MMA for both, each block holding 128 rows of P, half of Q's columns and 128
// rows of the accumulator.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of `p` in block `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_u32(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
// Relaxed: what these two signal is in tensor memory or arrives by TMA, and a
// release waits for the SM's stores in flight (2 x 14336 x 4096: 14.9 ms with
// it, 14.1 without).
__device__ __forceinline__ void peer_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void peer_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ uint32_t peer_load(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// Into this block's shared memory, counted on a barrier of either block.
__device__ __forceinline__ void pair_load_3d(void* dst, const void* desc, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(desc), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void pair_tmem_alloc(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void pair_umma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at this place in both blocks once the MMAs issued so
// far are complete.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// FP16 pairs [E, rows, pitch] of the workspace; what lies between cols and the
// pitch (fewer than 8) is written, and never read.
struct Pair {
  __half* hi;
  __half* lo;
  int64_t rows, cols, pitch;
};

// D [E, m, n] = P [E, m, k] Q [E, k, n], both FP16 pairs.
struct NsArgs {
  int m, n, k;
  int m_blocks, n_blocks;
  int k_split;          // k-blocks of a part (GRAM_PART), else all
  uint32_t tiles, tiles_per_matrix;
  int square;           // GRAM: P and Q are the same matrix
  Pair out;             // GRAM, POLY, APPLY
  Pair a;               // POLY: A
  float scale;          // of the accumulator: stored result = acc * scale (POLY: + A * a_scale + diag I)
  float a_scale, diag;
  int64_t pitch;        // GRAM_PART
  float* parts;         // [parts, E, m, pitch]
  int64_t part_elems;   // E * m * pitch
  void* result;         // FINAL: [E, m, n] in result_dtype
  int result_dtype;
  int update;           // FINAL: result = keep * result - rate * X' (weights), else X'
  float keep, rate;
  uint32_t* status;
};

// Tile -> (matrix, row block, column block, first k-block and their number).
// Symmetric products have the tiles on and above the diagonal; a product in
// parts has all tiles of one part before the next part's. Row blocks go in
// bands of BAND, in a band column by column, so that the tiles that run at once
// share both operands in L2 (2 x 14336 x 4096 with X's 56 row blocks in one
// column after the other read X from HBM 12 times a product).
constexpr int BAND = 8;
struct NsTile {
  int e, mb, nb, kb0, kbs, part;
};
template <int MODE>
__device__ __forceinline__ NsTile ns_tile(uint32_t tile, const NsArgs& a) {
  NsTile t;
  const int k_blocks = (a.k + BK - 1) / BK;
  t.kb0 = 0;
  t.kbs = k_blocks;
  t.part = 0;
  uint32_t matrix = tile / a.tiles_per_matrix;
  int i = static_cast<int>(tile - matrix * a.tiles_per_matrix);
  int mb0 = 0;   // the band's first row block
  if (MODE == GRAM || MODE == POLY) {
    int rows = min(BAND, a.m_blocks);
    for (;;) {
      const int in_band = rows * (rows + 1) / 2 + rows * (a.n_blocks - mb0 - rows);
      if (i < in_band) break;
      i -= in_band;
      mb0 += rows;
      rows = min(BAND, a.m_blocks - mb0);
    }
    const int corner = rows * (rows + 1) / 2;   // the band's triangle at the diagonal, column by column
    if (i < corner) {
      int col = 0;
      while (i > col) i -= ++col;
      t.mb = mb0 + i;
      t.nb = mb0 + col;
    } else {
      t.mb = mb0 + (i - corner) % rows;
      t.nb = mb0 + rows + (i - corner) / rows;
    }
  } else {
    mb0 = i / (BAND * a.n_blocks) * BAND;
    i -= mb0 * a.n_blocks;
    const int rows = min(BAND, a.m_blocks - mb0);
    t.mb = mb0 + i % rows;
    t.nb = i / rows;
  }
  if (MODE == GRAM_PART) {
    const uint32_t matrices = static_cast<uint32_t>(a.part_elems / (a.m * a.pitch));
    t.part = static_cast<int>(matrix / matrices);
    matrix -= t.part * matrices;
    t.kb0 = t.part * a.k_split;
    t.kbs = min(a.k_split, k_blocks - t.kb0);
  }
  t.e = static_cast<int>(matrix);
  return t;
}

// A warp's 32 x 32 block (lane: row, v: its columns) as FP16 pairs into its
// staging tiles, 32 rows of 64 bytes each (16-byte chunk q of row r at chunk
// q ^ (r / 2 % 4): no bank conflicts either way), and from there to (row, col)
// of both planes, four lanes a row. MIRROR: the transposed block, at (col, row).
template <bool MIRROR>
__device__ __forceinline__ void store_pairs(uint32_t tile, const Pair& out, int e, int row, int col, const float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  __syncwarp();   // the last block has left the tiles
  if (MIRROR) {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      __half h, l;
      split_half(v[j], &h, &l);
      const uint32_t at = tile + j * 64 + (((lane >> 3) ^ ((j >> 1) & 3)) << 4) + (lane & 7) * 2;
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(__half_as_ushort(h)) : "memory");
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + 2048), "h"(__half_as_ushort(l)) : "memory");
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t h[4], l[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) split_half2(v[q * 8 + 2 * j], v[q * 8 + 2 * j + 1], &h[j], &l[j]);
      const uint32_t at = tile + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4);
      st_shared_v4(at, h[0], h[1], h[2], h[3]);
      st_shared_v4(at + 2048, l[0], l[1], l[2], l[3]);
    }
  }
  __syncwarp();
  const int r0 = MIRROR ? col : row, c0 = (MIRROR ? row : col) + (lane & 3) * 8;
  if (c0 >= out.pitch) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2);
    const uint32_t at = tile + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4);
    if (r0 + r < out.rows) {
      const int64_t to = (static_cast<int64_t>(e) * out.rows + r0 + r) * out.pitch + c0;
      *reinterpret_cast<uint4*>(out.hi + to) = ld_shared_v4(at);
      *reinterpret_cast<uint4*>(out.lo + to) = ld_shared_v4(at + 2048);
    }
  }
}

// The 32 x 32 block of `in` at (row, col): in two parts, so that the loads run
// while the accumulator is read. Past the matrix: anything.
__device__ __forceinline__ void load_pairs(const Pair& in, int e, int row, int col, uint4 (&hi)[4], uint4 (&lo)[4]) {
  const int lane = threadIdx.x & 31, c = col + (lane & 3) * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = row + i * 8 + (lane >> 2);
    hi[i] = lo[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < in.rows && c < in.pitch) {
      const int64_t at = (static_cast<int64_t>(e) * in.rows + r) * in.pitch + c;
      hi[i] = *reinterpret_cast<const uint4*>(in.hi + at);
      lo[i] = *reinterpret_cast<const uint4*>(in.lo + at);
    }
  }
}
// v = raw * scale + (this lane's row of the loaded block) * block_scale
__device__ __forceinline__ void add_pairs(uint32_t tile, const uint4 (&hi)[4], const uint4 (&lo)[4], float block_scale,
                                          const uint32_t (&raw)[32], float scale, float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2);
    const uint32_t at = tile + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4);
    st_shared_v4(at, hi[i].x, hi[i].y, hi[i].z, hi[i].w);
    st_shared_v4(at + 2048, lo[i].x, lo[i].y, lo[i].z, lo[i].w);
  }
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t at = tile + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4);
    const uint4 h = ld_shared_v4(at), l = ld_shared_v4(at + 2048);
    const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&hw[j]));
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&lw[j]));
      v[q * 8 + 2 * j] = fmaf(__uint_as_float(raw[q * 8 + 2 * j]), scale, (x.x + y.x) * block_scale);
      v[q * 8 + 2 * j + 1] = fmaf(__uint_as_float(raw[q * 8 + 2 * j + 1]), scale, (x.y + y.y) * block_scale);
    }
  }
}

// A warp's block of the last product through its staging tile (FP32, 32 rows of
// 128 bytes, 16-byte chunk q of row r at chunk q ^ (r % 8)), so that a warp
// reads and writes 32 neighbouring elements of a row.
template <typename T>
__device__ __forceinline__ void store_result(const NsArgs& a, float* tile, int row, int col, int e, const float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 8; ++q)
    *reinterpret_cast<float4*>(tile + lane * 32 + ((q ^ (lane & 7)) << 2)) =
        make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
  __syncwarp();
  const bool in = col + lane < a.n;
  T* p = static_cast<T*>(a.result) + (static_cast<int64_t>(e) * a.m + row) * a.n + col + lane;
  constexpr int G = 8;    // rows whose weights are loaded together
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += G) {
    T old[G];
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (a.update && in && row + r0 + i < a.m) old[i] = p[static_cast<int64_t>(r0 + i) * a.n];
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int r = r0 + i;
      const float x = tile[r * 32 + ((((lane >> 2) ^ (r & 7)) << 2) | (lane & 3))];
      if (in && row + r < a.m)
        p[static_cast<int64_t>(r) * a.n] = from_f32<T>(a.update ? fmaf(a.keep, to_f32(old[i]), -a.rate * x) : x);
    }
  }
}

template <int MODE, bool P_MN, bool Q_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NUM_THREADS, 1)
    ns_kernel(const __grid_constant__ CUtensorMap p_hi, const __grid_constant__ CUtensorMap p_lo,
              const __grid_constant__ CUtensorMap q_hi, const __grid_constant__ CUtensorMap q_lo,
              const __grid_constant__ NsArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SMEM_BAR);   // block 0's are used
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;   // [2]
  uint64_t* tempty = tfull + 2;       // [2], block 0's are used
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + SMEM_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SMEM_MISC + 4);
  uint32_t* issued_stages = reinterpret_cast<uint32_t*>(smem + SMEM_MISC + 8);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 2);          // each block arms its own copies
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * NUM_EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *issued_stages = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&p_hi);
    tma_prefetch_desc(&p_lo);
    tma_prefetch_desc(&q_hi);
    tma_prefetch_desc(&q_lo);
  }
  __syncwarp();
  if (warp == 1) pair_tmem_alloc(tmem_holder, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both blocks' barriers are there before either one's copies and arrivals
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  grid_dependency_wait();
  launch_dependents();

  // Columns of a tile, of which each block brings half.
  auto n_of = [&](const NsTile& t) { return min(TILE, (args.n - t.nb * TILE + 31) & ~31); };
  // A whole tile on the diagonal of M M^T: both operands are the same rows.
  auto same_operand = [&](const NsTile& t) {
    return (MODE == GRAM || MODE == POLY || MODE == GRAM_PART) && args.square && t.mb == t.nb && n_of(t) == TILE;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (uint32_t tile = pair; ok && tile < args.tiles; tile += pairs) {
        const NsTile t = ns_tile<MODE>(tile, args);
        const int m0 = t.mb * TILE + static_cast<int>(rank) * BM;
        const int n0 = t.nb * TILE + static_cast<int>(rank) * (n_of(t) / 2);
        const bool same = same_operand(t);
        for (int kb = t.kb0; kb < t.kb0 + t.kbs; ++kb) {
          ok = mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, args.status, ST_PRODUCER_EMPTY, WAIT_LIMIT_NS);
          if (!ok) break;
          uint8_t* st = smem + stage * STAGE_BYTES;
          const uint32_t bar = peer_u32(&full[stage], 0);
          peer_arrive_expect_tx(bar, same ? STAGE_BYTES / 2 : STAGE_BYTES);
          const int k0 = kb * BK;
          auto load = [&](uint8_t* dst, const CUtensorMap* map, bool mn_major, int at) {
            if (!mn_major) {
              pair_load_3d(dst, map, bar, k0, at, t.e);
            } else {
              for (int q = 0; q < BM / 64; ++q) pair_load_3d(dst + q * BOX, map, bar, at + 64 * q, k0, t.e);
            }
          };
          load(st, &p_hi, P_MN, m0);
          if (!same) load(st + 2 * OP_BYTES, &q_hi, Q_MN, n0);
          load(st + OP_BYTES, &p_lo, P_MN, m0);
          if (!same) load(st + 3 * OP_BYTES, &q_lo, Q_MN, n0);
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      *issued_stages = issued;
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (block 0, for both)
    if (lane == 0) {
      if (rank == 0) {
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        uint32_t it = 0;
        for (uint32_t tile = pair; ok && tile < args.tiles; tile += pairs, ++it) {
          const NsTile t = ns_tile<MODE>(tile, args);
          const uint32_t idesc = idesc_f16_major(false, TILE, n_of(t), P_MN, Q_MN);
          const uint32_t acc = it & 1u;
          ok = mbar_wait_bounded(&tempty[acc], ((it >> 1) & 1u) ^ 1u, abort_flag, args.status, ST_MMA_TMEM_EMPTY,
                                 WAIT_LIMIT_NS);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem_base + acc * TILE;
          for (int kb = t.kb0; kb < t.kb0 + t.kbs; ++kb) {
            ok = mbar_wait_bounded(&full[stage], phase, abort_flag, args.status, ST_MMA_FULL, WAIT_LIMIT_NS);
            if (!ok) break;
            tc_fence_after();
            const uint32_t ph = smem_u32(smem + stage * STAGE_BYTES), pl = ph + OP_BYTES;
            const uint32_t qh = same_operand(t) ? ph : ph + 2 * OP_BYTES, ql = qh + OP_BYTES;
            const int n_sub = min(BK / UMMA_K, (args.k - kb * BK + UMMA_K - 1) / UMMA_K);
            for (int k = 0; k < n_sub; ++k) {
              auto pd = [&](uint32_t at) {
                return P_MN ? sdesc_mnmajor_sw128(at + k * 2048, BOX, 1024) : sdesc_kmajor_sw128(at + k * UMMA_K * 2);
              };
              auto qd = [&](uint32_t at) {
                return Q_MN ? sdesc_mnmajor_sw128(at + k * 2048, BOX, 1024) : sdesc_kmajor_sw128(at + k * UMMA_K * 2);
              };
              pair_umma_f16(d, pd(ph), qd(qh), idesc, (kb > t.kb0 || k > 0) ? 1u : 0u);
              pair_umma_f16(d, pd(pl), qd(qh), idesc, 1u);
              pair_umma_f16(d, pd(ph), qd(ql), idesc, 1u);
            }
            pair_commit(&empty[stage]);
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          pair_commit(&tfull[acc]);
        }
        pair_commit(drain);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3;
    const int half = (warp - 2) >> 2;
    uint8_t* staging = smem + SMEM_STAGING + (warp - 2) * STAGING_BYTES;
    const uint32_t tile_at = smem_u32(staging);
    uint32_t it = 0;
    for (uint32_t tile = pair; tile < args.tiles; tile += pairs, ++it) {
      const NsTile t = ns_tile<MODE>(tile, args);
      const uint32_t acc = it & 1u;
      const bool ok = mbar_wait_bounded(&tfull[acc], (it >> 1) & 1u, abort_flag, args.status, ST_EPI_TMEM_FULL,
                                        WAIT_LIMIT_NS);
      if (!__all_sync(FULL_MASK, ok)) break;
      tc_fence_after();
      const uint32_t t_lane = tmem_base + acc * TILE + (static_cast<uint32_t>(quad * 32) << 16);
      const int row = t.mb * TILE + static_cast<int>(rank) * BM + quad * 32;   // of lane 0
      for (int c0 = 32 * half; c0 < TILE; c0 += 64) {
        const int col = t.nb * TILE + c0;
        if (col >= args.n || row >= args.m) break;
        uint4 a_hi[4], a_lo[4];
        if (MODE == POLY) load_pairs(args.a, t.e, row, col, a_hi, a_lo);
        uint32_t raw[32];
        tmem_ld_32x32b_x32(t_lane + static_cast<uint32_t>(c0), raw);
        tmem_ld_wait();
        float v[32];
        if (MODE == GRAM || MODE == POLY) {
          if (MODE == GRAM) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(raw[j]) * args.scale;
          } else {
            add_pairs(tile_at, a_hi, a_lo, args.a_scale, raw, args.scale, v);
            const int diag = row + lane - col;
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] += diag == j ? args.diag : 0.0f;
          }
          store_pairs<false>(tile_at, args.out, t.e, row, col, v);
          if (t.nb != t.mb) store_pairs<true>(tile_at, args.out, t.e, row, col, v);
        } else if (MODE == GRAM_PART) {
          if (row + lane < args.m) {
            float* p = args.parts + t.part * args.part_elems + (static_cast<int64_t>(t.e) * args.m + row + lane) * args.pitch +
                       col;
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (col + q * 4 < args.pitch)
                reinterpret_cast<uint4*>(p)[q] = make_uint4(raw[4 * q], raw[4 * q + 1], raw[4 * q + 2], raw[4 * q + 3]);
          }
        } else if (MODE == APPLY) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(raw[j]) * args.scale;
          store_pairs<false>(tile_at, args.out, t.e, row, col, v);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(raw[j]) * args.scale;
          float* stage = reinterpret_cast<float*>(staging);
          if (args.result_dtype == MOE_F32) store_result<float>(args, stage, row, col, t.e, v);
          else if (args.result_dtype == MOE_F16) store_result<__half>(args, stage, row, col, t.e, v);
          else store_result<__nv_bfloat16>(args, stage, row, col, t.e, v);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) peer_arrive(peer_u32(&tempty[acc], 0));
    }
  }

  tc_fence_before();
  __syncthreads();
  // Every MMA has read its operands, and every commit has arrived, before either block leaves.
  if (threadIdx.x == 0) mbar_wait_bounded(drain, 0, nullptr, args.status, ST_MMA_DRAIN, WAIT_LIMIT_NS);
  __syncwarp();
  cluster_sync();
  if (*abort_flag != 0 || peer_load(peer_u32(const_cast<int*>(abort_flag), rank ^ 1u)) != 0) {
    // A role gave up: the copies that nobody waited for land before the blocks
    // exit. A stage that one block alone has issued is armed here for the other.
    if (threadIdx.x == 0 && rank == 0) {
      const uint32_t mine = *issued_stages, other = peer_load(peer_u32(issued_stages, 1));
      for (uint32_t n = min(mine, other); n < max(mine, other); ++n) mbar_arrive(&full[n % STAGES]);
      drain_ring(max(mine, other), STAGES, [&](uint32_t slot, uint32_t parity) {
        mbar_wait_bounded(&full[slot], parity, nullptr, args.status, ST_PRODUCER_DRAIN, WAIT_LIMIT_NS);
      });
    }
    __syncthreads();
  }
  cluster_sync();   // nothing is left that reads or signals the other block's shared memory
  if (warp == 1) {
    tc_fence_after();
    pair_tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// A from the parts of GRAM_PART, added in order.
__global__ void __launch_bounds__(PRE_THREADS) join_parts_kernel(const float* parts, int64_t part_elems, int count,
                                                                 float scale, __half* hi, __half* lo) {
  grid_dependency_wait();
  launch_dependents();
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * PRE_THREADS + threadIdx.x) * 4;
  if (at >= part_elems) return;
  float4 v = *reinterpret_cast<const float4*>(parts + at);
#pragma unroll 4
  for (int p = 1; p < count; ++p) {
    const float4 w = *reinterpret_cast<const float4*>(parts + p * part_elems + at);
    v.x += w.x;
    v.y += w.y;
    v.z += w.z;
    v.w += w.w;
  }
  uint2 h, l;
  split_half2(v.x * scale, v.y * scale, &h.x, &l.x);
  split_half2(v.z * scale, v.w * scale, &h.y, &l.y);
  *reinterpret_cast<uint2*>(hi + at) = h;
  *reinterpret_cast<uint2*>(lo + at) = l;
}

// ---------------------------------------------------------------- short sides up to 128: one launch

// All steps of a matrix whose short side is at most 128 in one launch: a cluster
// of 1 to 16 blocks holds X in shared memory, each block the FP16 pairs of up to
// 192 columns (wide; rows where r > c, transposed as they are loaded), as tiles
// of 128 rows x 64 columns with 128-byte rows, swizzled: K-major operands of X
// X^T and an MN-major one of B X alike. A step:
//   each block's part of A = X X^T goes from TMEM to the blocks that own its
//   rows, s / C each; the owners add the parts in order and store their rows of
//   A, as pairs, into every block;
//   each block has all of B = a I + b A + c A A (over A), and X = B X of its
//   columns, in place.
// Rows of X past the short side up to a multiple of 16, and columns past the
// long side, are zeros and stay zeros; rows past that are never read but as
// rows of the 128 of an MMA whose results are not read either.
//
// Bound by latency: a step is three MMA chains of 24 to 36 instructions, each
// with a trip through TMEM and registers, and two cluster barriers. 1 x 128 x
// 2048, 16 blocks: 69 us, of which the parts' way to their owners 11, A's way to
// all blocks 14, the MMAs of the pairs' lo parts 8; the products above take 159
// in 22 launches. 512 threads a block are no faster.
constexpr int CL_THREADS = 256;
constexpr int CL_STEP = CL_THREADS / 128 * 32;           // columns that a quarter of the accumulator's rows is read in
constexpr int CL_SIDE = 128, CL_TILES = 3;               // rows, and 64-column tiles of a block at most
constexpr int CL_BOX = CL_SIDE * 128;                    // bytes of a tile
constexpr int CL_X = 0;                                  // hi tiles, lo tiles
constexpr int CL_A = CL_X + 2 * CL_TILES * CL_BOX;       // two hi tiles, two lo tiles
constexpr int CL_PARTS = CL_A + 4 * CL_BOX;              // the parts of the owned rows, FP32; in the end the warps' staging
constexpr int CL_PARTS_BYTES = CL_SIDE * CL_SIDE * 4;
constexpr int CL_MISC = CL_PARTS + CL_PARTS_BYTES;       // barrier, TMEM address, abort flag
constexpr int CL_BYTES = 1024 + CL_MISC + 16;
constexpr uint32_t CL_TMEM_A = 0, CL_TMEM_B = 128, CL_TMEM_X = 256;
constexpr int MAX_CLUSTER = 16;
static_assert(CL_BYTES <= 227 * 1024, "shared memory budget");
static_assert(CL_PARTS_BYTES >= CL_THREADS / 32 * STAGING_BYTES, "staging of the last product");

constexpr uint32_t ST_CLUSTER = 0x47;

struct ClusterArgs {
  PreArgs pre;          // the matrices, their norms' parts
  NsArgs f;             // FINAL: m, n, scale, result ..
  int tiles;            // of a block
  int steps;
};

// Generic writes of this thread, in any block's shared memory, before later MMAs.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// Byte of the 8 columns of chunk q (of all columns) of a row of 128-byte-swizzled tiles.
__device__ __forceinline__ uint32_t cl_chunk(int row, int q) {
  return static_cast<uint32_t>((q >> 3) * CL_BOX + row * 128 + (((q & 7) ^ (row & 7)) << 4));
}
// Byte of chunk q (4 columns) of an owned row in a part: the rows of a chunk side
// by side, because a warp's store takes one chunk of 32 rows (with a row's chunks
// side by side instead 1 x 128 x 2048 took 77 us, not 66 at that time), turned by the chunk so
// that the owner's reads of a row meet different banks.
__device__ __forceinline__ uint32_t cl_part(int q, int in, int owned) {
  return static_cast<uint32_t>(q * owned + (in + (q >> 1)) % owned) * 16;
}
// 32 values of a row from column c0 on as pairs into tiles, lo `lo_at` bytes behind hi.
__device__ __forceinline__ void cl_store_pairs(uint32_t tiles, uint32_t lo_at, int row, int c0, const float (&v)[32]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) split_half2(v[q * 8 + 2 * j], v[q * 8 + 2 * j + 1], &h[j], &l[j]);
    const uint32_t at = tiles + cl_chunk(row, c0 / 8 + q);
    st_shared_v4(at, h[0], h[1], h[2], h[3]);
    st_shared_v4(at + lo_at, l[0], l[1], l[2], l[3]);
  }
}
// The last product's block of a tall matrix: lane: a column, v: its 32 rows from j0 on.
template <typename T>
__device__ __forceinline__ void store_column(const NsArgs& a, int col, int j0, int e, const float (&v)[32]) {
  if (col >= a.n) return;
  T* p = static_cast<T*>(a.result) + (static_cast<int64_t>(e) * a.m + j0) * a.n + col;
  constexpr int G = 16;
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += G) {
    T old[G];
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (a.update && j0 + r0 + i < a.m) old[i] = p[static_cast<int64_t>(r0 + i) * a.n];
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (j0 + r0 + i < a.m)
        p[static_cast<int64_t>(r0 + i) * a.n] =
            from_f32<T>(a.update ? fmaf(a.keep, to_f32(old[i]), -a.rate * v[r0 + i]) : v[r0 + i]);
  }
}

template <typename T, bool MOMENTUM, bool TALL>
__global__ void __launch_bounds__(CL_THREADS, 1) ns_cluster_kernel(const __grid_constant__ ClusterArgs args, int cluster) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* done = reinterpret_cast<uint64_t*>(smem + CL_MISC);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + CL_MISC + 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + CL_MISC + 12);
  __shared__ float2 factors;
  const PreArgs& pre = args.pre;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = cluster > 1 ? static_cast<int>(blockIdx.x) % cluster : 0;
  const int64_t e = blockIdx.x / cluster;
  const int s = TALL ? pre.c : pre.r, l = TALL ? pre.r : pre.c;
  const int s16 = (s + 15) & ~15, cols = args.tiles * 64, first = rank * cols;
  if (threadIdx.x == 0) {
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    tmem_alloc(tmem_holder, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  if (cluster > 1) cluster_sync();   // every block runs before another one writes into it
  grid_dependency_wait();
  launch_dependents();

  // X = u / (norm + eps)
  if (warp == 1) {
    double sum = 0.0;
    for (int i = lane; i < pre.chunks; i += 32) sum += pre.partial[e * pre.chunks + i];
    sum = warp_sum(sum);
    if (lane == 0) factors = scale_of(sum, pre.eps);
  }
  __syncthreads();
  const float s1 = factors.x, s2 = factors.y;
  const T* gp = static_cast<const T*>(pre.g) + e * pre.n;
  const float* mp = MOMENTUM ? pre.m + e * pre.n : nullptr;
  const uint32_t x_at = smem_u32(smem + CL_X), a_at = smem_u32(smem + CL_A), parts_at = smem_u32(smem + CL_PARTS);
  constexpr uint32_t X_LO = CL_TILES * CL_BOX, A_LO = 2 * CL_BOX;
  if (!TALL) {
    const int per_row = cols / 8, groups = per_row * s16;
    for (int i0 = threadIdx.x; i0 < groups; i0 += PRE_GROUP * CL_THREADS) {
      Eight<T> g[PRE_GROUP];
      Eight<float> m[PRE_GROUP];
#pragma unroll
      for (int k = 0; k < PRE_GROUP; ++k) {
        const int i = i0 + k * CL_THREADS, row = i / per_row, col = first + (i - row * per_row) * 8;
        const int n = i < groups && row < s ? max(min(l - col, 8), 0) : 0;
        const int64_t at = static_cast<int64_t>(row) * l + col;
        if (pre.vec && l % 8 == 0 && n == 8) {
          load8<T>(gp + at, g[k]);
          if (MOMENTUM) load8<float>(mp + at, m[k]);
        } else {
          load_some<T>(gp + at, n, g[k]);
          if (MOMENTUM) load_some<float>(mp + at, n, m[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < PRE_GROUP; ++k) {
        const int i = i0 + k * CL_THREADS, row = i / per_row, q = i - row * per_row;
        if (i >= groups) continue;
        uint32_t h[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float u[2];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            u[b] = to_f32(g[k].e[2 * j + b]);
            if (MOMENTUM) u[b] = update_of(pre, u[b], m[k].e[2 * j + b]);
            u[b] = u[b] * s1 * s2;
          }
          split_half2(u[0], u[1], &h[j], &lo[j]);
        }
        const uint32_t to = x_at + cl_chunk(row, q);
        st_shared_v4(to, h[0], h[1], h[2], h[3]);
        st_shared_v4(to + X_LO, lo[0], lo[1], lo[2], lo[3]);
      }
    }
  } else {
    // A warp takes rows of G (one column of X each), a lane every 32nd element.
    constexpr int ROWS = 4, PART = CL_SIDE / 32;
    for (int j0 = warp * ROWS; j0 < cols; j0 += CL_THREADS / 32 * ROWS) {
      T g[ROWS][PART];
      float m[ROWS][PART];
#pragma unroll
      for (int k = 0; k < ROWS; ++k)
#pragma unroll
        for (int b = 0; b < PART; ++b) {
          const int j = first + j0 + k, i = lane + 32 * b;
          const int64_t at = static_cast<int64_t>(j) * s + i;
          const bool in = j < l && i < s;
          g[k][b] = in ? gp[at] : from_f32<T>(0.0f);
          if (MOMENTUM) m[k][b] = in ? mp[at] : 0.0f;
        }
#pragma unroll
      for (int k = 0; k < ROWS; ++k)
#pragma unroll
        for (int b = 0; b < PART; ++b) {
          const int j = j0 + k, i = lane + 32 * b;
          if (i >= s16) continue;
          float u = to_f32(g[k][b]);
          if (MOMENTUM) u = update_of(pre, u, m[k][b]);
          __half h, lo;
          split_half(u * s1 * s2, &h, &lo);
          uint8_t* to = smem + CL_X + cl_chunk(i, j >> 3) + (j & 7) * 2;
          *reinterpret_cast<__half*>(to) = h;
          *reinterpret_cast<__half*>(to + X_LO) = lo;
        }
    }
  }
  fence_proxy_async_all();
  __syncthreads();

  // One product at a time; after a give-up none is issued, and every wait ends at once.
  uint32_t parity = 0;
  bool in_flight = false;   // (the issuer's) a product whose end has not been seen
  auto finish = [&]() {
    if (mbar_wait_bounded(done, parity, abort_flag, args.f.status, ST_CLUSTER, WAIT_LIMIT_NS)) {
      parity ^= 1u;
      in_flight = false;
    }
    __syncwarp();
    tc_fence_after();
  };
  // D = P Q over k16 blocks of 16, both pairs.
  auto mma = [&](uint32_t d, uint32_t p, uint32_t p_lo, uint32_t q, uint32_t q_lo, bool q_mn, int n, int k16) {
    if (*abort_flag != 0) return;
    const uint32_t idesc = idesc_f16_major(false, CL_SIDE, n, false, q_mn);
    for (int k = 0; k < k16; ++k) {
      const uint32_t at = (k >> 2) * CL_BOX + (k & 3) * UMMA_K * 2;
      const uint64_t ph = sdesc_kmajor_sw128(p + at), pl = sdesc_kmajor_sw128(p + p_lo + at);
      const uint64_t qh = q_mn ? sdesc_mnmajor_sw128(q + k * 2048, CL_BOX, 1024) : sdesc_kmajor_sw128(q + at);
      const uint64_t ql = q_mn ? sdesc_mnmajor_sw128(q + q_lo + k * 2048, CL_BOX, 1024) : sdesc_kmajor_sw128(q + q_lo + at);
      umma_f16(d, ph, qh, idesc, k > 0 ? 1u : 0u);
      umma_f16(d, pl, qh, idesc, 1u);
      umma_f16(d, ph, ql, idesc, 1u);
    }
    umma_commit(done);
    in_flight = true;
  };
  const int quad = warp & 3, half = warp >> 2;
  const int row = quad * 32 + lane;   // of an accumulator
  const uint32_t t_lane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
  const bool rows_used = quad * 32 < s16;   // of the warp
  constexpr float A_SCALE = pow2(A_EXP - 2 * X_EXP);
  const int owned = s16 / cluster;   // rows of A that this block adds up (cluster divides 16)
  for (int step = 0; step < args.steps; ++step) {
    if (threadIdx.x == 0) mma(tmem + CL_TMEM_A, x_at, X_LO, x_at, X_LO, false, s16, cols / 16);
    finish();
    if (rows_used) {
      const int owner = row / owned, in = row - owner * owned;
      const uint32_t part = cluster > 1 && row < s16 ? peer_u32(smem + CL_PARTS, owner) + rank * owned * 512 : 0;
      for (int c0 = 32 * half; c0 < s16; c0 += CL_STEP) {
        uint32_t raw[32];
        __syncwarp();
        tmem_ld_32x32b_x32(t_lane + CL_TMEM_A + c0, raw);
        tmem_ld_wait();
        if (row >= s16) continue;
        if (cluster == 1) {
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(raw[j]) * A_SCALE;
          cl_store_pairs(a_at, A_LO, row, c0, v);
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            st_cluster_v4(part + cl_part(c0 / 4 + q, in, owned), raw[4 * q], raw[4 * q + 1], raw[4 * q + 2], raw[4 * q + 3]);
        }
      }
    }
    __syncwarp();
    if (cluster > 1) {
      cluster_sync();
      // The owned rows: 8 columns a thread, the parts in order.
      const int per_row = s16 / 8;
      for (int i = threadIdx.x; i < owned * per_row; i += CL_THREADS) {
        const int in = i / per_row, q = i - in * per_row, to_row = rank * owned + in;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        for (int b = 0; b < cluster; ++b) {
          const uint8_t* at = smem + CL_PARTS + b * owned * 512;
          const float4 x = *reinterpret_cast<const float4*>(at + cl_part(2 * q, in, owned));
          const float4 y = *reinterpret_cast<const float4*>(at + cl_part(2 * q + 1, in, owned));
          v[0] += x.x;
          v[1] += x.y;
          v[2] += x.z;
          v[3] += x.w;
          v[4] += y.x;
          v[5] += y.y;
          v[6] += y.z;
          v[7] += y.w;
        }
        uint32_t h[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) split_half2(v[2 * j] * A_SCALE, v[2 * j + 1] * A_SCALE, &h[j], &lo[j]);
        for (int b = 0; b < cluster; ++b) {
          const uint32_t to = peer_u32(smem + CL_A, b) + cl_chunk(to_row, q);
          st_cluster_v4(to, h[0], h[1], h[2], h[3]);
          st_cluster_v4(to + A_LO, lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_proxy_async_all();
      __syncwarp();
      cluster_sync();
    }
    fence_proxy_async_all();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // B over A: A's products are complete before B is stored.
    if (threadIdx.x == 0) mma(tmem + CL_TMEM_B, a_at, A_LO, a_at, A_LO, false, s16, s16 / 16);
    finish();
    if (rows_used)
      for (int c0 = 32 * half; c0 < s16; c0 += CL_STEP) {
        uint32_t raw[32];
        __syncwarp();
        tmem_ld_32x32b_x32(t_lane + CL_TMEM_B + c0, raw);
        tmem_ld_wait();
        if (row >= s16) continue;
        float v[32];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t at = a_at + cl_chunk(row, c0 / 8 + q);
          const uint4 h = ld_shared_v4(at), lo = ld_shared_v4(at + A_LO);
          const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&hw[j]));
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&lw[j]));
            v[q * 8 + 2 * j] = x.x + y.x;
            v[q * 8 + 2 * j + 1] = x.y + y.y;
          }
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          v[j] = fmaf(__uint_as_float(raw[j]), NS_C * pow2(B_EXP - 2 * A_EXP), v[j] * (NS_B * pow2(B_EXP - A_EXP)));
          if (c0 + j == row) v[j] += NS_A * pow2(B_EXP);
        }
        cl_store_pairs(a_at, A_LO, row, c0, v);
      }
    fence_proxy_async_all();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0) mma(tmem + CL_TMEM_X, a_at, A_LO, x_at, X_LO, true, cols, s16 / 16);
    finish();
    const bool last = step + 1 == args.steps;
    if (rows_used)
      for (int c0 = 32 * half; c0 < cols; c0 += CL_STEP) {
        uint32_t raw[32];
        __syncwarp();
        tmem_ld_32x32b_x32(t_lane + CL_TMEM_X + c0, raw);
        tmem_ld_wait();
        const float scale = last ? args.f.scale : pow2(-B_EXP);
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(raw[j]) * scale;
        if (!last) {
          if (row < s16) cl_store_pairs(x_at, X_LO, row, c0, v);
        } else if (TALL) {
          if (args.f.result_dtype == MOE_F32) store_column<float>(args.f, row, first + c0, static_cast<int>(e), v);
          else if (args.f.result_dtype == MOE_F16) store_column<__half>(args.f, row, first + c0, static_cast<int>(e), v);
          else store_column<__nv_bfloat16>(args.f, row, first + c0, static_cast<int>(e), v);
        } else {
          float* stage = reinterpret_cast<float*>(smem + CL_PARTS + warp * STAGING_BYTES);
          if (args.f.result_dtype == MOE_F32) store_result<float>(args.f, stage, quad * 32, first + c0, static_cast<int>(e), v);
          else if (args.f.result_dtype == MOE_F16) store_result<__half>(args.f, stage, quad * 32, first + c0, static_cast<int>(e), v);
          else store_result<__nv_bfloat16>(args.f, stage, quad * 32, first + c0, static_cast<int>(e), v);
        }
      }
    fence_proxy_async_all();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  if (in_flight) mbar_wait_bounded(done, parity, nullptr, args.f.status, ST_CLUSTER, WAIT_LIMIT_NS);
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, TMEM_COLS);
}

// ---------------------------------------------------------------- host side

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// FP16 [E][rows][cols] with rows `pitch` elements apart, as boxes of 64
// columns x box_rows rows.
bool enc(CUtensorMap* m, const __half* p, int64_t E, int64_t rows, int64_t cols, int64_t pitch, uint32_t box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(E)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch) * 2, static_cast<cuuint64_t>(rows * pitch) * 2};
  const cuuint32_t box[3] = {64, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half*>(p), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int64_t MAX_PART_TILES = 128;   // tiles times parts of a split product

struct Layout {
  size_t partial, x0, x1, a, b, t, b1, parts, total;
  int64_t x_pitch, s_pitch;
};
Layout layout(int64_t E, int64_t r, int64_t c) {
  Layout l;
  const int64_t s = std::min(r, c);
  l.x_pitch = (c + 7) / 8 * 8;
  l.s_pitch = (s + 7) / 8 * 8;
  const size_t x = align_up(static_cast<size_t>(E * r * l.x_pitch) * 2, 256);
  const size_t g = align_up(static_cast<size_t>(E * s * l.s_pitch) * 2, 256);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t p = at;
    at += bytes;
    return p;
  };
  l.partial = take(align_up(static_cast<size_t>(E * chunk_count(E, r * c)) * sizeof(double), 256));
  l.x0 = take(2 * x);
  l.x1 = take(2 * x);
  l.a = take(2 * g);
  l.b = take(2 * g);
  l.t = take(2 * g);
  l.b1 = take(2 * g);
  // The parts of a split product: none where its tiles alone fill the machine.
  const int64_t blocks = (s + TILE - 1) / TILE, tiles = E * blocks * blocks;
  l.parts = take(tiles <= MAX_PART_TILES / 2 ? align_up(static_cast<size_t>(MAX_PART_TILES / tiles * E * s * l.s_pitch) * 4, 256) : 0);
  l.total = at;
  return l;
}

// The tensor maps of a call's matrices, each encoded once (encoding them for
// every launch was half of a small call's time).
class Maps {
 public:
  explicit Maps(int64_t E) : E_(E) {}
  // hi and lo of p, two maps; NULL if they cannot be had.
  const CUtensorMap* of(const Pair& p, uint32_t box_rows) {
    for (int i = 0; i < n_; ++i)
      if (entry_[i].p == p.hi && entry_[i].box_rows == box_rows) return entry_[i].m;
    if (n_ == MAX) return nullptr;
    Entry& e = entry_[n_];
    if (!enc(&e.m[0], p.hi, E_, p.rows, p.cols, p.pitch, box_rows) ||
        !enc(&e.m[1], p.lo, E_, p.rows, p.cols, p.pitch, box_rows))
      return nullptr;
    e.p = p.hi;
    e.box_rows = box_rows;
    ++n_;
    return e.m;
  }

 private:
  static constexpr int MAX = 8;   // X and X' in two boxes, A, B, T, B1
  struct Entry {
    CUtensorMap m[2];
    const __half* p;
    uint32_t box_rows;
  };
  Entry entry_[MAX];
  int n_ = 0;
  int64_t E_;
};

template <int MODE, bool P_MN, bool Q_MN>
cudaError_t launch_product(int64_t E, Maps& maps, const Pair& p, const Pair& q, NsArgs args, int num_pairs, cudaStream_t s,
                           const char** why, int parts = 1) {
  const CUtensorMap* pm = maps.of(p, P_MN ? 64 : BM);
  const CUtensorMap* qm = maps.of(q, Q_MN ? 64 : BM);
  if (pm == nullptr || qm == nullptr) {
    *why = "cuTensorMapEncodeTiled rejected an operand";
    return cudaErrorInvalidValue;
  }
  args.m_blocks = (args.m + TILE - 1) / TILE;
  args.n_blocks = (args.n + TILE - 1) / TILE;
  const int64_t per = MODE == GRAM || MODE == POLY ? static_cast<int64_t>(args.n_blocks) * (args.n_blocks + 1) / 2
                                                   : static_cast<int64_t>(args.m_blocks) * args.n_blocks;
  args.tiles_per_matrix = static_cast<uint32_t>(per);
  args.tiles = static_cast<uint32_t>(E * per * parts);
  const int64_t pairs = std::min<int64_t>(args.tiles, num_pairs);
  return launch_dependent(ns_kernel<MODE, P_MN, Q_MN>, dim3(static_cast<unsigned>(2 * pairs)), dim3(NUM_THREADS),
                          SMEM_BYTES, s, pm[0], pm[1], qm[0], qm[1], args);
}

// A matrix's X X^T in parts of K, where whole tiles would leave most block
// pairs idle: the number of parts (1: not split). With few tiles a pair is
// bound by the 64 KB that each of its k-blocks brings into one SM: one 128 x
// 2048 matrix took 33 us in one tile.
int gram_parts(int64_t E, int64_t s, int64_t l, int num_pairs) {
  const int64_t blocks = (s + TILE - 1) / TILE, tiles = E * blocks * blocks, k_blocks = (l + BK - 1) / BK;
  const int64_t parts = std::min<int64_t>(std::min<int64_t>(num_pairs, MAX_PART_TILES) / tiles, k_blocks / 2);
  return parts < 2 ? 1 : static_cast<int>(parts);
}

// Two steps at once, X'' = B1 (B X) = (B1 B) X with B1 from X' X'^T = B A B,
// take three more s x s products instead of a second X X^T and B X: 3 s^2 (l - s)
// multiplications less a matrix (symmetric products count half), and two
// launches more, about 10 us or 2e9 of them.
bool two_steps_pay(int64_t E, int64_t s, int64_t l) {
  return static_cast<double>(E) * s * s * (l - s) > 2e9;
}

cudaError_t allow_shared_memory() {
  const void* kernels[] = {
      reinterpret_cast<const void*>(ns_kernel<GRAM, false, false>),
      reinterpret_cast<const void*>(ns_kernel<GRAM, true, true>),
      reinterpret_cast<const void*>(ns_kernel<GRAM_PART, false, false>),
      reinterpret_cast<const void*>(ns_kernel<GRAM_PART, true, true>),
      reinterpret_cast<const void*>(ns_kernel<POLY, false, false>),
      reinterpret_cast<const void*>(ns_kernel<APPLY, false, false>),
      reinterpret_cast<const void*>(ns_kernel<APPLY, false, true>),
      reinterpret_cast<const void*>(ns_kernel<FINAL, false, false>),
      reinterpret_cast<const void*>(ns_kernel<FINAL, false, true>),
  };
  for (const void* k : kernels) {
    const cudaError_t err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

// Block pairs that the current device runs at once: SMs left single in a
// cluster of SMs take none, and a pair too many would run after all the others.
// Once per device, with the kernels' shared memory.
cudaError_t resident_pairs(int* pairs) {
  constexpr int MAX_DEVICES = 64;
  static std::atomic<int> known[MAX_DEVICES];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < MAX_DEVICES && (*pairs = known[dev].load(std::memory_order_acquire)) > 0) return cudaSuccess;
  if ((err = allow_shared_memory()) != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  err = cudaOccupancyMaxActiveClusters(pairs, ns_kernel<POLY, false, false>, &cfg);
  if (err != cudaSuccess) return err;
  if (*pairs < 1) return cudaErrorLaunchOutOfResources;
  if (dev < MAX_DEVICES) known[dev].store(*pairs, std::memory_order_release);
  return cudaSuccess;
}

// Clusters of a size (16 >> i) that the current device runs at once; 0 for none.
cudaError_t resident_clusters(int i, int* count) {
  constexpr int MAX_DEVICES = 64;
  static std::atomic<int> known[MAX_DEVICES][5];   // one more than the count
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < MAX_DEVICES && (*count = known[dev][i].load(std::memory_order_acquire) - 1) >= 0) return cudaSuccess;
  const auto kernel = ns_cluster_kernel<float, false, false>;
  if ((err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, CL_BYTES)) != cudaSuccess ||
      (err = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
    return err;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {static_cast<unsigned>(MAX_CLUSTER >> i), 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(MAX_CLUSTER >> i));
  cfg.blockDim = dim3(CL_THREADS);
  cfg.dynamicSmemBytes = CL_BYTES;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  err = cudaOccupancyMaxActiveClusters(count, kernel, &cfg);
  if (err == cudaErrorInvalidClusterSize) {   // a device that does not take clusters of this size
    cudaGetLastError();
    *count = 0;
  } else if (err != cudaSuccess) {
    return err;
  }
  if (dev < MAX_DEVICES) known[dev][i].store(*count + 1, std::memory_order_release);
  return cudaSuccess;
}

// Blocks of a matrix's cluster, and 64-column tiles of a block; 0 blocks: the
// matrices go through the products above. By the time that either takes, in
// microseconds for five steps, fitted to sides of 16 to 128 x 64 to 2048 and 1
// to 1000 matrices: waves of clusters against 22 launches and their tiles.
// Measured, clusters against products: 1 x 128 x 2048 69 / 159, 8 x 128 x 2048
// 134 / 166, 16 x 128 x 2048 199 / 197, 128 x 128 x 192 50 / 188, 128 x 64 x 512
// 141 / 209, 1000 x 64 x 64 149 / 367, 32 x 128 x 1500 209 / 233.
struct ClusterShape {
  int blocks, tiles;
};
cudaError_t cluster_shape(int64_t E, int64_t s, int64_t l, ClusterShape* best) {
  *best = {0, 0};
  if (s > CL_SIDE || l > 64 * CL_TILES * MAX_CLUSTER) return cudaSuccess;
  const double side = static_cast<double>((s + 15) / 16) / 8, long_side = static_cast<double>(l);
  double least = 90.0 + 0.026 * long_side + static_cast<double>(E) * (0.2 + 0.00125 * long_side);
  for (int i = 0; i < 5; ++i) {
    const int64_t blocks = MAX_CLUSTER >> i, tiles = ((l + blocks - 1) / blocks + 63) / 64;
    if (tiles > CL_TILES) continue;
    int count = 0;
    const cudaError_t err = resident_clusters(i, &count);
    if (err != cudaSuccess) return err;
    if (count < 1) continue;
    constexpr double EXCHANGE[] = {26.0, 18.0, 12.0, 10.0, 0.0};   // of A's parts, by i
    const double wave = 20.0 + side * (10.0 + 4.0 * static_cast<double>(tiles)) + side * side * EXCHANGE[i];
    const double time = static_cast<double>((E + count - 1) / count) * wave;
    if (time < least) {
      least = time;
      *best = {static_cast<int>(blocks), static_cast<int>(tiles)};
    }
  }
  return cudaSuccess;
}

template <typename T, bool MOMENTUM>
cudaError_t launch_squares(const PreArgs& a, int64_t E, cudaStream_t s) {
  return launch_dependent(squares_kernel<T, MOMENTUM>, dim3(a.chunks, static_cast<unsigned>(E)), dim3(PRE_THREADS), 0, s,
                          a);
}

// What can be refused is refused before the squares' launch, which updates the momentum.
template <typename T, bool MOMENTUM, bool TALL>
cudaError_t launch_cluster(const ClusterArgs& a, int64_t E, int blocks, cudaStream_t s) {
  const auto kernel = ns_cluster_kernel<T, MOMENTUM, TALL>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, CL_BYTES);
  if (err == cudaSuccess) err = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (err == cudaSuccess) err = launch_squares<T, MOMENTUM>(a.pre, E, s);
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(blocks), 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(E * blocks));
  cfg.blockDim = dim3(CL_THREADS);
  cfg.dynamicSmemBytes = CL_BYTES;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = blocks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, blocks);
}

template <typename T, bool MOMENTUM>
cudaError_t launch_small(const ClusterArgs& a, int64_t E, int blocks, cudaStream_t s) {
  return a.pre.r > a.pre.c ? launch_cluster<T, MOMENTUM, true>(a, E, blocks, s)
                           : launch_cluster<T, MOMENTUM, false>(a, E, blocks, s);
}
template <typename T>
cudaError_t launch_small(const ClusterArgs& a, int64_t E, int blocks, cudaStream_t s) {
  return a.pre.m != nullptr ? launch_small<T, true>(a, E, blocks, s) : launch_small<T, false>(a, E, blocks, s);
}

template <typename T, bool MOMENTUM>
cudaError_t launch_pre(const PreArgs& a, int64_t E, cudaStream_t s) {
  const cudaError_t err = launch_squares<T, MOMENTUM>(a, E, s);
  if (err != cudaSuccess) return err;
  // Several rounds a block where there is work for all SMs: its start costs as much as one.
  const int64_t groups = a.pitch / 8 * a.r;
  const int64_t rounds = std::max<int64_t>(1, std::min<int64_t>(8, E * groups / (PRE_BLOCKS * PRE_THREADS * PRE_GROUP)));
  const int64_t per_block = rounds * PRE_GROUP * PRE_THREADS;
  return launch_dependent(first_x_kernel<T, MOMENTUM>,
                          dim3(static_cast<unsigned>((groups + per_block - 1) / per_block), static_cast<unsigned>(E)),
                          dim3(PRE_THREADS), 0, s, a);
}
template <typename T>
cudaError_t launch_pre(const PreArgs& a, int64_t E, cudaStream_t s) {
  return a.m != nullptr ? launch_pre<T, true>(a, E, s) : launch_pre<T, false>(a, E, s);
}

}  // namespace

size_t newton_schulz_scratch_bytes(int64_t E, int64_t r, int64_t c) { return layout(E, r, c).total; }

int64_t newton_schulz_tiles(int64_t E, int64_t r, int64_t c) {
  const int64_t most = std::max(r, c);
  return E * ((most + BM - 1) / BM) * ((most + BM - 1) / BM);
}

cudaError_t launch_newton_schulz(const NewtonSchulz& o, void* scratch, cudaStream_t stream, const char** why) {
  const int64_t E = o.E, r = o.rows, c = o.cols, s = std::min(r, c);
  if (E == 0 || r == 0 || c == 0) return cudaSuccess;
  uint32_t* status = nullptr;
  cudaError_t err = device_status_ptr(&status);
  if (err != cudaSuccess) return err;
  int pairs = 0;
  err = resident_pairs(&pairs);
  if (err != cudaSuccess) return err;
  const Layout l = layout(E, r, c);
  uint8_t* base = static_cast<uint8_t*>(scratch);
  auto pair = [&](size_t at, int64_t rows, int64_t cols, int64_t pitch) {
    Pair p;
    p.hi = reinterpret_cast<__half*>(base + at);
    p.lo = reinterpret_cast<__half*>(base + at + align_up(static_cast<size_t>(E * rows * pitch) * 2, 256));
    p.rows = rows;
    p.cols = cols;
    p.pitch = pitch;
    return p;
  };
  Pair x = pair(l.x0, r, c, l.x_pitch), next = pair(l.x1, r, c, l.x_pitch);
  const Pair a = pair(l.a, s, s, l.s_pitch), b = pair(l.b, s, s, l.s_pitch);
  const Pair t = pair(l.t, s, s, l.s_pitch), b1 = pair(l.b1, s, s, l.s_pitch);

  PreArgs pre{};
  pre.g = o.grad;
  pre.m = o.momentum;
  pre.partial = reinterpret_cast<double*>(base + l.partial);
  pre.hi = x.hi;
  pre.lo = x.lo;
  pre.n = r * c;
  pre.chunk = chunk_elems(E, pre.n);
  pre.pitch = l.x_pitch;
  pre.r = static_cast<int>(r);
  pre.c = static_cast<int>(c);
  pre.chunks = static_cast<int>(chunk_count(E, pre.n));
  pre.nesterov = o.nesterov;
  pre.vec = pre.n % 8 == 0 && reinterpret_cast<uintptr_t>(o.grad) % 16 == 0 &&
            reinterpret_cast<uintptr_t>(o.momentum) % 16 == 0;
  pre.mu = o.momentum_decay;
  pre.eps = o.eps;
  NsArgs f{};   // of the last product
  f.status = status;
  f.m = static_cast<int>(r);
  f.n = static_cast<int>(c);
  f.k = static_cast<int>(s);
  f.result = o.result;
  f.result_dtype = o.result_dtype;
  f.update = o.update;
  f.keep = o.keep;
  f.rate = o.rate;
  // A result over gradients of another size (or place) would end up on matrices
  // that are yet to be read: other clusters start later.
  const size_t from_bytes = static_cast<size_t>(E * pre.n) * dtype_size(static_cast<moe_dtype>(o.grad_dtype));
  const size_t to_bytes = static_cast<size_t>(E * pre.n) * dtype_size(static_cast<moe_dtype>(o.result_dtype));
  const uintptr_t from = reinterpret_cast<uintptr_t>(o.grad), to = reinterpret_cast<uintptr_t>(o.result);
  const bool over = from < to + to_bytes && to < from + from_bytes && (from != to || from_bytes != to_bytes);
  ClusterShape shape{0, 0};
  if (!over && (err = cluster_shape(E, s, std::max(r, c), &shape)) != cudaSuccess) return err;
  if (shape.blocks > 0) {
    ClusterArgs args{pre, f, shape.tiles, o.steps};
    args.f.scale = pow2(-B_EXP - X_EXP);
    return o.grad_dtype == MOE_F32   ? launch_small<float>(args, E, shape.blocks, stream)
           : o.grad_dtype == MOE_F16 ? launch_small<__half>(args, E, shape.blocks, stream)
                                     : launch_small<__nv_bfloat16>(args, E, shape.blocks, stream);
  }

  // The maps that the products will ask for: one that cannot be had is an error
  // before the first launch, which updates the momentum.
  const bool tall = r > c, by_two = two_steps_pay(E, s, std::max(r, c));
  Maps maps(E);
  const uint32_t gram_box = tall ? 64 : BM, apply_box = tall ? BM : 64;   // of X along its rows, or across
  bool have = maps.of(x, gram_box) && maps.of(x, apply_box) && maps.of(a, BM) && maps.of(b, BM);
  if (by_two && o.steps >= 2) have = have && maps.of(t, BM) && maps.of(b1, BM);
  if (o.steps > (by_two ? 2 : 1)) have = have && maps.of(next, gram_box) && maps.of(next, apply_box);
  if (!have) {
    *why = "cuTensorMapEncodeTiled rejected an operand";
    return cudaErrorInvalidValue;
  }

  err = o.grad_dtype == MOE_F32   ? launch_pre<float>(pre, E, stream)
        : o.grad_dtype == MOE_F16 ? launch_pre<__half>(pre, E, stream)
                                  : launch_pre<__nv_bfloat16>(pre, E, stream);
  if (err != cudaSuccess) return err;

  // Every part has k-blocks: the last ones may take fewer.
  int parts = gram_parts(E, s, std::max(r, c), pairs);
  const int k_blocks = static_cast<int>((std::max(r, c) + BK - 1) / BK);
  const int split = (k_blocks + parts - 1) / parts;
  parts = (k_blocks + split - 1) / split;
  NsArgs sq{};
  sq.status = status;
  sq.m = sq.n = static_cast<int>(s);
  sq.pitch = l.s_pitch;
  // out = X X^T (X^T X)
  auto gram = [&](const Pair& out) {
    NsArgs g = sq;
    g.k = static_cast<int>(tall ? r : c);
    g.square = 1;
    g.out = out;
    g.scale = pow2(A_EXP - 2 * X_EXP);
    if (parts == 1)
      return tall ? launch_product<GRAM, true, true>(E, maps, x, x, g, pairs, stream, why)
                  : launch_product<GRAM, false, false>(E, maps, x, x, g, pairs, stream, why);
    g.parts = reinterpret_cast<float*>(base + l.parts);
    g.part_elems = E * s * l.s_pitch;
    g.k_split = split;
    const cudaError_t e = tall ? launch_product<GRAM_PART, true, true>(E, maps, x, x, g, pairs, stream, why, parts)
                               : launch_product<GRAM_PART, false, false>(E, maps, x, x, g, pairs, stream, why, parts);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (g.part_elems / 4 + PRE_THREADS - 1) / PRE_THREADS;
    return launch_dependent(join_parts_kernel, dim3(static_cast<unsigned>(blocks)), dim3(PRE_THREADS), 0, stream,
                            static_cast<const float*>(g.parts), g.part_elems, parts, g.scale, out.hi, out.lo);
  };
  // out = a I + b A + c A A
  auto poly = [&](const Pair& in, const Pair& out) {
    NsArgs p = sq;
    p.k = static_cast<int>(s);
    p.square = 1;
    p.out = out;
    p.a = in;
    p.scale = NS_C * pow2(B_EXP - 2 * A_EXP);
    p.a_scale = NS_B * pow2(B_EXP - A_EXP);
    p.diag = NS_A * pow2(B_EXP);
    return launch_product<POLY, false, false>(E, maps, in, in, p, pairs, stream, why);
  };
  // out = P Q of polynomials in the same A: symmetric
  auto product = [&](const Pair& p, const Pair& q, const Pair& out, int exp) {
    NsArgs g = sq;
    g.k = static_cast<int>(s);
    g.out = out;
    g.scale = pow2(exp);
    return launch_product<GRAM, false, false>(E, maps, p, q, g, pairs, stream, why);
  };
  for (int left = o.steps; left > 0;) {
    const int now = by_two && left >= 2 ? 2 : 1;
    left -= now;
    if ((err = gram(a)) != cudaSuccess || (err = poly(a, b)) != cudaSuccess) return err;
    Pair q = b;
    int q_exp = B_EXP;
    if (now == 2) {
      // X'' = B1 B X with B1 from A1 = X' X'^T = B A B
      if ((err = product(b, a, t, A_EXP - A_EXP - B_EXP)) != cudaSuccess ||
          (err = product(t, b, a, A_EXP - A_EXP - B_EXP)) != cudaSuccess || (err = poly(a, b1)) != cudaSuccess ||
          (err = product(b1, b, t, BB_EXP - 2 * B_EXP)) != cudaSuccess)
        return err;
      q = t;
      q_exp = BB_EXP;
    }
    if (left > 0) {
      f.out = next;
      f.scale = pow2(-q_exp);
      err = tall ? launch_product<APPLY, false, false>(E, maps, x, q, f, pairs, stream, why)
                 : launch_product<APPLY, false, true>(E, maps, q, x, f, pairs, stream, why);
    } else {
      f.scale = pow2(-q_exp - X_EXP);
      err = tall ? launch_product<FINAL, false, false>(E, maps, x, q, f, pairs, stream, why)
                 : launch_product<FINAL, false, true>(E, maps, q, x, f, pairs, stream, why);
    }
    if (err != cudaSuccess) return err;
    std::swap(x, next);
  }
  return cudaSuccess;
}

}  // namespace moe
