// Orthogonalised updates by Newton-Schulz products, on the tensor cores.
//
// For each matrix G [r, c] of a batch (s = min(r, c), the short side):
//   X = G / (|G|_F + eps), then per step, with A = X X^T (X^T X where r > c)
//   and a, b, c = 3.4445, -4.7750, 2.0315:
//   X <- B X (X B),  B = a I + b A + c A A = a I + A (b I + c A)
// which moves every singular value of X from (0, 1] towards the interval
// [0.7, 1.21] and keeps its singular vectors. Three grouped products a step:
//   GRAM   A and C = b I + c A   (symmetric: the tiles on and above the
//          diagonal are computed, each also stored mirrored)
//   POLY   B = A C + a I         (symmetric too)
//   APPLY  X' = B X, or X B; in the last step its epilogue writes the result
//          (16-bit, or the weights' update) instead of X'
//
// Precision. The map multiplies small singular values by 3.4 a step, 485 in
// five, and with them every rounding error made before: 16-bit operands alone
// (half a step of 2^-11 or 2^-8) leave errors of 5 % and more along the weak
// directions. Operands are pairs of FP16 instead, v = hi + lo, lo the FP16 of
// v - hi, and a product is hi hi + hi lo + lo hi: 22 bits, for three MMAs.
// FP16 rather than BF16 pairs (16 bits) because every value here is bounded:
// |X| <= 1.21 (its largest singular value: the quintic maps [0, 1.21] into
// itself), |A| <= 1.47, |C| <= 4.78, |B| <= 3.45. Stored times 2^14 (X, A) or
// 2^13 (C, B) they stay under FP16's 65504, and lo of an entry as small as
// 2^-14 is still a normal FP16.
//
// Structure: one persistent CTA per SM, tiles of 128 x 256 with K in blocks of
// 64; warp 0 issues the TMA copies, warp 1 the MMAs, warps 2..9 drain TMEM,
// whose two 256-column accumulators let one tile's epilogue run under the next
// one's MMAs. Operands along their rows (K contiguous) are K-major tiles, X as
// a right-hand side and X^T X read X as it is stored, MN-major. Waits are
// bounded; one that runs out records a code and the CTA winds down.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "moe_common.cuh"
#include "moe_internal.h"
#include "ring_drain.h"

namespace moe {
namespace {

constexpr float NS_A = 3.4445f, NS_B = -4.7750f, NS_C = 2.0315f;
constexpr float pow2(int e) { return e == 0 ? 1.0f : e > 0 ? 2.0f * pow2(e - 1) : 0.5f * pow2(e + 1); }
constexpr int X_EXP = 14, A_EXP = 14, C_EXP = 13, B_EXP = 13;   // stored = value * 2^EXP
// Accumulators to stored values, and what is added on the diagonal.
constexpr float GRAM_TO_A = pow2(A_EXP - 2 * X_EXP), GRAM_TO_C = NS_C * pow2(C_EXP - 2 * X_EXP);
constexpr float C_DIAG = NS_B * pow2(C_EXP), B_DIAG = NS_A * pow2(B_EXP);
constexpr float POLY_TO_B = pow2(B_EXP - A_EXP - C_EXP), APPLY_TO_X = pow2(-B_EXP);
constexpr float APPLY_TO_RESULT = pow2(-B_EXP - X_EXP);

// ---------------------------------------------------------------- norm, momentum, first X

constexpr int PRE_THREADS = 256;
constexpr int MAX_CHUNKS = 256;      // partial sums per matrix
constexpr int64_t MIN_CHUNK = 16384; // elements

__host__ __device__ inline int64_t chunk_elems(int64_t n) {
  const int64_t c = (n + MAX_CHUNKS - 1) / MAX_CHUNKS;
  return (c < MIN_CHUNK ? MIN_CHUNK : c + 7) / 8 * 8;
}
inline int64_t chunk_count(int64_t n) { return (n + chunk_elems(n) - 1) / chunk_elems(n); }

template <typename T>
struct alignas(16) Eight {
  T e[8];
};
template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, bool vec, float (&v)[8]) {
  if (vec) {
    Eight<T> x;
    const uint4* s = reinterpret_cast<const uint4*>(p);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(x) / 16); ++i) reinterpret_cast<uint4*>(&x)[i] = s[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(x.e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32(p[i]) : 0.0f;
  }
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

__device__ __forceinline__ double block_sum(double v, double* sm) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(FULL_MASK, v, off);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < PRE_THREADS / 32 ? sm[threadIdx.x & 31] : 0.0;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(FULL_MASK, v, off);
  return v;
}

struct PreArgs {
  const void* g;       // [E, r, c]
  float* m;            // momentum [E, r, c] or NULL
  double* partial;     // [E, chunks]
  __half* hi;          // X [E, r, pitch]
  __half* lo;
  int64_t n, chunk;    // elements of a matrix, of a chunk
  int64_t pitch;
  int r, c, chunks, nesterov, vec;
  float mu;
  double eps;
};

// u of the momentum step: what is orthogonalised.
__device__ __forceinline__ float update_of(const PreArgs& a, float g, float m) {
  return a.nesterov ? fmaf(a.mu, m, g) : m;
}

// partial[e][chunk]: the sum of squares of the chunk's u; updates the momentum.
template <typename T>
__global__ void __launch_bounds__(PRE_THREADS) squares_kernel(const PreArgs a) {
  __shared__ double sm[PRE_THREADS / 32];
  grid_dependency_wait();
  launch_dependents();
  const int64_t base = blockIdx.y * a.n;
  const int64_t lo = blockIdx.x * a.chunk, hi = min(lo + a.chunk, a.n);
  double total = 0.0;
  // Rounds of a few elements in FP32, the rounds in FP64.
  constexpr int G = 4;
  for (int64_t i0 = lo; i0 < hi; i0 += PRE_THREADS * 8 * G) {
    Squares s{0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < G; ++k) {
      const int64_t i = i0 + (k * PRE_THREADS + static_cast<int64_t>(threadIdx.x)) * 8;
      if (i >= hi) continue;
      const int n = static_cast<int>(min(hi - i, int64_t{8}));
      const bool vec = a.vec && n == 8;
      float g[8];
      load8<T>(static_cast<const T*>(a.g) + base + i, n, vec, g);
      if (a.m != nullptr) {
        float m[8];
        float* p = a.m + base + i;
        load8<float>(p, n, vec, m);
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = fmaf(a.mu, m[j], g[j]);
        if (vec) {
          reinterpret_cast<float4*>(p)[0] = make_float4(m[0], m[1], m[2], m[3]);
          reinterpret_cast<float4*>(p)[1] = make_float4(m[4], m[5], m[6], m[7]);
        } else {
          for (int j = 0; j < n; ++j) p[j] = m[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = update_of(a, g[j], m[j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) s.add(g[j]);
    }
    total += s.total();
  }
  total = block_sum(total, sm);
  if (threadIdx.x == 0) a.partial[static_cast<int64_t>(blockIdx.y) * a.chunks + blockIdx.x] = total;
}

__device__ __forceinline__ void split_half(float v, __half* hi, __half* lo) {
  *hi = __float2half_rn(v);
  *lo = __float2half_rn(v - __half2float(*hi));
}

// X = u / (norm + eps), as FP16 pairs.
template <typename T>
__global__ void __launch_bounds__(PRE_THREADS) first_x_kernel(const PreArgs a) {
  __shared__ double sm[PRE_THREADS / 32];
  grid_dependency_wait();
  launch_dependents();
  const int64_t e = blockIdx.y;
  double sum = static_cast<int>(threadIdx.x) < a.chunks ? a.partial[e * a.chunks + threadIdx.x] : 0.0;
  static_assert(MAX_CHUNKS <= PRE_THREADS, "one partial sum a thread");
  sum = block_sum(sum, sm);
  // 2^14 / (norm + eps) as two FP32 factors, both far from FP32's ends. A
  // matrix with a NaN or an infinity becomes NaN as a whole.
  const double scale = isfinite(sum) ? 0x1p14 / (sqrt(sum) + a.eps) : nan("");
  int ex = 0;
  const double frac = frexp(scale, &ex);
  const float s1 = static_cast<float>(ldexp(frac, ex - ex / 2)), s2 = static_cast<float>(ldexp(1.0, ex / 2));
  const int64_t per_row = a.pitch / 8, groups = per_row * a.r;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * PRE_THREADS + threadIdx.x; i < groups;
       i += static_cast<int64_t>(gridDim.x) * PRE_THREADS) {
    const int64_t row = i / per_row, col = (i - row * per_row) * 8;
    const int n = static_cast<int>(min(a.c - col, int64_t{8}));
    const int64_t at = e * a.n + row * a.c + col;
    const bool vec = a.vec && a.c % 8 == 0;
    float g[8];
    load8<T>(static_cast<const T*>(a.g) + at, n, vec, g);
    if (a.m != nullptr) {
      float m[8];
      load8<float>(a.m + at, n, vec, m);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = update_of(a, g[j], m[j]);
    }
    Eight<__half> h, l;
#pragma unroll
    for (int j = 0; j < 8; ++j) split_half(g[j] * s1 * s2, &h.e[j], &l.e[j]);
    const int64_t to = (e * a.r + row) * a.pitch + col;
    *reinterpret_cast<uint4*>(a.hi + to) = *reinterpret_cast<const uint4*>(&h);
    *reinterpret_cast<uint4*>(a.lo + to) = *reinterpret_cast<const uint4*>(&l);
  }
}

// ---------------------------------------------------------------- the products

enum NsMode { GRAM = 0, POLY = 1, APPLY = 2, FINAL = 3 };

constexpr int BM = 128, BN = 256, BK = 64, UMMA_K = 16;
constexpr int BOX = 64 * 128;                        // 64 x 64 elements, or 64 rows of 128 bytes
constexpr int P_BYTES = BM * BK * 2, Q_BYTES = BN * BK * 2;
constexpr int STAGE_BYTES = 2 * (P_BYTES + Q_BYTES); // hi and lo of both operands
constexpr int STAGES = 2;
constexpr uint32_t TMEM_COLS = 512;
constexpr int NUM_EPI_WARPS = 8;
constexpr int NUM_THREADS = 32 * (2 + NUM_EPI_WARPS);
constexpr uint64_t WAIT_LIMIT_NS = 1000000000ull;
constexpr int SMEM_BAR = STAGES * STAGE_BYTES;
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

// D [E, m, n] = P [E, m, k] Q [E, k, n], both FP16 pairs.
struct NsArgs {
  int m, n, k;
  int m_blocks, n_blocks;
  uint32_t tiles, tiles_per_matrix;
  __half* out_hi;       // GRAM A, POLY B, APPLY X': [E, m, pitch]
  __half* out_lo;
  __half* out2_hi;      // GRAM C
  __half* out2_lo;
  int64_t pitch;
  void* result;         // FINAL: [E, m, n] in result_dtype
  int result_dtype;
  int result_vec;       // rows and pointer 16-byte aligned
  int update;           // FINAL: result = keep * result - rate * X' (weights), else X'
  float keep, rate;
  uint32_t* status;
};

// Tile -> (matrix, row block, column block). Symmetric products have the
// tiles whose 256 columns reach the diagonal or lie right of it.
struct NsTile {
  int e, mb, nb;
};
template <bool TRI>
__device__ __forceinline__ NsTile ns_tile(uint32_t tile, const NsArgs& a) {
  NsTile t;
  t.e = static_cast<int>(tile / a.tiles_per_matrix);
  int i = static_cast<int>(tile % a.tiles_per_matrix);
  if (TRI) {
    t.mb = 0;
    while (i >= a.n_blocks - t.mb / 2) {
      i -= a.n_blocks - t.mb / 2;
      ++t.mb;
    }
    t.nb = t.mb / 2 + i;
  } else {
    t.mb = i % a.m_blocks;
    t.nb = i / a.m_blocks;
  }
  return t;
}

// 32 columns of a row as FP16 pairs, at [row][col ..]; columns up to the pitch
// are written (those past n are zeros).
__device__ __forceinline__ void store_pairs(__half* hi, __half* lo, int64_t row_off, int64_t pitch, int col,
                                            const float (&v)[32]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (col + q * 8 < pitch) {
      Eight<__half> h, l;
#pragma unroll
      for (int j = 0; j < 8; ++j) split_half(v[q * 8 + j], &h.e[j], &l.e[j]);
      *reinterpret_cast<uint4*>(hi + row_off + col + q * 8) = *reinterpret_cast<const uint4*>(&h);
      *reinterpret_cast<uint4*>(lo + row_off + col + q * 8) = *reinterpret_cast<const uint4*>(&l);
    }
  }
}

// The same block mirrored: the 32 lanes' row numbers are the columns.
__device__ __forceinline__ void store_pairs_mirrored(__half* hi, __half* lo, int64_t matrix_off, int64_t pitch, int row,
                                                     int col, int n, const float (&v)[32]) {
  for (int j = 0; j < 32; ++j) {
    if (col + j < n && row < n) {
      __half h, l;
      split_half(v[j], &h, &l);
      const int64_t at = matrix_off + (col + j) * pitch + row;
      hi[at] = h;
      lo[at] = l;
    }
  }
}

template <typename T>
__device__ __forceinline__ void store_result(const NsArgs& a, int64_t at, int cols, const float (&v)[32]) {
  T* p = static_cast<T*>(a.result) + at;
  if (a.result_vec && cols >= 32) {
    constexpr int N = 16 / sizeof(T);
#pragma unroll
    for (int q = 0; q < 32 / N; ++q) {
      uint4 raw = make_uint4(0u, 0u, 0u, 0u);
      T* e = reinterpret_cast<T*>(&raw);
      if (a.update) raw = reinterpret_cast<const uint4*>(p)[q];
#pragma unroll
      for (int j = 0; j < N; ++j)
        e[j] = from_f32<T>(a.update ? fmaf(a.keep, to_f32(e[j]), -a.rate * v[q * N + j]) : v[q * N + j]);
      reinterpret_cast<uint4*>(p)[q] = raw;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < cols) p[j] = from_f32<T>(a.update ? fmaf(a.keep, to_f32(p[j]), -a.rate * v[j]) : v[j]);
  }
}

template <int MODE, bool P_MN, bool Q_MN>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    ns_kernel(const __grid_constant__ CUtensorMap p_hi, const __grid_constant__ CUtensorMap p_lo,
              const __grid_constant__ CUtensorMap q_hi, const __grid_constant__ CUtensorMap q_lo, const NsArgs args) {
  constexpr bool TRI = MODE == GRAM || MODE == POLY;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SMEM_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;   // [2]
  uint64_t* tempty = tfull + 2;       // [2]
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + SMEM_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SMEM_MISC + 4);
  uint32_t* issued_stages = reinterpret_cast<uint32_t*>(smem + SMEM_MISC + 8);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], NUM_EPI_WARPS);
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
  if (warp == 1) {
    tmem_alloc(tmem_holder, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int k_blocks = (args.k + BK - 1) / BK;
  grid_dependency_wait();
  launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (uint32_t tile = blockIdx.x; ok && tile < args.tiles; tile += gridDim.x) {
        const NsTile t = ns_tile<TRI>(tile, args);
        for (int kb = 0; kb < k_blocks; ++kb) {
          ok = mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, args.status, ST_PRODUCER_EMPTY, WAIT_LIMIT_NS);
          if (!ok) break;
          uint8_t* st = smem + stage * STAGE_BYTES;
          mbar_arrive_expect_tx(&full[stage], STAGE_BYTES);
          const int k0 = kb * BK;
          auto load = [&](uint8_t* dst, const CUtensorMap* map, bool mn_major, int rows, int at) {
            if (!mn_major) {
              tma_load_3d(dst, map, &full[stage], k0, at, t.e);
            } else {
              for (int q = 0; q < rows / 64; ++q) tma_load_3d(dst + q * BOX, map, &full[stage], at + 64 * q, k0, t.e);
            }
          };
          load(st, &p_hi, P_MN, BM, t.mb * BM);
          load(st + 2 * P_BYTES, &q_hi, Q_MN, BN, t.nb * BN);
          load(st + P_BYTES, &p_lo, P_MN, BM, t.mb * BM);
          load(st + 2 * P_BYTES + Q_BYTES, &q_lo, Q_MN, BN, t.nb * BN);
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
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      uint32_t it = 0;
      for (uint32_t tile = blockIdx.x; ok && tile < args.tiles; tile += gridDim.x, ++it) {
        const NsTile t = ns_tile<TRI>(tile, args);
        const int n_len = min(BN, (args.n - t.nb * BN + 15) & ~15);
        const uint32_t idesc = idesc_f16_major(false, BM, n_len, P_MN, Q_MN);
        const uint32_t acc = it & 1u;
        ok = mbar_wait_bounded(&tempty[acc], ((it >> 1) & 1u) ^ 1u, abort_flag, args.status, ST_MMA_TMEM_EMPTY,
                               WAIT_LIMIT_NS);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem_base + acc * BN;
        for (int kb = 0; kb < k_blocks; ++kb) {
          ok = mbar_wait_bounded(&full[stage], phase, abort_flag, args.status, ST_MMA_FULL, WAIT_LIMIT_NS);
          if (!ok) break;
          tc_fence_after();
          const uint32_t ph = smem_u32(smem + stage * STAGE_BYTES), pl = ph + P_BYTES;
          const uint32_t qh = ph + 2 * P_BYTES, ql = qh + Q_BYTES;
          const int n_sub = min(BK / UMMA_K, (args.k - kb * BK + UMMA_K - 1) / UMMA_K);
          for (int k = 0; k < n_sub; ++k) {
            auto pd = [&](uint32_t at) {
              return P_MN ? sdesc_mnmajor_sw128(at + k * 2048, BOX, 1024) : sdesc_kmajor_sw128(at + k * UMMA_K * 2);
            };
            auto qd = [&](uint32_t at) {
              return Q_MN ? sdesc_mnmajor_sw128(at + k * 2048, BOX, 1024) : sdesc_kmajor_sw128(at + k * UMMA_K * 2);
            };
            umma_f16(d, pd(pl), qd(qh), idesc, (kb > 0 || k > 0) ? 1u : 0u);
            umma_f16(d, pd(ph), qd(ql), idesc, 1u);
            umma_f16(d, pd(ph), qd(qh), idesc, 1u);
          }
          umma_commit(&empty[stage]);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit(&tfull[acc]);
      }
      umma_commit(drain);
      mbar_wait_bounded(drain, 0, nullptr, args.status, ST_MMA_DRAIN, WAIT_LIMIT_NS);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3;
    const int half = (warp - 2) >> 2;
    uint32_t it = 0;
    for (uint32_t tile = blockIdx.x; tile < args.tiles; tile += gridDim.x, ++it) {
      const NsTile t = ns_tile<TRI>(tile, args);
      const uint32_t acc = it & 1u;
      const bool ok = mbar_wait_bounded(&tfull[acc], (it >> 1) & 1u, abort_flag, args.status, ST_EPI_TMEM_FULL,
                                        WAIT_LIMIT_NS);
      if (!__all_sync(FULL_MASK, ok)) break;
      tc_fence_after();
      const uint32_t t_lane = tmem_base + acc * BN + (static_cast<uint32_t>(quad * 32) << 16);
      const int row = t.mb * BM + quad * 32 + lane;
      const int64_t matrix_off = static_cast<int64_t>(t.e) * args.m * args.pitch;
      const int64_t row_off = matrix_off + static_cast<int64_t>(row) * args.pitch;
      for (int c0 = 32 * half; c0 < BN; c0 += 64) {
        const int col = t.nb * BN + c0;
        if (col >= args.n) break;
        uint32_t raw[32];
        tmem_ld_32x32b_x32(t_lane + static_cast<uint32_t>(c0), raw);
        tmem_ld_wait();
        float v[32];
        if (MODE == GRAM || MODE == POLY) {
          // The mirrored block's own tile is computed only if its columns reach the diagonal.
          const bool mirror = col / BM > t.mb / 2 * 2 + 1;
          if (MODE == GRAM) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(raw[j]) * GRAM_TO_A;
            if (row < args.m) store_pairs(args.out_hi, args.out_lo, row_off, args.pitch, col, v);
            if (mirror) store_pairs_mirrored(args.out_hi, args.out_lo, matrix_off, args.pitch, row, col, args.n, v);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              v[j] = fmaf(__uint_as_float(raw[j]), GRAM_TO_C,
                          row == col + j ? C_DIAG : 0.0f);
            if (row < args.m) store_pairs(args.out2_hi, args.out2_lo, row_off, args.pitch, col, v);
            if (mirror) store_pairs_mirrored(args.out2_hi, args.out2_lo, matrix_off, args.pitch, row, col, args.n, v);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              v[j] = fmaf(__uint_as_float(raw[j]), POLY_TO_B,
                          row == col + j ? B_DIAG : 0.0f);
            if (row < args.m) store_pairs(args.out_hi, args.out_lo, row_off, args.pitch, col, v);
            if (mirror) store_pairs_mirrored(args.out_hi, args.out_lo, matrix_off, args.pitch, row, col, args.n, v);
          }
        } else if (MODE == APPLY) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(raw[j]) * APPLY_TO_X;
          if (row < args.m) store_pairs(args.out_hi, args.out_lo, row_off, args.pitch, col, v);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(raw[j]) * APPLY_TO_RESULT;
          if (row < args.m) {
            const int64_t at = (static_cast<int64_t>(t.e) * args.m + row) * args.n + col;
            const int cols = args.n - col;
            if (args.result_dtype == MOE_F32) store_result<float>(args, at, cols, v);
            else if (args.result_dtype == MOE_F16) store_result<__half>(args, at, cols, v);
            else store_result<__nv_bfloat16>(args, at, cols, v);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag != 0) {
    // A role gave up: the copies that nobody waited for land before the block exits.
    if (threadIdx.x == 0)
      drain_ring(*issued_stages, STAGES, [&](uint32_t slot, uint32_t parity) {
        mbar_wait_bounded(&full[slot], parity, nullptr, args.status, ST_PRODUCER_DRAIN, WAIT_LIMIT_NS);
      });
    __syncwarp();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
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

// A pair [E, rows, pitch] of the workspace.
struct Pair {
  __half* hi;
  __half* lo;
  int64_t rows, cols, pitch;
};

struct Layout {
  size_t partial, x0, x1, a, c, b, total;
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
  l.partial = take(align_up(static_cast<size_t>(E * chunk_count(r * c)) * sizeof(double), 256));
  l.x0 = take(2 * x);
  l.x1 = take(2 * x);
  l.a = take(2 * g);
  l.c = take(2 * g);
  l.b = take(2 * g);
  l.total = at;
  return l;
}

template <int MODE, bool P_MN, bool Q_MN>
cudaError_t launch_product(int64_t E, const Pair& p, const Pair& q, NsArgs args, int num_sms, cudaStream_t s,
                           const char** why) {
  CUtensorMap m[4];
  if (!enc(&m[0], p.hi, E, p.rows, p.cols, p.pitch, P_MN ? 64 : BM) ||
      !enc(&m[1], p.lo, E, p.rows, p.cols, p.pitch, P_MN ? 64 : BM) ||
      !enc(&m[2], q.hi, E, q.rows, q.cols, q.pitch, Q_MN ? 64 : BN) ||
      !enc(&m[3], q.lo, E, q.rows, q.cols, q.pitch, Q_MN ? 64 : BN)) {
    *why = "cuTensorMapEncodeTiled rejected an operand";
    return cudaErrorInvalidValue;
  }
  args.m_blocks = (args.m + BM - 1) / BM;
  args.n_blocks = (args.n + BN - 1) / BN;
  int64_t per = 0;
  if (MODE == GRAM || MODE == POLY)
    for (int mb = 0; mb < args.m_blocks; ++mb) per += args.n_blocks - mb / 2;
  else
    per = static_cast<int64_t>(args.m_blocks) * args.n_blocks;
  args.tiles_per_matrix = static_cast<uint32_t>(per);
  args.tiles = static_cast<uint32_t>(E * per);
  auto kern = ns_kernel<MODE, P_MN, Q_MN>;
  const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (err != cudaSuccess) return err;
  const int grid = static_cast<int>(std::min<int64_t>(args.tiles, num_sms));
  return launch_dependent(kern, dim3(grid), dim3(NUM_THREADS), SMEM_BYTES, s, m[0], m[1], m[2], m[3], args);
}

template <typename T>
cudaError_t launch_pre(const PreArgs& a, int64_t E, cudaStream_t s) {
  cudaError_t err = launch_dependent(squares_kernel<T>, dim3(a.chunks, static_cast<unsigned>(E)), dim3(PRE_THREADS), 0,
                                     s, a);
  if (err != cudaSuccess) return err;
  const int64_t groups = a.pitch / 8 * a.r;
  const int64_t blocks = std::min<int64_t>((groups + PRE_THREADS - 1) / PRE_THREADS, 2 * MAX_CHUNKS);
  return launch_dependent(first_x_kernel<T>, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(E)),
                          dim3(PRE_THREADS), 0, s, a);
}

}  // namespace

size_t newton_schulz_scratch_bytes(int64_t E, int64_t r, int64_t c) { return layout(E, r, c).total; }

int64_t newton_schulz_tiles(int64_t E, int64_t r, int64_t c) {
  const int64_t most = std::max(r, c);
  return E * ((most + BM - 1) / BM) * ((most + BM - 1) / BM);
}

cudaError_t launch_newton_schulz(const NewtonSchulz& o, void* scratch, int num_sms, cudaStream_t stream,
                                 const char** why) {
  const int64_t E = o.E, r = o.rows, c = o.cols, s = std::min(r, c);
  if (E == 0 || r == 0 || c == 0) return cudaSuccess;
  uint32_t* status = nullptr;
  cudaError_t err = device_status_ptr(&status);
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
  const Pair a = pair(l.a, s, s, l.s_pitch), cc = pair(l.c, s, s, l.s_pitch), b = pair(l.b, s, s, l.s_pitch);

  PreArgs pre{};
  pre.g = o.grad;
  pre.m = o.momentum;
  pre.partial = reinterpret_cast<double*>(base + l.partial);
  pre.hi = x.hi;
  pre.lo = x.lo;
  pre.n = r * c;
  pre.chunk = chunk_elems(pre.n);
  pre.pitch = l.x_pitch;
  pre.r = static_cast<int>(r);
  pre.c = static_cast<int>(c);
  pre.chunks = static_cast<int>(chunk_count(pre.n));
  pre.nesterov = o.nesterov;
  pre.vec = pre.n % 8 == 0 && reinterpret_cast<uintptr_t>(o.grad) % 16 == 0 &&
            reinterpret_cast<uintptr_t>(o.momentum) % 16 == 0;
  pre.mu = o.momentum_decay;
  pre.eps = o.eps;
  err = o.grad_dtype == MOE_F32   ? launch_pre<float>(pre, E, stream)
        : o.grad_dtype == MOE_F16 ? launch_pre<__half>(pre, E, stream)
                                  : launch_pre<__nv_bfloat16>(pre, E, stream);
  if (err != cudaSuccess) return err;

  const bool tall = r > c;
  NsArgs sq{};
  sq.status = status;
  sq.m = sq.n = static_cast<int>(s);
  sq.pitch = l.s_pitch;
  for (int step = 0; step < o.steps; ++step) {
    NsArgs g = sq;
    g.k = static_cast<int>(tall ? r : c);
    g.out_hi = a.hi;
    g.out_lo = a.lo;
    g.out2_hi = cc.hi;
    g.out2_lo = cc.lo;
    err = tall ? launch_product<GRAM, true, true>(E, x, x, g, num_sms, stream, why)
               : launch_product<GRAM, false, false>(E, x, x, g, num_sms, stream, why);
    if (err != cudaSuccess) return err;
    NsArgs p = sq;
    p.k = static_cast<int>(s);
    p.out_hi = b.hi;
    p.out_lo = b.lo;
    err = launch_product<POLY, false, false>(E, a, cc, p, num_sms, stream, why);
    if (err != cudaSuccess) return err;
    NsArgs f{};
    f.status = status;
    f.m = static_cast<int>(r);
    f.n = static_cast<int>(c);
    f.k = static_cast<int>(s);
    f.pitch = l.x_pitch;
    f.out_hi = next.hi;
    f.out_lo = next.lo;
    if (step + 1 < o.steps) {
      err = tall ? launch_product<APPLY, false, false>(E, x, b, f, num_sms, stream, why)
                 : launch_product<APPLY, false, true>(E, b, x, f, num_sms, stream, why);
    } else {
      f.result = o.result;
      f.result_dtype = o.result_dtype;
      f.result_vec = (c * static_cast<int64_t>(dtype_size(o.result_dtype))) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(o.result) % 16 == 0;
      f.update = o.update;
      f.keep = o.keep;
      f.rate = o.rate;
      err = tall ? launch_product<FINAL, false, false>(E, x, b, f, num_sms, stream, why)
                 : launch_product<FINAL, false, true>(E, b, x, f, num_sms, stream, why);
    }
    if (err != cudaSuccess) return err;
    std::swap(x, next);
  }
  return cudaSuccess;
}

}  // namespace moe
