// The norm before a block and the join after it, forward and backward.
//
//   norm(v; w) = v * r(v) * w,  r(v) = 1 / sqrt(mean(v^2) + eps)
//   join:  out = round(alpha x + beta g * norm(f; w1)),  y = norm(out; w2)
//
// f is the block's output, or (combine) the routing-weighted sum of a token's
// expert rows, kept in FP32; the norm of f, the gate g and the next block's
// norm of out are each optional, and the norm before a block is the join
// without f. y is the norm of out as it is stored, so that the backward, which
// has the stored out, differentiates the function that ran.
//
// Backward, from dout and dy (per row, G = w1 * g):
//   S2 = sum w2 dy out,  dO = dout + r2 (w2 dy - out r2^2 S2 / H)
//   dx = alpha dO,  dw2 = sum over rows of dy out r2
//   Q  = sum dO G f,  df = beta r1 (G dO - f r1^2 Q / H)
//   dw1 = sum over rows of beta g dO f r1,  dg = beta dO f r1 w1, summed over
//   what the gate is shared by.
// dO depends on row sums, but Q expands into sums of products of the inputs,
//   Q = sum dout G f + r2 sum w2 dy G f - r2^3 (S2 / H) sum out G f,
// so that one reduction of six sums per row gives everything and each input is
// read once. A token's gate is left out of the sums: its own gradient is
// beta r1 Q then.
//
// All sums are FP32: a thread's 8 columns in order, then a fixed tree over the
// row's threads; a column's sum over the rows is a block's rows in order, then
// the blocks in order, so results do not depend on timing.
//
// Layout: a thread owns 8 columns of a row (16 or 32 bytes), a row up to 4096
// columns one block, more a cluster of up to 8 blocks that exchange their sums
// through distributed shared memory. Short rows share a block.
#include <cooperative_groups.h>

#include <algorithm>
#include <initializer_list>

#include "moe_common.cuh"
#include "moe_internal.h"
#include "ring_drain.h"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int COLS = 8;               // columns of a thread
constexpr int MAX_TPR = 512;          // threads of a row in one block
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_WARPS = MAX_TPR / 32;
constexpr int BLOCK = 256;            // threads of a block that short rows share

static_assert(COLS * MAX_TPR * MAX_CLUSTER == BLOCK_NORM_MAX_H, "widest row");

struct RowShape {
  int tpr;       // threads per row and block, a multiple of 32
  int rows;      // rows of a block side by side
  int cluster;   // blocks of a row
};

RowShape row_shape(int64_t H) {
  RowShape s;
  s.cluster = 1;
  while (static_cast<int64_t>(s.cluster) * MAX_TPR * COLS < H) s.cluster *= 2;
  const int64_t per = (H + s.cluster - 1) / s.cluster;
  s.tpr = static_cast<int>((per + COLS * 32 - 1) / (COLS * 32)) * 32;
  s.rows = s.tpr >= BLOCK ? 1 : BLOCK / s.tpr;
  return s;
}

// ---------------------------------------------------------------- a thread's 8 columns

// Its columns: 8 neighbours (VEC: rows and pointers are 16-byte aligned and H
// is a multiple of 8), or every tpr-th one.
template <bool VEC>
struct Cols {
  int first, step, H;
  __device__ Cols(int tid, int tpr, int rank, int H_) : H(H_) {
    first = rank * tpr * COLS + (VEC ? tid * COLS : tid);
    step = VEC ? 1 : tpr;
  }
  __device__ bool any() const { return first < H; }
  __device__ int col(int j) const { return first + j * step; }
};

template <typename T>
struct alignas(16) Eight {
  T e[COLS];
};

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, const Cols<VEC>& c, Eight<T>& v) {
  if (VEC) {
    if (c.any()) {
      const uint4* p = reinterpret_cast<const uint4*>(row + c.first);
      uint4* q = reinterpret_cast<uint4*>(&v);
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(v) / 16); ++i) q[i] = p[i];
      return;
    }
#pragma unroll
    for (int j = 0; j < COLS; ++j) v.e[j] = from_f32<T>(0.0f);
  } else {
#pragma unroll
    for (int j = 0; j < COLS; ++j) v.e[j] = c.col(j) < c.H ? row[c.col(j)] : from_f32<T>(0.0f);
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* row, const Cols<VEC>& c, const Eight<T>& v) {
  if (VEC) {
    if (!c.any()) return;
    uint4* p = reinterpret_cast<uint4*>(row + c.first);
    const uint4* q = reinterpret_cast<const uint4*>(&v);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(v) / 16); ++i) p[i] = q[i];
  } else {
#pragma unroll
    for (int j = 0; j < COLS; ++j)
      if (c.col(j) < c.H) row[c.col(j)] = v.e[j];
  }
}

// To FP32 and back (rounded to nearest even), two 16-bit values at a time.
__device__ __forceinline__ void unpack8(const Eight<float>& v, float (&f)[COLS]) {
#pragma unroll
  for (int j = 0; j < COLS; ++j) f[j] = v.e[j];
}
__device__ __forceinline__ void unpack8(const Eight<__half>& v, float (&f)[COLS]) {
#pragma unroll
  for (int j = 0; j < COLS / 2; ++j) {
    const float2 p = __half22float2(reinterpret_cast<const __half2*>(&v)[j]);
    f[2 * j] = p.x;
    f[2 * j + 1] = p.y;
  }
}
__device__ __forceinline__ void unpack8(const Eight<__nv_bfloat16>& v, float (&f)[COLS]) {
#pragma unroll
  for (int j = 0; j < COLS / 2; ++j) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(&v)[j];
    f[2 * j] = __uint_as_float(w << 16);
    f[2 * j + 1] = __uint_as_float(w & 0xFFFF0000u);
  }
}
template <typename T>
__device__ __forceinline__ void pack8(const float (&f)[COLS], Eight<T>& v) {
#pragma unroll
  for (int j = 0; j < COLS / 2; ++j) reinterpret_cast<uint32_t*>(&v)[j] = pack2<T>(f[2 * j], f[2 * j + 1]);
}
template <>
__device__ __forceinline__ void pack8<float>(const float (&f)[COLS], Eight<float>& v) {
#pragma unroll
  for (int j = 0; j < COLS; ++j) v.e[j] = f[j];
}

// A vector over the columns, in T or FP32; 1 where there is none.
template <typename T, bool VEC>
__device__ __forceinline__ void load_vector(const void* p, bool f32, const Cols<VEC>& c, float (&w)[COLS]) {
  if (p == nullptr) {
#pragma unroll
    for (int j = 0; j < COLS; ++j) w[j] = 1.0f;
  } else if (f32) {
    Eight<float> v;
    load8<float, VEC>(static_cast<const float*>(p), c, v);
#pragma unroll
    for (int j = 0; j < COLS; ++j) w[j] = v.e[j];
  } else {
    Eight<T> v;
    load8<T, VEC>(static_cast<const T*>(p), c, v);
#pragma unroll
    for (int j = 0; j < COLS; ++j) w[j] = to_f32(v.e[j]);
  }
}

// ---------------------------------------------------------------- sums over a row

// N <= 8 sums over a row, for every thread of it. One barrier per call: the
// two halves of `sm` are used in turn, and a half is written again only after
// the barrier of the call between, which every reader of the half has passed.
// In a warp the sums are added by exchanging: with 8 sums a lane gives half of
// its sums away three times and ends with one of them over 8 lanes, 9 shuffles
// for the warp's 8 sums in place of 40.
template <int N>
struct RowSums {
  static constexpr int PAD = N == 1 ? 1 : 8;
  float v[2][PAD][MAX_CLUSTER * MAX_WARPS];   // [half][sum][block of the cluster * warps + warp]
};

__device__ __forceinline__ float lanes_sum(float v, int from) {
  for (int off = from; off > 0; off >>= 1) v += __shfl_xor_sync(FULL_MASK, v, off);
  return v;
}

// One value per lane: the warp's sum number lane / 4 (of 8).
__device__ __forceinline__ float exchange_sums(const float (&s)[8]) {
  const int lane = threadIdx.x & 31;
  float a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float keep = lane & 16 ? s[i + 4] : s[i], give = lane & 16 ? s[i] : s[i + 4];
    a[i] = keep + __shfl_xor_sync(FULL_MASK, give, 16);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float keep = lane & 8 ? a[i + 2] : a[i], give = lane & 8 ? a[i] : a[i + 2];
    b[i] = keep + __shfl_xor_sync(FULL_MASK, give, 8);
  }
  const float keep = lane & 4 ? b[1] : b[0], give = lane & 4 ? b[0] : b[1];
  float c = keep + __shfl_xor_sync(FULL_MASK, give, 4);
  c += __shfl_xor_sync(FULL_MASK, c, 2);
  return c + __shfl_xor_sync(FULL_MASK, c, 1);
}

template <int N>
__device__ __forceinline__ void row_sum(float (&s)[N], RowSums<N>* sm, int& half, int tpr, int cluster, int rank) {
  static_assert(N == 1 || N == 6, "one sum, or eight slots for six");
  const int lane = threadIdx.x & 31, warps = tpr >> 5;
  float mine;
  if (N == 1) {
    mine = lanes_sum(s[0], 16);
    s[0] = mine;
  } else {
    const float e[8] = {s[0], s[1 % N], s[2 % N], s[3 % N], s[4 % N], s[5 % N], 0.0f, 0.0f};
    mine = exchange_sums(e);
  }
  if (tpr > 32 || cluster > 1) {
    const int slot0 = static_cast<int>(threadIdx.y) * warps;   // rows side by side have slots of their own
    const int which = N == 1 ? 0 : lane >> 2;
    const int slot = slot0 + rank * warps + static_cast<int>(threadIdx.x >> 5);
    if (cluster == 1) {
      if (N == 1 ? lane == 0 : (lane & 3) == 0) sm->v[half][which][slot] = mine;
      __syncthreads();
    } else {
      cg::cluster_group cl = cg::this_cluster();
      // N == 1: lane i writes to block i; else the four lanes of a sum share the blocks.
      for (int to = N == 1 ? lane : lane & 3; to < cluster; to += N == 1 ? 32 : 4)
        *cl.map_shared_rank(&sm->v[half][which][slot], to) = mine;
      cl.sync();
    }
    mine = 0.0f;
    for (int w = N == 1 ? lane : lane & 3; w < cluster * warps; w += N == 1 ? 32 : 4) mine += sm->v[half][which][slot0 + w];
    half ^= 1;
    if (N == 1) {
      s[0] = lanes_sum(mine, 16);
      return;
    }
    mine = lanes_sum(mine, 2);
  }
  if (N > 1)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = __shfl_sync(FULL_MASK, mine, 4 * i);
}

__device__ __forceinline__ float weight_at(const void* p, int dtype, int64_t i) {
  if (dtype == MOE_F32) return static_cast<const float*>(p)[i];
  if (dtype == MOE_F16) return to_f32(static_cast<const __half*>(p)[i]);
  return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
}
template <typename T>
__device__ __forceinline__ float token_gate(const void* p, bool f32, int64_t t) {
  return f32 ? static_cast<const float*>(p)[t] : to_f32(static_cast<const T*>(p)[t]);
}

// ---------------------------------------------------------------- rows ahead of their use

// A ring of rounds in shared memory: one thread copies what a round reads, as
// whole rows by bulk copies (16-byte aligned: VEC rows), several rounds before
// its turn. An SM needs some 70 KB of loads in flight for its share of HBM's
// rate; in registers one round ahead is all there is room for (the backward of
// 8192 x 4096 BF16 rows ran at 1.9 TB/s that way).
constexpr int MAX_STAGES = 8;
constexpr uint64_t WAIT_LIMIT_NS = 1000000000ull;
constexpr uint32_t ST_ROWS = 0x51, ST_ROWS_DRAIN = 0x52;

struct Ring {
  uint64_t full[MAX_STAGES];
  int abort_flag;
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void ring_init(Ring& ring, int stages) {
  if (threadIdx.x == 0 && threadIdx.y == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(&ring.full[i], 1);
    ring.abort_flag = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
}

// A place in the ring and the parity of its barrier's phase, round after round.
struct Turn {
  int slot;
  uint32_t parity;
  __device__ void next(int stages) {
    if (++slot == stages) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

// A round's rows are there; a wait that runs out leaves its results undefined.
// Every thread of the block waits here: the clock is read after many tries only.
__device__ __forceinline__ void ring_wait(Ring& ring, const Turn& turn, uint32_t* status) {
  uint64_t* bar = &ring.full[turn.slot];
  for (int tries = 0; tries < 256; ++tries)
    if (mbar_try_wait(bar, turn.parity)) return;
  mbar_wait_bounded(bar, turn.parity, &ring.abort_flag, status, ST_ROWS, WAIT_LIMIT_NS);
}

// Before the block exits: the copies that nobody waited for (after a give-up).
__device__ __forceinline__ void ring_end(Ring& ring, uint32_t issued, int stages, uint32_t* status) {
  __syncthreads();
  if (ring.abort_flag != 0 && threadIdx.x == 0 && threadIdx.y == 0)
    drain_ring(issued, stages, [&](uint32_t slot, uint32_t parity) {
      mbar_wait_bounded(&ring.full[slot], parity, nullptr, status, ST_ROWS_DRAIN, WAIT_LIMIT_NS);
    });
  __syncthreads();
}

// This thread's columns of a row in a stage.
template <typename T>
__device__ __forceinline__ void stage8(const uint8_t* mine, bool any, Eight<T>& v) {
  if (any) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(v) / 16); ++i)
      reinterpret_cast<uint4*>(&v)[i] = reinterpret_cast<const uint4*>(mine)[i];
  } else {
#pragma unroll
    for (int j = 0; j < COLS; ++j) v.e[j] = from_f32<T>(0.0f);
  }
}

// ---------------------------------------------------------------- forward

// BRANCH: 0 none (the norm alone), 1 rows of f, 2 the combine of expert rows.
// ELEMENT: a gate for every element.
//
// Bound by HBM: x and f in (combine: top_k rows), out and y out. BULK: rounds
// come through the ring; else (unaligned rows, calls of one round a block, many
// slots) they are loaded when their turn comes.

// Threads that an SM holds: 1024 of 64 registers where that is enough.
constexpr int join_threads(size_t size, bool vec, int branch, bool element) {
  return size == 2 && vec && branch < 2 && !element ? 1024 : 512;
}
template <typename T, bool VEC, bool BULK, int BRANCH, bool ELEMENT>
__global__ void __launch_bounds__(MAX_TPR, join_threads(sizeof(T), VEC, BRANCH, ELEMENT) / MAX_TPR)
    join_kernel(const JoinArgs a, int cluster, int stages) {
  __shared__ RowSums<1> sums;
  __shared__ Ring ring;
  extern __shared__ __align__(128) uint8_t stage_smem[];
  const int tpr = blockDim.x;
  const int rank = cluster > 1 ? static_cast<int>(blockIdx.x) % cluster : 0;
  const int64_t unit = blockIdx.x / cluster, units = gridDim.x / cluster;
  const int64_t step = units * blockDim.y;
  const Cols<VEC> c(threadIdx.x, tpr, rank, a.H);
  const int lane = threadIdx.x & 31;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  const bool post = BRANCH != 0 && a.norm_weight != nullptr;
  const bool next = BRANCH == 0 || a.next_weight != nullptr;
  int half = 0;
  if (BULK) ring_init(ring, stages);
  if (cluster > 1) cg::this_cluster().sync();   // every block runs before another one writes to its sums
  grid_dependency_wait();
  launch_dependents();

  // The ring: a stage holds x, then f or the expert rows, then the gates, each
  // of this block's columns.
  const int cols = min(tpr * COLS, a.H - rank * tpr * COLS);
  const size_t row_bytes = static_cast<size_t>(cols) * sizeof(T), block_bytes = row_bytes * blockDim.y;
  const size_t stage_bytes = block_bytes * (1 + (BRANCH == 2 ? a.top_k : BRANCH) + (ELEMENT ? 1 : 0));
  uint32_t issued = 0;
  // Combine: lane j's expert row (and weight) of the round to be issued next
  // and of the one at work.
  auto slot_of = [&](int64_t t0) {
    const int64_t t = min(t0 + threadIdx.y, a.T - 1);
    return lane < a.top_k && t0 < a.T ? a.inv[t * a.top_k + lane] : 0xFFFFFFFFu;
  };
  uint32_t ahead = BRANCH == 2 && BULK ? slot_of(unit * blockDim.y) : 0;
  int64_t issue_t0 = unit * blockDim.y;
  Turn fill{0, 0u};
  auto issue = [&]() {   // by the first warp of the block
    const int64_t t0 = issue_t0;
    if (t0 >= a.T) return;
    const int n = static_cast<int>(min(static_cast<int64_t>(blockDim.y), a.T - t0));
    uint8_t* dst = stage_smem + fill.slot * stage_bytes;
    uint64_t* bar = &ring.full[fill.slot];
    const int64_t at = t0 * a.H + rank * tpr * COLS;
    const uint32_t bytes = static_cast<uint32_t>(row_bytes * n);
    const bool good = BRANCH == 2 && ahead < a.rows;
    if (BRANCH == 2) {
      const uint32_t rows = __popc(__ballot_sync(FULL_MASK, good));
      if (lane == 0) mbar_arrive_expect_tx(bar, bytes * ((ELEMENT ? 2 : 1) + rows));
      __syncwarp();
      if (good)
        bulk_load(dst + (1 + lane) * row_bytes,
                  static_cast<const T*>(a.f) + static_cast<int64_t>(ahead) * a.H + rank * tpr * COLS, bytes, bar);
    }
    if (lane == 0) {
      if (BRANCH != 2) mbar_arrive_expect_tx(bar, bytes * (1 + BRANCH + (ELEMENT ? 1 : 0)));
      bulk_load(dst, static_cast<const T*>(a.x) + at, bytes, bar);
      if (BRANCH == 1) bulk_load(dst + block_bytes, static_cast<const T*>(a.f) + at, bytes, bar);
      if (ELEMENT) bulk_load(dst + stage_bytes - block_bytes, static_cast<const T*>(a.gate) + at, bytes, bar);
    }
    ++issued;
    fill.next(stages);
    issue_t0 += step;
    if (BRANCH == 2) ahead = slot_of(issue_t0);
  };
  const bool issuer = BULK && threadIdx.x < 32 && threadIdx.y == 0;
  if (issuer)
    for (int i = 0; i < stages; ++i) issue();

  float w1[COLS], w2[COLS];
  if (BRANCH != 0) {
    load_vector<T, VEC>(a.norm_weight, a.vec_f32, c, w1);
    if (a.gate_kind == MOE_GATE_CHANNEL) {
      float g[COLS];
      load_vector<T, VEC>(a.gate, a.vec_f32, c, g);
#pragma unroll
      for (int j = 0; j < COLS; ++j) w1[j] *= g[j];
    }
  }
  load_vector<T, VEC>(a.next_weight, a.vec_f32, c, w2);

  // Every thread of a block takes part in every round (the barriers), with a
  // row past the end as a row that is not stored.
  Turn turn{0, 0u};
  const uint8_t* mine = stage_smem + (static_cast<size_t>(threadIdx.y) * cols + threadIdx.x * COLS) * sizeof(T);
  const bool row_barrier = tpr > 32 || cluster > 1;
  for (int64_t t0 = unit * blockDim.y; t0 < a.T; t0 += step) {
    const bool live = t0 + threadIdx.y < a.T;
    const int64_t t = live ? t0 + threadIdx.y : a.T - 1;
    const int64_t at = t * a.H;
    Eight<T> raw, gv;
    float x[COLS], f[COLS];
    float g = a.beta;
    if (BRANCH != 0 && a.gate_kind == MOE_GATE_TOKEN) g *= token_gate<T>(a.gate, a.vec_f32, t);
    uint32_t slot = 0;
    float weight = 0.0f;
    if (BRANCH == 2 && lane < a.top_k) {
      slot = a.inv[t * a.top_k + lane];
      weight = weight_at(a.weights, a.weights_dtype, t * a.top_k + lane);
    }
    const uint8_t* stage = mine + turn.slot * stage_bytes;
    if (BULK) {
      ring_wait(ring, turn, a.status);
      turn.next(stages);
      stage8<T>(stage, c.any(), raw);
      if (ELEMENT) stage8<T>(stage + stage_bytes - block_bytes, c.any(), gv);
    } else {
      load8<T, VEC>(static_cast<const T*>(a.x) + at, c, raw);
      if (ELEMENT) load8<T, VEC>(static_cast<const T*>(a.gate) + at, c, gv);
    }
    unpack8(raw, x);
    if (BRANCH == 1) {
      if (BULK) stage8<T>(stage + block_bytes, c.any(), raw);
      else load8<T, VEC>(static_cast<const T*>(a.f) + at, c, raw);
      unpack8(raw, f);
    }
    if (BRANCH == 2) {
      // Slot order, as moe_combine; a bad row number makes the token NaN.
#pragma unroll
      for (int j = 0; j < COLS; ++j) f[j] = 0.0f;
      bool bad = false;
      constexpr int G = 4;   // rows whose loads are in flight together
      for (int first = 0; first < a.top_k; first += 32) {
        if (first > 0 && first + lane < a.top_k) {
          slot = a.inv[t * a.top_k + first + lane];
          weight = weight_at(a.weights, a.weights_dtype, t * a.top_k + first + lane);
        }
        const int here = min(a.top_k - first, 32);
        for (int k0 = 0; k0 < here; k0 += G) {
          Eight<T> v[G];
          float w[G];
#pragma unroll
          for (int i = 0; i < G; ++i) {
            uint32_t row = __shfl_sync(FULL_MASK, slot, (k0 + i) & 31);
            w[i] = __shfl_sync(FULL_MASK, weight, (k0 + i) & 31);
            if (k0 + i < here) {
              if (row >= a.rows) {
                bad = true;
                row = 0;
              }
              if (BULK) stage8<T>(stage + (1 + k0 + i) * row_bytes, c.any(), v[i]);
              else load8<T, VEC>(static_cast<const T*>(a.f) + static_cast<int64_t>(row) * a.H, c, v[i]);
            }
          }
#pragma unroll
          for (int i = 0; i < G; ++i)
            if (k0 + i < here) {
              float y[COLS];
              unpack8(v[i], y);
#pragma unroll
              for (int j = 0; j < COLS; ++j) f[j] = fmaf(w[i], y[j], f[j]);
            }
        }
      }
      if (bad)
#pragma unroll
        for (int j = 0; j < COLS; ++j) f[j] = __int_as_float(0x7FC00000);
    }
    // The first of the round's barriers after which the stage may be copied over.
    bool freed = !BULK;
    auto free_stage = [&](bool barrier) {
      if (freed) return;
      freed = true;
      if (!barrier) __syncthreads();
      if (issuer) issue();
    };
    if (BRANCH != 0) {
      if (post) {
        float s[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < COLS; ++j)
          if (VEC || c.col(j) < c.H) s[0] = fmaf(f[j], f[j], s[0]);
        if (VEC && !c.any()) s[0] = 0.0f;   // a thread past the row may hold a token's NaN
        row_sum<1>(s, &sums, half, tpr, cluster, rank);
        free_stage(row_barrier);
        g *= rsqrtf(fmaf(s[0], inv_h, a.eps));
      }
      float gate[COLS];
      if (ELEMENT) unpack8(gv, gate);
#pragma unroll
      for (int j = 0; j < COLS; ++j) x[j] = fmaf(a.alpha, x[j], f[j] * g * w1[j] * (ELEMENT ? gate[j] : 1.0f));
      pack8<T>(x, raw);
      if (live) store8<T, VEC>(static_cast<T*>(a.out) + at, c, raw);
      if (next) unpack8(raw, x);
    }
    if (next) {
      float s[1] = {0.0f};
#pragma unroll
      for (int j = 0; j < COLS; ++j)
        if (VEC || c.col(j) < c.H) s[0] = fmaf(x[j], x[j], s[0]);
      if (VEC && !c.any()) s[0] = 0.0f;
      row_sum<1>(s, &sums, half, tpr, cluster, rank);
      free_stage(row_barrier);
      const float r = rsqrtf(fmaf(s[0], inv_h, a.eps));
#pragma unroll
      for (int j = 0; j < COLS; ++j) x[j] = x[j] * r * w2[j];
      pack8<T>(x, raw);
      if (live) store8<T, VEC>(static_cast<T*>(a.y) + at, c, raw);
    }
    free_stage(false);
  }
  if (BULK) ring_end(ring, issued, stages, a.status);
}

// ---------------------------------------------------------------- backward

// HAS_F: the join's branch is there; NEXT: the norm of out is there. Column
// sums go to partial[unit][column array][H], arrays in the order dw1, dgate
// (a channel gate's), dw2, those that are asked for. A channel's gate and w1
// multiply the same sum, S = sum over rows of beta r1 dO f (times the other
// gates): dw1 = gate S, dgate = w1 S.
//
// Bound by HBM (join: dout, dy, out, f in, dx, df out). BULK as in the forward.
template <typename T, bool VEC, bool BULK, bool HAS_F, bool NEXT, bool ELEMENT>
__global__ void __launch_bounds__(MAX_TPR) join_backward_kernel(const JoinBackwardArgs a, int cluster, int stages) {
  __shared__ RowSums<6> sums;
  __shared__ Ring ring;
  extern __shared__ __align__(128) uint8_t stage_smem[];   // the ring; in the end [rows of the block - 1][tpr * COLS] sums
  float* fold = reinterpret_cast<float*>(stage_smem);
  const int tpr = blockDim.x;
  const int rank = cluster > 1 ? static_cast<int>(blockIdx.x) % cluster : 0;
  const int64_t unit = blockIdx.x / cluster, units = gridDim.x / cluster;
  const int64_t step = units * blockDim.y;
  const Cols<VEC> c(threadIdx.x, tpr, rank, a.H);
  const float inv_h = 1.0f / static_cast<float>(a.H);
  const bool post = HAS_F && a.norm_weight != nullptr;
  const bool token = HAS_F && a.gate_kind == MOE_GATE_TOKEN;
  const bool channel = HAS_F && a.gate_kind == MOE_GATE_CHANNEL;
  const bool has_d = a.dout != nullptr;
  int half = 0;
  if (BULK) ring_init(ring, stages);
  if (cluster > 1) cg::this_cluster().sync();   // every block runs before another one writes to its sums
  grid_dependency_wait();
  launch_dependents();

  // A stage: dout, f, out and dy, the gates, of this block's columns.
  const int cols = min(tpr * COLS, a.H - rank * tpr * COLS);
  const size_t block_bytes = static_cast<size_t>(cols) * sizeof(T) * blockDim.y;
  constexpr int ARRAYS = 1 + (HAS_F ? 1 : 0) + (NEXT ? 2 : 0) + (ELEMENT ? 1 : 0);
  constexpr int AT_F = 1, AT_O = 1 + (HAS_F ? 1 : 0), AT_Y = AT_O + 1, AT_G = ARRAYS - 1;
  const size_t stage_bytes = block_bytes * ARRAYS;
  uint32_t issued = 0;
  int64_t issue_t0 = unit * blockDim.y;
  Turn fill{0, 0u};
  auto issue = [&]() {
    const int64_t t0 = issue_t0;
    if (t0 >= a.T) return;
    const int n = static_cast<int>(min(static_cast<int64_t>(blockDim.y), a.T - t0));
    uint8_t* dst = stage_smem + fill.slot * stage_bytes;
    uint64_t* bar = &ring.full[fill.slot];
    const int64_t at = t0 * a.H + rank * tpr * COLS;
    const uint32_t bytes = static_cast<uint32_t>(static_cast<size_t>(cols) * sizeof(T) * n);
    mbar_arrive_expect_tx(bar, bytes * (ARRAYS - (has_d ? 0 : 1)));
    if (has_d) bulk_load(dst, static_cast<const T*>(a.dout) + at, bytes, bar);
    if (HAS_F) bulk_load(dst + AT_F * block_bytes, static_cast<const T*>(a.f) + at, bytes, bar);
    if (NEXT) {
      bulk_load(dst + AT_O * block_bytes, static_cast<const T*>(a.joined) + at, bytes, bar);
      bulk_load(dst + AT_Y * block_bytes, static_cast<const T*>(a.dnormed) + at, bytes, bar);
    }
    if (ELEMENT) bulk_load(dst + AT_G * block_bytes, static_cast<const T*>(a.gate) + at, bytes, bar);
    ++issued;
    fill.next(stages);
    issue_t0 += step;
  };
  const bool issuer = BULK && threadIdx.x == 0 && threadIdx.y == 0;
  if (issuer)
    for (int i = 0; i < stages; ++i) issue();

  float w1[COLS], w2[COLS];   // w1: with a channel's gate
  float s1[COLS], s2[COLS];   // column sums S and dw2
#pragma unroll
  for (int j = 0; j < COLS; ++j) s1[j] = s2[j] = 0.0f;
  if (HAS_F) {
    load_vector<T, VEC>(a.norm_weight, a.vec_f32, c, w1);
    if (channel) {
      float g[COLS];
      load_vector<T, VEC>(a.gate, a.vec_f32, c, g);
#pragma unroll
      for (int j = 0; j < COLS; ++j) w1[j] *= g[j];
    }
  }
  if (NEXT) load_vector<T, VEC>(a.next_weight, a.vec_f32, c, w2);

  Turn turn{0, 0u};
  const uint8_t* mine = stage_smem + (static_cast<size_t>(threadIdx.y) * cols + threadIdx.x * COLS) * sizeof(T);
  for (int64_t t0 = unit * blockDim.y; t0 < a.T; t0 += step) {
    const bool live = t0 + threadIdx.y < a.T;
    const int64_t t = live ? t0 + threadIdx.y : a.T - 1;
    const int64_t at = t * a.H;
    const float gt = token ? token_gate<T>(a.gate, a.vec_f32, t) : 1.0f;
    Eight<T> vd, vf, vo, vy, vg;
    if (BULK) {
      const uint8_t* stage = mine + turn.slot * stage_bytes;
      ring_wait(ring, turn, a.status);
      turn.next(stages);
      stage8<T>(stage, c.any() && has_d, vd);
      if (HAS_F) stage8<T>(stage + AT_F * block_bytes, c.any(), vf);
      if (NEXT) {
        stage8<T>(stage + AT_O * block_bytes, c.any(), vo);
        stage8<T>(stage + AT_Y * block_bytes, c.any(), vy);
      }
      if (ELEMENT) stage8<T>(stage + AT_G * block_bytes, c.any(), vg);
    } else {
      if (has_d) {
        load8<T, VEC>(static_cast<const T*>(a.dout) + at, c, vd);
      } else {
#pragma unroll
        for (int j = 0; j < COLS; ++j) vd.e[j] = from_f32<T>(0.0f);
      }
      if (HAS_F) load8<T, VEC>(static_cast<const T*>(a.f) + at, c, vf);
      if (NEXT) {
        load8<T, VEC>(static_cast<const T*>(a.joined) + at, c, vo);
        load8<T, VEC>(static_cast<const T*>(a.dnormed) + at, c, vy);
      }
      if (ELEMENT) load8<T, VEC>(static_cast<const T*>(a.gate) + at, c, vg);
    }
    float s[6] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    {
      float d[COLS], f[COLS], o[COLS], y[COLS], g[COLS];
      unpack8(vd, d);
      if (HAS_F) unpack8(vf, f);
      if (NEXT) unpack8(vo, o);
      if (NEXT) unpack8(vy, y);
      if (ELEMENT) unpack8(vg, g);
#pragma unroll
      for (int j = 0; j < COLS; ++j) {
        const float gf = HAS_F ? w1[j] * f[j] * (ELEMENT ? g[j] : 1.0f) : 0.0f;
        if (NEXT) {
          const float wy = w2[j] * y[j];
          s[0] = fmaf(o[j], o[j], s[0]);
          s[1] = fmaf(wy, o[j], s[1]);
          if (HAS_F) {
            s[4] = fmaf(wy, gf, s[4]);
            s[5] = fmaf(o[j], gf, s[5]);
          }
        }
        if (HAS_F) {
          s[2] = fmaf(f[j], f[j], s[2]);
          s[3] = fmaf(d[j], gf, s[3]);
        }
      }
    }
    row_sum<6>(s, &sums, half, tpr, cluster, rank);
    if (BULK) {   // the stage may be copied over
      if (tpr == 32 && cluster == 1) __syncthreads();
      if (issuer) issue();
    }
    const float r2 = NEXT ? rsqrtf(fmaf(s[0], inv_h, a.eps)) : 0.0f;
    const float m2 = r2 * r2 * (s[1] * inv_h);                      // r2^2 S2 / H
    const float r1 = post ? rsqrtf(fmaf(s[2], inv_h, a.eps)) : 1.0f;
    const float q = s[3] + r2 * (s[4] - m2 * s[5]);
    const float m1 = post ? r1 * r1 * (q * inv_h) : 0.0f;           // r1^2 Q / H
    const float b = a.beta * r1;
    if (token && live && threadIdx.x == 0 && rank == 0) static_cast<float*>(a.dgate)[t] = b * q;
    float d[COLS];
    unpack8(vd, d);
    if (NEXT) {
      float o[COLS], y[COLS];
      unpack8(vo, o);
      unpack8(vy, y);
#pragma unroll
      for (int j = 0; j < COLS; ++j) {
        d[j] = fmaf(r2, fmaf(-o[j], m2, w2[j] * y[j]), d[j]);       // dO
        if (live) s2[j] = fmaf(y[j], o[j] * r2, s2[j]);
      }
    }
    if (HAS_F) {
      float f[COLS], g[COLS];
      unpack8(vf, f);
      if (ELEMENT) unpack8(vg, g);
      const float bm = b * m1;
#pragma unroll
      for (int j = 0; j < COLS; ++j) {
        const float bd = b * d[j], bdf = bd * f[j];                 // beta r1 dO, and times f
        f[j] = gt * fmaf(ELEMENT ? w1[j] * g[j] : w1[j], bd, -f[j] * bm);
        if (live) s1[j] = fmaf(bdf, ELEMENT ? g[j] * gt : gt, s1[j]);
        if (ELEMENT) g[j] = bdf * w1[j];
      }
      pack8<T>(f, vf);
      if (live) store8<T, VEC>(static_cast<T*>(a.dbranch) + at, c, vf);
      if (ELEMENT) {
        pack8<T>(g, vg);
        if (live) store8<T, VEC>(static_cast<T*>(a.dgate) + at, c, vg);
      }
    }
#pragma unroll
    for (int j = 0; j < COLS; ++j) d[j] *= a.alpha;
    pack8<T>(d, vd);
    if (live) store8<T, VEC>(static_cast<T*>(a.dresidual) + at, c, vd);
  }
  if (BULK) ring_end(ring, issued, stages, a.status);
  // The block's rows side by side are added in order, then stored, times the
  // vector that the array's column sums are short of.
  float* part = a.partial + unit * a.arrays * static_cast<int64_t>(a.H);
  auto fold_rows = [&](float (&v)[COLS]) {
    if (blockDim.y == 1) return;
    __syncthreads();
    if (threadIdx.y > 0)
#pragma unroll
      for (int j = 0; j < COLS; ++j) fold[((threadIdx.y - 1) * COLS + j) * tpr + threadIdx.x] = v[j];
    __syncthreads();
    if (threadIdx.y == 0)
      for (int y = 1; y < static_cast<int>(blockDim.y); ++y)
#pragma unroll
        for (int j = 0; j < COLS; ++j) v[j] += fold[((y - 1) * COLS + j) * tpr + threadIdx.x];
  };
  auto put = [&](const float (&v)[COLS], const void* times) {
    if (threadIdx.y == 0) {
      float m[COLS];
      load_vector<T, VEC>(times, a.vec_f32, c, m);
      if (VEC) {
        if (c.any()) {
          float4* p = reinterpret_cast<float4*>(part + c.first);
          p[0] = make_float4(v[0] * m[0], v[1] * m[1], v[2] * m[2], v[3] * m[3]);
          p[1] = make_float4(v[4] * m[4], v[5] * m[5], v[6] * m[6], v[7] * m[7]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < COLS; ++j)
          if (c.col(j) < c.H) part[c.col(j)] = v[j] * m[j];
      }
    }
    part += a.H;
  };
  if (HAS_F && (post || channel)) {
    fold_rows(s1);
    if (post) put(s1, channel ? a.gate : nullptr);
    if (channel) put(s1, a.norm_weight);
  }
  if (NEXT) {
    fold_rows(s2);
    put(s2, nullptr);
  }
}

// out[i] = the sum over the units of partial[unit][i]: 8 slices of the units,
// each in order, then the slices in order.
__global__ void __launch_bounds__(BLOCK) column_sum_kernel(const float* partial, int units, int arrays, int H,
                                                           float* out0, float* out1, float* out2) {
  __shared__ float sm[8][32];
  grid_dependency_wait();
  launch_dependents();
  const int x = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int64_t n = static_cast<int64_t>(arrays) * H, i = static_cast<int64_t>(blockIdx.x) * 32 + x;
  float s = 0.0f;
  if (i < n) {
    constexpr int G = 10;   // loads in flight: half of a slice of 152 units
    for (int u0 = slice; u0 < units; u0 += 8 * G) {
      float v[G];
#pragma unroll
      for (int k = 0; k < G; ++k) v[k] = u0 + 8 * k < units ? partial[(u0 + 8 * k) * n + i] : 0.0f;
#pragma unroll
      for (int k = 0; k < G; ++k) s += v[k];
    }
  }
  sm[slice][x] = s;
  __syncthreads();
  if (slice == 0 && i < n) {
    for (int k = 1; k < 8; ++k) s += sm[k][x];
    float* out = i < H ? out0 : i < 2 * static_cast<int64_t>(H) ? out1 : out2;
    out[i % H] = s;
  }
}

// ---------------------------------------------------------------- launches

constexpr size_t SM_STAGE_BYTES = 200 * 1024;   // of an SM's shared memory, for the rings

template <typename K, typename A>
cudaError_t launch_rows(K kernel, const RowShape& s, int64_t units, size_t smem, int stages, const A& args,
                        cudaStream_t stream) {
  if (smem > 32 * 1024) {   // with the static part possibly past the default of 48 KB
    const cudaError_t err =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (err != cudaSuccess) return err;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * s.cluster));
  cfg.blockDim = dim3(s.tpr, s.rows);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(s.cluster), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = s.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args, s.cluster, stages);
}

// Stages of a ring whose rounds read `arrays` rows of a block's columns, with
// `resident` blocks on an SM: none where a block has one round only.
int ring_stages(const RowShape& s, int64_t H, size_t size, int64_t arrays, int64_t resident, int64_t rounds) {
  const size_t stage = static_cast<size_t>(std::min<int64_t>(H, s.tpr * COLS) * s.rows * arrays) * size;
  const int64_t fit = static_cast<int64_t>(SM_STAGE_BYTES / resident / stage);
  if (rounds < 2 || fit < 2) return 0;
  return static_cast<int>(std::min<int64_t>(std::min<int64_t>(fit, MAX_STAGES), rounds));
}

bool vec_ok(moe_dtype dtype, int64_t H, std::initializer_list<const void*> ptrs) {
  if (H % COLS != 0) return false;
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
  return true;
}

template <typename T, bool VEC, bool BULK>
auto pick_join(int branch, bool element) {
  if (branch == 0) return join_kernel<T, VEC, BULK, 0, false>;
  if (branch == 1) return element ? join_kernel<T, VEC, BULK, 1, true> : join_kernel<T, VEC, BULK, 1, false>;
  return element ? join_kernel<T, VEC, BULK, 2, true> : join_kernel<T, VEC, BULK, 2, false>;
}

template <typename T>
cudaError_t launch_join_t(moe_dtype dtype, JoinArgs a, int branch, int num_sms, cudaStream_t stream) {
  RowShape s = row_shape(a.H);
  const bool vec = vec_ok(dtype, a.H, {a.f, a.x, a.out, a.y, a.norm_weight, a.next_weight,
                                       a.gate_kind == MOE_GATE_TOKEN ? nullptr : a.gate});
  const bool element = a.gate_kind == MOE_GATE_ELEMENT;
  // The expert rows of one token at a time.
  if (branch == 2) s.rows = 1;
  const int64_t groups = (a.T + s.rows - 1) / s.rows;
  // One wave: as many blocks as an SM's registers hold, each row after row.
  const int64_t resident = std::max(1, std::min(16, join_threads(sizeof(T), vec, branch, element) / (s.tpr * s.rows)));
  const int64_t units = std::min<int64_t>(groups, std::max<int64_t>(1, resident * num_sms / s.cluster));
  const int64_t arrays = 1 + (branch == 2 ? a.top_k : branch) + (element ? 1 : 0);
  const int stages = vec && (branch != 2 || a.top_k <= 32)
                         ? ring_stages(s, a.H, sizeof(T), arrays, resident, (groups + units - 1) / units) : 0;
  const size_t smem = static_cast<size_t>(std::min<int64_t>(a.H, s.tpr * COLS) * s.rows * arrays * stages) * sizeof(T);
  return launch_rows(stages > 0 ? pick_join<T, true, true>(branch, element)
                     : vec      ? pick_join<T, true, false>(branch, element)
                                : pick_join<T, false, false>(branch, element),
                     s, units, smem, stages, a, stream);
}

template <typename T, bool VEC, bool BULK>
auto pick_backward(bool has_f, bool next, bool element) {
  if (!has_f) return join_backward_kernel<T, VEC, BULK, false, true, false>;
  if (next)
    return element ? join_backward_kernel<T, VEC, BULK, true, true, true> : join_backward_kernel<T, VEC, BULK, true, true, false>;
  return element ? join_backward_kernel<T, VEC, BULK, true, false, true> : join_backward_kernel<T, VEC, BULK, true, false, false>;
}

template <typename T>
cudaError_t launch_join_backward_t(moe_dtype dtype, const JoinBackwardArgs& a, int64_t units, cudaStream_t stream) {
  const RowShape s = row_shape(a.H);
  const bool vec = vec_ok(dtype, a.H, {a.dout, a.dnormed, a.f, a.joined, a.norm_weight, a.next_weight, a.dbranch,
                                       a.dresidual, a.gate_kind == MOE_GATE_TOKEN ? nullptr : a.gate,
                                       a.gate_kind == MOE_GATE_ELEMENT ? a.dgate : nullptr});
  const bool f = a.f != nullptr, next = a.next_weight != nullptr, element = a.gate_kind == MOE_GATE_ELEMENT;
  const int64_t arrays = 1 + (f ? 1 : 0) + (next ? 2 : 0) + (element ? 1 : 0);
  const int64_t groups = (a.T + s.rows - 1) / s.rows;
  const int64_t resident = std::max(1, MAX_TPR / (s.tpr * s.rows));
  const int stages = vec ? ring_stages(s, a.H, sizeof(T), arrays, resident, (groups + units - 1) / units) : 0;
  const size_t ring = static_cast<size_t>(std::min<int64_t>(a.H, s.tpr * COLS) * s.rows * arrays * stages) * sizeof(T);
  const size_t fold = static_cast<size_t>(s.rows - 1) * s.tpr * COLS * sizeof(float);
  return launch_rows(stages > 0 ? pick_backward<T, true, true>(f, next, element)
                     : vec      ? pick_backward<T, true, false>(f, next, element)
                                : pick_backward<T, false, false>(f, next, element),
                     s, units, std::max(ring, fold), stages, a, stream);
}

}  // namespace

// One wave: a unit keeps its column sums in registers, 512 threads of them
// fill an SM (of JOIN_BACKWARD_SMS).
int64_t join_backward_units(int64_t T, int64_t H) {
  const RowShape s = row_shape(H);
  const int64_t groups = (T + s.rows - 1) / s.rows;
  return std::min<int64_t>(groups, std::max<int64_t>(1, JOIN_BACKWARD_SMS * MAX_TPR / (s.tpr * s.rows * s.cluster)));
}

cudaError_t launch_join(moe_dtype dtype, const JoinArgs& a, int branch, int num_sms, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  JoinArgs args = a;
  const cudaError_t err = device_status_ptr(&args.status);
  if (err != cudaSuccess) return err;
  switch (dtype) {
    case MOE_F32: return launch_join_t<float>(dtype, args, branch, num_sms, stream);
    case MOE_F16: return launch_join_t<__half>(dtype, args, branch, num_sms, stream);
    default: return launch_join_t<__nv_bfloat16>(dtype, args, branch, num_sms, stream);
  }
}

cudaError_t launch_join_backward(moe_dtype dtype, const JoinBackwardArgs& a, float* dnorm_weight, float* dnext_weight,
                                 cudaStream_t stream) {
  const int64_t units = join_backward_units(a.T, a.H);
  cudaError_t err = cudaSuccess;
  if (a.T > 0) {
    JoinBackwardArgs args = a;
    err = device_status_ptr(&args.status);
    if (err != cudaSuccess) return err;
    switch (dtype) {
      case MOE_F32: err = launch_join_backward_t<float>(dtype, args, units, stream); break;
      case MOE_F16: err = launch_join_backward_t<__half>(dtype, args, units, stream); break;
      default: err = launch_join_backward_t<__nv_bfloat16>(dtype, args, units, stream); break;
    }
    if (err != cudaSuccess) return err;
  }
  if (a.arrays == 0) return cudaSuccess;
  float* out[3] = {nullptr, nullptr, nullptr};
  int n = 0;
  if (a.f != nullptr && a.norm_weight != nullptr) out[n++] = dnorm_weight;
  if (a.f != nullptr && a.gate_kind == MOE_GATE_CHANNEL) out[n++] = static_cast<float*>(a.dgate);
  if (a.next_weight != nullptr) out[n++] = dnext_weight;
  const int64_t cols = static_cast<int64_t>(a.arrays) * a.H;
  return launch_dependent(column_sum_kernel, dim3(static_cast<unsigned>((cols + 31) / 32)), dim3(BLOCK), 0, stream,
                          static_cast<const float*>(a.partial), static_cast<int>(units), a.arrays, a.H, out[0], out[1],
                          out[2]);
}

}  // namespace moe
