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
// Layout: a thread owns 8 columns of a row (16 or 32 bytes; in the backward
// twice 8 from 1024 columns on), a row up to 4096 columns one block, more a
// cluster of up to 8 blocks that exchange their sums through distributed shared
// memory. Short rows share a block.
//
// Bound by HBM, 8192 x 4096 BF16 rows: the norm 23 us (5.8 TB/s over the 134 MB
// that it has to move), its backward 51 us (5.3 TB/s over 268 MB), the join's
// backward 78 us (5.2 TB/s over 403 MB). The join of 16384 x 2048 F16 rows 51 us
// (5.3 TB/s over 268 MB), with the combine of 4096 x 8 expert rows 43 us (4.3 TB/s
// over 185 MB). A call for 16 tokens takes 3 to 5 us on the GPU, less than its
// host side.
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
  int tpr;       // threads of a row in a block, a multiple of 32
  int rows;      // rows of a block side by side
  int cluster;   // blocks of a row
};

// chunks: groups of COLS columns that a thread owns.
RowShape row_shape(int64_t H, int chunks = 1) {
  RowShape s;
  s.cluster = 1;
  while (static_cast<int64_t>(s.cluster) * MAX_TPR * COLS < H) s.cluster *= 2;
  const int64_t per = (H + s.cluster - 1) / s.cluster;
  s.tpr = static_cast<int>((per + chunks * COLS * 32 - 1) / (chunks * COLS * 32)) * 32;
  s.rows = s.tpr >= BLOCK / chunks ? 1 : BLOCK / chunks / s.tpr;
  return s;
}

// ---------------------------------------------------------------- a thread's 8 columns

// Its columns: 8 neighbours (VEC: rows and pointers are 16-byte aligned and H
// is a multiple of 8), or every tpr-th one.
template <bool VEC>
struct Cols {
  int first, step, H;
  __device__ Cols() {}
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
  } else if (c.col(COLS - 1) < c.H) {
    T* p = row + c.first;
#pragma unroll
    for (int j = 0; j < COLS; ++j) p[j * c.step] = v.e[j];
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

// COUNT sums (of one row, or one of each of two), for every thread of the rows,
// in two parts with one barrier between them: the two halves of `sm` are used in
// turn, and a half is written again only after the barrier of the call between,
// which every reader of the half has passed. In a warp the values, V of them
// (COUNT rounded up to a power of two), are added by exchanging: a lane gives
// half of its values away until it holds one, number lane / (32 / V), over 32 / V
// lanes: for six sums 9 shuffles in place of 30.
constexpr int pow2_at_least(int n) { return n <= 1 ? 1 : 2 * pow2_at_least((n + 1) / 2); }

template <int COUNT>
struct RowSums {
  static constexpr int V = pow2_at_least(COUNT);
  static constexpr int SLOTS = MAX_CLUSTER * MAX_WARPS;   // block of the cluster * warps + warp, rows side by side in turn
  float v[2][V][SLOTS];
};

// HAVE values of a lane at distance 16, 8, ... (DIST the first) down to one.
template <int HAVE, int DIST>
__device__ __forceinline__ float exchange(const float* v) {
  if constexpr (HAVE == 1) {
    float s = v[0];
#pragma unroll
    for (int off = DIST; off > 0; off >>= 1) s += __shfl_xor_sync(FULL_MASK, s, off);
    return s;
  } else {
    const bool upper = (threadIdx.x & DIST) != 0;
    float kept[HAVE / 2];
#pragma unroll
    for (int i = 0; i < HAVE / 2; ++i) {
      const float keep = upper ? v[i + HAVE / 2] : v[i], give = upper ? v[i] : v[i + HAVE / 2];
      kept[i] = keep + __shfl_xor_sync(FULL_MASK, give, DIST);
    }
    return exchange<HAVE / 2, DIST / 2>(kept);
  }
}

// First part: the warp's sums, one per lane, and into `half` of sm.
template <int COUNT>
__device__ __forceinline__ float post_sums(const float (&s)[COUNT], RowSums<COUNT>* sm, int half, int tpr, int cluster,
                                           int rank) {
  constexpr int V = RowSums<COUNT>::V, LANES = 32 / V;   // lanes of a value
  const int lane = threadIdx.x & 31, which = lane / LANES, part = lane % LANES;
  float all[V];
#pragma unroll
  for (int i = 0; i < V; ++i) all[i] = i < COUNT ? s[i < COUNT ? i : 0] : 0.0f;
  const float mine = exchange<V, 16>(all);
  if (tpr > 32 || cluster > 1) {
    const int warps = tpr >> 5;
    float* at = &sm->v[half][which][threadIdx.y * warps];
    if (cluster == 1) {
      if (part == 0) at[threadIdx.x >> 5] = mine;
    } else {
      for (int to = part; to < cluster; to += LANES)
        *cg::this_cluster().map_shared_rank(at + rank * warps + (threadIdx.x >> 5), to) = mine;
    }
  }
  return mine;
}
// The barrier between the two parts.
__device__ __forceinline__ void sums_barrier(int cluster) {
  if (cluster == 1) __syncthreads();
  else cg::this_cluster().sync();
}
// Second part, with the first one's value: the row's sums.
template <int COUNT>
__device__ __forceinline__ void take_sums(float (&s)[COUNT], float mine, const RowSums<COUNT>* sm, int half, int tpr,
                                          int cluster) {
  constexpr int V = RowSums<COUNT>::V, LANES = 32 / V;
  const int lane = threadIdx.x & 31, which = lane / LANES, part = lane % LANES;
  if (tpr > 32 || cluster > 1) {
    const int warps = tpr >> 5;
    const float* at = &sm->v[half][which][threadIdx.y * warps];
    mine = 0.0f;
    for (int w = part; w < cluster * warps; w += LANES) mine += at[w];
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) mine += __shfl_xor_sync(FULL_MASK, mine, off);
  }
  if (V == 1) {
    s[0] = mine;
  } else {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) s[i] = __shfl_sync(FULL_MASK, mine, i * LANES);
  }
}
template <int COUNT>
__device__ __forceinline__ void row_sum(float (&s)[COUNT], RowSums<COUNT>* sm, int& half, int tpr, int cluster, int rank) {
  const float mine = post_sums<COUNT>(s, sm, half, tpr, cluster, rank);
  if (tpr > 32 || cluster > 1) sums_barrier(cluster);
  take_sums<COUNT>(s, mine, sm, half, tpr, cluster);
  half ^= 1;
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

// A ring of rounds in shared memory: one warp copies what a round reads, as whole
// rows by bulk copies, several rounds before its turn. An SM needs some 70 KB of
// loads in flight for its share of HBM's rate; in registers one round ahead is
// all there is room for (the backward of 8192 x 4096 BF16 rows ran at 1.9 TB/s
// that way).
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

// Whether a round's rows are there; a wait that runs out leaves the call's
// results undefined.
// Every thread of the block waits here: the clock is read after many tries only.
__device__ __forceinline__ bool ring_wait(Ring& ring, const Turn& turn, uint32_t* status) {
  uint64_t* bar = &ring.full[turn.slot];
  for (int tries = 0; tries < 256; ++tries) {
    if (mbar_try_wait(bar, turn.parity)) return true;
    if (*static_cast<volatile int*>(&ring.abort_flag) != 0) return false;   // the rounds after a give-up end at once
  }
  return mbar_wait_bounded(bar, turn.parity, &ring.abort_flag, status, ST_ROWS, WAIT_LIMIT_NS);
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

// n rows of this block's columns: one copy where the block has whole rows.
template <typename T>
__device__ __forceinline__ void copy_rows(uint8_t* dst, const T* src, uint32_t n, uint32_t row_bytes, int H, int cluster,
                                          uint64_t* bar) {
  if (row_bytes == 0) return;
  if (cluster == 1) {
    bulk_load(dst, src, row_bytes * n, bar);
  } else {
    for (uint32_t r = 0; r < n; ++r) bulk_load(dst + r * row_bytes, src + r * static_cast<int64_t>(H), row_bytes, bar);
  }
}

// Rows that do not lie on 16-byte boundaries come as the 16-byte granules that
// they touch, to a place with room for that: a round's rows together where a
// block has whole rows, else row by row. What a granule holds of the rows beside
// them is not looked at (nor is it waited for: another block may be storing it).
__host__ __device__ constexpr uint32_t loose_pitch(uint32_t bytes) { return (bytes + 30) & ~15u; }
// Bytes from row to row in a stage, and of a round's rows.
__host__ __device__ constexpr uint32_t staged_row(uint32_t row_bytes, int cluster, bool vec) {
  return vec || cluster == 1 ? row_bytes : loose_pitch(row_bytes);
}
__host__ __device__ constexpr uint32_t staged_rows(uint32_t row_bytes, uint32_t rows, int cluster, bool vec) {
  return vec ? row_bytes * rows : cluster == 1 ? loose_pitch(row_bytes * rows) : loose_pitch(row_bytes) * rows;
}

// The copy of one such run: `bytes` (0: none) from `src` to `dst`.
struct LooseRow {
  const uint8_t* src;
  uint8_t* dst;
  uint32_t bytes;
};
// The copy of the run at `row` into its place, from a tensor [begin, end). A
// granule that is not the tensor's as a whole (its first, its last) is not
// copied; its elements are stored here.
template <typename T>
__device__ __forceinline__ LooseRow loose_row(uint8_t* place, const T* row, uint32_t row_bytes, const T* begin,
                                              const T* end) {
  const uintptr_t from = reinterpret_cast<uintptr_t>(row), to = from + row_bytes;
  uintptr_t lo = from & ~uintptr_t{15}, hi = (to + 15) & ~uintptr_t{15};
  const uintptr_t zero = lo;   // of the place
  const bool head = lo < reinterpret_cast<uintptr_t>(begin), tail = hi > reinterpret_cast<uintptr_t>(end);
  if (row_bytes == 0) return {nullptr, nullptr, 0u};
  if (head || tail) {
    if (head) lo += 16;
    if (tail && hi > lo) hi -= 16;
    const uintptr_t stop = min(lo, to);
    for (uintptr_t p = from; head && p < stop; p += sizeof(T))
      *reinterpret_cast<T*>(place + (p - zero)) = *reinterpret_cast<const T*>(p);
    for (uintptr_t p = max(hi, from); tail && p < to; p += sizeof(T))
      *reinterpret_cast<T*>(place + (p - zero)) = *reinterpret_cast<const T*>(p);
    fence_proxy_async_smem();   // before the next round's copies to this place
  }
  return {reinterpret_cast<const uint8_t*>(lo), place + (lo - zero), hi > lo ? static_cast<uint32_t>(hi - lo) : 0u};
}
__device__ __forceinline__ void loose_load(const LooseRow& r, uint64_t* bar) {
  if (r.bytes > 0) bulk_load(r.dst, r.src, r.bytes, bar);
}
// Where in its place the run from that element on starts.
__device__ __forceinline__ uint32_t loose_start(const void* tensor, uint32_t element, uint32_t size) {
  return (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(tensor)) + element * size) & 15u;
}
// A thread's columns of such a row (at its first column, `tid` in).
template <typename T>
__device__ __forceinline__ void loose8(const uint8_t* row, const Cols<false>& c, int tid, Eight<T>& v) {
  const T* p = reinterpret_cast<const T*>(row) + tid;
  if (c.col(COLS - 1) < c.H) {
#pragma unroll
    for (int j = 0; j < COLS; ++j) v.e[j] = p[j * c.step];
  } else {
#pragma unroll
    for (int j = 0; j < COLS; ++j) v.e[j] = c.col(j) < c.H ? p[j * c.step] : from_f32<T>(0.0f);
  }
}

// This thread's columns of a row in a stage (a thread past the row's columns is
// given any others: it adds and stores nothing).
template <typename T>
__device__ __forceinline__ void stage8(const uint8_t* mine, Eight<T>& v) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(v) / 16); ++i)
    reinterpret_cast<uint4*>(&v)[i] = reinterpret_cast<const uint4*>(mine)[i];
}

// ---------------------------------------------------------------- forward

// BRANCH: 0 none (the norm alone), 1 rows of f, 2 the combine of expert rows.
// ELEMENT: a gate for every element.
//
// Bound by HBM: x and f in (combine: top_k rows), out and y out. BULK: rounds
// come through the ring; else (calls of one round a block, many slots) they are
// loaded when their turn comes. Loose rows (not VEC) leave the ring and the
// kernel element by element, 32 neighbours a warp: in FP32 that keeps up with HBM
// (join of 8192 x 4095 92 us, of 4096 columns 95), in 16 bits as many narrow loads
// and stores take as long (87 us, 53; without the ring 148).

// Threads that an SM holds: 1024 of 64 registers where that is enough (loose rows,
// 2048 x 8191 BF16: 25 us, 30 with 512).
constexpr int join_threads(size_t size, int branch, bool element) {
  return size == 2 && branch < 1 && !element ? 1024 : 512;
}
// Rows of a thread in a round: two share a round's barriers and index
// arithmetic, which are most of a row's instructions.
constexpr int join_rows(bool bulk, int branch) { return bulk && branch != 2 ? 2 : 1; }

template <typename T, bool VEC, bool BULK, int BRANCH, bool ELEMENT>
__global__ void __launch_bounds__(MAX_TPR, join_threads(sizeof(T), BRANCH, ELEMENT) / MAX_TPR)
    join_kernel(const JoinArgs a, int cluster, int stages) {
  constexpr int R = join_rows(BULK, BRANCH);
  __shared__ RowSums<R> sums;
  __shared__ Ring ring;
  extern __shared__ __align__(128) uint8_t stage_smem[];
  const int tpr = blockDim.x;
  const int rank = cluster > 1 ? static_cast<int>(blockIdx.x) % cluster : 0;
  const uint32_t rows = static_cast<uint32_t>(a.T), round_rows = blockDim.y * R;
  const uint32_t step = gridDim.x / cluster * round_rows, first_row = blockIdx.x / cluster * round_rows;
  const Cols<VEC> c(threadIdx.x, tpr, rank, a.H);
  const int lane = threadIdx.x & 31;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  const bool post = BRANCH != 0 && a.norm_weight != nullptr;
  const bool next = BRANCH == 0 || a.next_weight != nullptr;
  const bool token = BRANCH != 0 && a.gate_kind == MOE_GATE_TOKEN;
  int half = 0;
  if (BULK) ring_init(ring, stages);
  if (cluster > 1) cg::this_cluster().sync();   // every block runs before another one writes to its sums
  grid_dependency_wait();
  launch_dependents();

  // The ring: a stage holds x, then f or the expert rows, then the gates, each
  // of this block's columns.
  const int cols = max(min(tpr * COLS, a.H - rank * tpr * COLS), 0);
  const uint32_t row_bytes = cols * static_cast<uint32_t>(sizeof(T));
  const uint32_t row_pitch = staged_row(row_bytes, cluster, VEC);
  const uint32_t block_bytes = staged_rows(row_bytes, round_rows, cluster, VEC);
  const uint32_t stage_bytes = block_bytes * (1 + (BRANCH == 2 ? a.top_k : BRANCH) + (ELEMENT ? 1 : 0));
  // Combine: lane j's expert row of a token's first 32 slots.
  auto slot_of = [&](uint32_t t) {
    return lane < a.top_k && t < rows ? a.inv[static_cast<int64_t>(t) * a.top_k + lane] : 0xFFFFFFFFu;
  };
  auto weight_of = [&](uint32_t t) {
    return lane < a.top_k && t < rows ? weight_at(a.weights, a.weights_dtype, static_cast<int64_t>(t) * a.top_k + lane)
                                      : 0.0f;
  };
  uint32_t issued = 0, issue_t0 = first_row;
  Turn fill{0, 0u};
  uint32_t ahead = BRANCH == 2 && BULK ? slot_of(issue_t0) : 0;   // slots of the round to be issued next
  auto issue = [&]() {   // by the first warp of the block
    if (issue_t0 >= rows) return;
    uint8_t* dst = stage_smem + fill.slot * stage_bytes;
    uint64_t* bar = &ring.full[fill.slot];
    const int64_t at = static_cast<int64_t>(issue_t0) * a.H + rank * tpr * COLS;
    const uint32_t n = min(round_rows, rows - issue_t0);
    const bool good = BRANCH == 2 && ahead < a.rows;
    if (!VEC) {   // a lane a run
      const int64_t total = static_cast<int64_t>(rows) * a.H, mine = at + lane * static_cast<int64_t>(a.H);
      LooseRow copies[4] = {};
      auto take = [&](int i, uint32_t offset, const void* tensor, int64_t first, uint32_t bytes, int64_t elements) {
        const T* p = static_cast<const T*>(tensor);
        copies[i] = loose_row<T>(dst + offset, p + first, bytes, p, p + elements);
      };
      if (static_cast<uint32_t>(lane) < (cluster == 1 ? 1u : n)) {
        const uint32_t place = lane * row_pitch, bytes = cluster == 1 ? row_bytes * n : row_bytes;
        take(0, place, a.x, mine, bytes, total);
        if (BRANCH == 1) take(1, block_bytes + place, a.f, mine, bytes, total);
        if (ELEMENT) take(2, stage_bytes - block_bytes + place, a.gate, mine, bytes, total);
      }
      if (good)
        take(3, (1 + lane) * block_bytes, a.f, static_cast<int64_t>(ahead) * a.H + rank * tpr * COLS, row_bytes,
             static_cast<int64_t>(a.rows) * a.H);
      uint32_t bytes = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) bytes += copies[i].bytes;
      bytes = __reduce_add_sync(FULL_MASK, bytes);
      __syncwarp();   // the lanes' stores (loose_row) before the arrive, which the sum alone does not order
      if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
      __syncwarp();   // the expected bytes before the copies that bring them
#pragma unroll
      for (int i = 0; i < 4; ++i) loose_load(copies[i], bar);
    } else if (BRANCH == 2) {
      const uint32_t found = __popc(__ballot_sync(FULL_MASK, good));
      if (lane == 0) mbar_arrive_expect_tx(bar, row_bytes * ((ELEMENT ? 2 : 1) + found));
      __syncwarp();
      if (good && cols > 0)
        bulk_load(dst + (1 + lane) * row_bytes,
                  static_cast<const T*>(a.f) + static_cast<int64_t>(ahead) * a.H + rank * tpr * COLS, row_bytes, bar);
    }
    if (VEC && lane == 0) {
      if (BRANCH != 2) mbar_arrive_expect_tx(bar, row_bytes * n * (1 + BRANCH + (ELEMENT ? 1 : 0)));
      copy_rows<T>(dst, static_cast<const T*>(a.x) + at, n, row_bytes, a.H, cluster, bar);
      if (BRANCH == 1) copy_rows<T>(dst + block_bytes, static_cast<const T*>(a.f) + at, n, row_bytes, a.H, cluster, bar);
      if (ELEMENT)
        copy_rows<T>(dst + stage_bytes - block_bytes, static_cast<const T*>(a.gate) + at, n, row_bytes, a.H, cluster, bar);
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
  // row past the end as a row that is not stored. A round's scalars are loaded
  // a round ahead.
  Turn turn{0, 0u};
  const uint8_t* mine = stage_smem + threadIdx.y * R * row_pitch +
                        (VEC && c.any() ? threadIdx.x * (COLS * static_cast<uint32_t>(sizeof(T))) : 0u);
  // This thread's columns of a row in its stage; `first`: the run's first row.
  auto staged = [&](const uint8_t* place, const void* tensor, uint32_t first, Eight<T>& v) {
    if constexpr (VEC)
      stage8<T>(place, v);
    else
      loose8<T>(place + loose_start(tensor, first * static_cast<uint32_t>(a.H) + rank * tpr * COLS, sizeof(T)), c,
                threadIdx.x, v);
  };
  const bool row_barrier = tpr > 32 || cluster > 1;
  uint32_t t = first_row + threadIdx.y * R;   // this thread's first row
  auto gate_of = [&](uint32_t row) { return token && row < rows ? token_gate<T>(a.gate, a.vec_f32, row) : 1.0f; };
  float gate_next[R];
#pragma unroll
  for (int r = 0; r < R; ++r) gate_next[r] = gate_of(t + r);
  uint32_t slot_next = BRANCH == 2 ? slot_of(t) : 0;
  float weight_next = BRANCH == 2 ? weight_of(t) : 0.0f;
  for (uint32_t t0 = first_row; t0 < rows; t0 += step, t += step) {
    float g[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      g[r] = a.beta * gate_next[r];
      gate_next[r] = gate_of(t + step + r);
    }
    uint32_t slot = slot_next;
    float weight = weight_next;
    if (BRANCH == 2) {
      slot_next = slot_of(t + step);
      weight_next = weight_of(t + step);
    }
    const int64_t at = static_cast<int64_t>(min(t, rows - 1)) * a.H;
    Eight<T> raw, gv[R];
    float x[R][COLS], f[R][COLS];
    const uint8_t* stage = mine + turn.slot * stage_bytes;
    if (BULK) {
      issue_only_after(__all_sync(FULL_MASK, ring_wait(ring, turn, a.status)), issue_t0, rows);
      turn.next(stages);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t run = cluster == 1 ? t0 : t + r;
      if (BULK) staged(stage + r * row_pitch, a.x, run, raw);
      else load8<T, VEC>(static_cast<const T*>(a.x) + at, c, raw);
      unpack8(raw, x[r]);
      if (ELEMENT) {
        if (BULK) staged(stage + stage_bytes - block_bytes + r * row_pitch, a.gate, run, gv[r]);
        else load8<T, VEC>(static_cast<const T*>(a.gate) + at, c, gv[r]);
      }
      if (BRANCH == 1) {
        if (BULK) staged(stage + block_bytes + r * row_pitch, a.f, run, raw);
        else load8<T, VEC>(static_cast<const T*>(a.f) + at, c, raw);
        unpack8(raw, f[r]);
      }
    }
    if (BRANCH == 2) {
      // Slot order, as moe_combine; a bad row number makes the token NaN.
#pragma unroll
      for (int j = 0; j < COLS; ++j) f[0][j] = 0.0f;
      bool bad = __any_sync(FULL_MASK, lane < a.top_k && slot >= a.rows);
      if (BULK) {
#pragma unroll 4
        for (int k = 0; k < a.top_k; ++k) {
          Eight<T> v;
          float y[COLS];
          const float w = __shfl_sync(FULL_MASK, weight, k);
          const uint32_t row = VEC ? 0u : __shfl_sync(FULL_MASK, slot, k);
          staged(stage + (1 + k) * block_bytes, a.f, row, v);
          unpack8(v, y);
#pragma unroll
          for (int j = 0; j < COLS; ++j) f[0][j] = fmaf(w, y[j], f[0][j]);
        }
      }
      constexpr int G = 4;   // rows whose loads are in flight together
      const int64_t slot0 = static_cast<int64_t>(min(t, rows - 1)) * a.top_k;
      for (int first = 0; !BULK && first < a.top_k; first += 32) {
        if (first > 0 && first + lane < a.top_k) {
          slot = a.inv[slot0 + first + lane];
          weight = weight_at(a.weights, a.weights_dtype, slot0 + first + lane);
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
              load8<T, VEC>(static_cast<const T*>(a.f) + static_cast<int64_t>(row) * a.H, c, v[i]);
            }
          }
#pragma unroll
          for (int i = 0; i < G; ++i)
            if (k0 + i < here) {
              float y[COLS];
              unpack8(v[i], y);
#pragma unroll
              for (int j = 0; j < COLS; ++j) f[0][j] = fmaf(w[i], y[j], f[0][j]);
            }
        }
      }
      if (bad)
#pragma unroll
        for (int j = 0; j < COLS; ++j) f[0][j] = __int_as_float(0x7FC00000);
    }
    // The first of the round's barriers after which the stage may be copied over.
    bool freed = !BULK;
    auto free_stage = [&](bool barrier) {
      if (freed) return;
      freed = true;
      if (!barrier) __syncthreads();
      if (issuer) issue();
    };
    auto sum_squares = [&](const float (&v)[R][COLS], float (&s)[R]) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        s[r] = 0.0f;
#pragma unroll
        for (int j = 0; j < COLS; ++j)
          if (VEC || c.col(j) < c.H) s[r] = fmaf(v[r][j], v[r][j], s[r]);
        if (VEC && !c.any()) s[r] = 0.0f;   // a thread past the row may hold a token's NaN
      }
      row_sum<R>(s, &sums, half, tpr, cluster, rank);
      free_stage(row_barrier);
    };
    float s[R];
    if (BRANCH != 0) {
      if (post) {
        sum_squares(f, s);
#pragma unroll
        for (int r = 0; r < R; ++r) g[r] *= rsqrtf(fmaf(s[r], inv_h, a.eps));
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float gate[COLS];
        if (ELEMENT) unpack8(gv[r], gate);
#pragma unroll
        for (int j = 0; j < COLS; ++j)
          x[r][j] = fmaf(a.alpha, x[r][j], f[r][j] * g[r] * w1[j] * (ELEMENT ? gate[j] : 1.0f));
        pack8<T>(x[r], raw);
        if (t + r < rows) store8<T, VEC>(static_cast<T*>(a.out) + at + r * static_cast<int64_t>(a.H), c, raw);
        unpack8(raw, x[r]);
      }
    }
    if (next) {
      sum_squares(x, s);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float rs = rsqrtf(fmaf(s[r], inv_h, a.eps));
#pragma unroll
        for (int j = 0; j < COLS; ++j) x[r][j] = x[r][j] * rs * w2[j];
        pack8<T>(x[r], raw);
        if (t + r < rows) store8<T, VEC>(static_cast<T*>(a.y) + at + r * static_cast<int64_t>(a.H), c, raw);
      }
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
// Bound by HBM (join: dout, dy, out, f in, dx, df out). BULK as in the forward
// (loose rows of 8192 x 4095 144 us in BF16, 138 in FP32; without the ring 187 and
// 213; aligned ones 77 and 130). An aligned round's work is in two halves, the
// sums and, a round later, the results, so that one round's barrier and shuffles
// run beside another one's arithmetic; loose rows, whose narrow loads are dear,
// go in one (in two the 144 us were 389). A thread owns CHUNKS groups of 8
// columns: with two of them a row has half the shuffles, and two blocks of 256
// threads share an SM for rows of 4096.
template <typename T, bool VEC, int CHUNKS, bool BULK, bool HAS_F, bool NEXT, bool ELEMENT>
__global__ void __launch_bounds__(MAX_TPR / CHUNKS, CHUNKS) join_backward_kernel(const JoinBackwardArgs a, int cluster,
                                                                                 int stages) {
  static_assert(BULK || CHUNKS == 1, "rows from memory: one group of columns");
  // Sums of a row: out^2, w2 dy out, f^2, dout G f, w2 dy G f, out G f (those that are needed).
  constexpr int N = HAS_F && NEXT ? 6 : 2;
  constexpr int AT_FF = HAS_F && NEXT ? 2 : 0, AT_DF = AT_FF + 1, AT_YF = 4, AT_OF = 5;
  __shared__ RowSums<N> sums;
  __shared__ Ring ring;
  extern __shared__ __align__(128) uint8_t stage_smem[];   // the ring; in the end [rows of the block - 1][tpr * COLS] sums
  float* fold = reinterpret_cast<float*>(stage_smem);
  const int tpr = blockDim.x;
  const int rank = cluster > 1 ? static_cast<int>(blockIdx.x) % cluster : 0;
  const uint32_t rows = static_cast<uint32_t>(a.T), round_rows = blockDim.y;
  const int64_t unit = blockIdx.x / cluster;
  const uint32_t step = gridDim.x / cluster * round_rows, first_row = static_cast<uint32_t>(unit) * round_rows;
  const int block_cols = tpr * COLS * CHUNKS;
  Cols<VEC> c[CHUNKS];
#pragma unroll
  for (int k = 0; k < CHUNKS; ++k) {
    c[k] = Cols<VEC>(threadIdx.x, tpr, 0, a.H);
    c[k].first += rank * block_cols + k * tpr * COLS;
  }
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
  const int cols = max(min(block_cols, a.H - rank * block_cols), 0);   // a cluster's last block may have none
  const uint32_t row_bytes = cols * static_cast<uint32_t>(sizeof(T));
  const uint32_t row_pitch = staged_row(row_bytes, cluster, VEC);
  const uint32_t block_bytes = staged_rows(row_bytes, round_rows, cluster, VEC);
  constexpr int ARRAYS = 1 + (HAS_F ? 1 : 0) + (NEXT ? 2 : 0) + (ELEMENT ? 1 : 0);
  constexpr int AT_F = 1, AT_O = 1 + (HAS_F ? 1 : 0), AT_Y = AT_O + 1, AT_G = ARRAYS - 1;
  const uint32_t stage_bytes = block_bytes * ARRAYS;
  uint32_t issued = 0, issue_t0 = first_row;
  const uint32_t lane = threadIdx.x & 31;
  Turn fill{0, 0u};
  auto issue = [&]() {   // by the first thread of the block, loose rows by its first warp
    if (issue_t0 >= rows) return;
    uint8_t* dst = stage_smem + fill.slot * stage_bytes;
    uint64_t* bar = &ring.full[fill.slot];
    const int64_t at = static_cast<int64_t>(issue_t0) * a.H + rank * block_cols;
    const uint32_t n = min(round_rows, rows - issue_t0);   // a cluster's blocks have one row
    if (!VEC) {   // a lane an array
      const int64_t total = static_cast<int64_t>(rows) * a.H;
      const void* const tensors[5] = {has_d ? a.dout : nullptr, HAS_F ? a.f : nullptr, NEXT ? a.joined : nullptr,
                                      NEXT ? a.dnormed : nullptr, ELEMENT ? a.gate : nullptr};
      constexpr int PLACES[5] = {0, AT_F, AT_O, AT_Y, AT_G};
      LooseRow copy{};
#pragma unroll
      for (int i = 0; i < 5; ++i)
        if (lane == i && tensors[i] != nullptr) {
          const T* p = static_cast<const T*>(tensors[i]);
          copy = loose_row<T>(dst + PLACES[i] * block_bytes, p + at, row_bytes * n, p, p + total);
        }
      const uint32_t bytes = __reduce_add_sync(FULL_MASK, copy.bytes);
      __syncwarp();   // the lanes' stores (loose_row) before the arrive, which the sum alone does not order
      if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
      __syncwarp();   // the expected bytes before the copies that bring them
      loose_load(copy, bar);
    } else {
      const uint32_t bytes = row_bytes * n;
      auto copy = [&](int array, const void* src) {
        bulk_load(dst + array * block_bytes, static_cast<const T*>(src) + at, bytes, bar);
      };
      mbar_arrive_expect_tx(bar, bytes * (ARRAYS - (has_d ? 0 : 1)));
      if (bytes > 0) {
        if (has_d) copy(0, a.dout);
        if (HAS_F) copy(AT_F, a.f);
        if (NEXT) copy(AT_O, a.joined);
        if (NEXT) copy(AT_Y, a.dnormed);
        if (ELEMENT) copy(AT_G, a.gate);
      }
    }
    ++issued;
    fill.next(stages);
    issue_t0 += step;
  };
  const bool issuer = BULK && threadIdx.x < (VEC ? 1 : 32) && threadIdx.y == 0;
  if (issuer)
    for (int i = 0; i < stages; ++i) issue();

  float w1[CHUNKS][COLS], w2[CHUNKS][COLS];   // w1: with a channel's gate
  float s1[CHUNKS][COLS], s2[CHUNKS][COLS];   // column sums S and dw2
#pragma unroll
  for (int k = 0; k < CHUNKS; ++k) {
#pragma unroll
    for (int j = 0; j < COLS; ++j) s1[k][j] = s2[k][j] = 0.0f;
    if (HAS_F) {
      load_vector<T, VEC>(a.norm_weight, a.vec_f32, c[k], w1[k]);
      if (channel) {
        float g[COLS];
        load_vector<T, VEC>(a.gate, a.vec_f32, c[k], g);
#pragma unroll
        for (int j = 0; j < COLS; ++j) w1[k][j] *= g[j];
      }
    }
    if (NEXT) load_vector<T, VEC>(a.next_weight, a.vec_f32, c[k], w2[k]);
  }

  uint32_t mine[CHUNKS];   // this thread's columns in a stage
#pragma unroll
  for (int k = 0; k < CHUNKS; ++k)
    mine[k] = threadIdx.y * row_pitch +
              (VEC && c[k].any() ? (k * tpr + threadIdx.x) * (COLS * static_cast<uint32_t>(sizeof(T))) : 0u);
  auto gate_of = [&](uint32_t row) { return token && row < rows ? token_gate<T>(a.gate, a.vec_f32, row) : 1.0f; };
  struct Part {   // a thread's chunk of a row
    Eight<T> d, f, o, y, g;
  };
  auto load_part = [&](uint32_t t, int k, int slot, Part& v) {   // (threadIdx.y: its row's place in the round)
    if (BULK) {
      const uint8_t* row = stage_smem + slot * stage_bytes + mine[k];
      auto staged = [&](int array, const void* tensor, Eight<T>& to) {
        const uint8_t* place = row + array * block_bytes;
        if constexpr (VEC) {
          stage8<T>(place, to);
        } else {
          const uint32_t element = (t - threadIdx.y) * static_cast<uint32_t>(a.H) + rank * block_cols;
          loose8<T>(place + loose_start(tensor, element, sizeof(T)), c[k], k * tpr * COLS + threadIdx.x, to);
        }
      };
      if (has_d) {
        staged(0, a.dout, v.d);
      } else {
#pragma unroll
        for (int j = 0; j < COLS; ++j) v.d.e[j] = from_f32<T>(0.0f);
      }
      if (HAS_F) staged(AT_F, a.f, v.f);
      if (NEXT) staged(AT_O, a.joined, v.o);
      if (NEXT) staged(AT_Y, a.dnormed, v.y);
      if (ELEMENT) staged(AT_G, a.gate, v.g);
    } else {
      const int64_t at = static_cast<int64_t>(min(t, rows - 1)) * a.H;
      if (has_d) {
        load8<T, VEC>(static_cast<const T*>(a.dout) + at, c[k], v.d);
      } else {
#pragma unroll
        for (int j = 0; j < COLS; ++j) v.d.e[j] = from_f32<T>(0.0f);
      }
      if (HAS_F) load8<T, VEC>(static_cast<const T*>(a.f) + at, c[k], v.f);
      if (NEXT) load8<T, VEC>(static_cast<const T*>(a.joined) + at, c[k], v.o);
      if (NEXT) load8<T, VEC>(static_cast<const T*>(a.dnormed) + at, c[k], v.y);
      if (ELEMENT) load8<T, VEC>(static_cast<const T*>(a.gate) + at, c[k], v.g);
    }
  };
  auto add_up = [&](const Part& v, int k, float (&p)[N]) {
    float d[COLS], f[COLS], o[COLS], y[COLS], g[COLS];
    if (HAS_F) unpack8(v.d, d);
    if (HAS_F) unpack8(v.f, f);
    if (NEXT) unpack8(v.o, o);
    if (NEXT) unpack8(v.y, y);
    if (ELEMENT) unpack8(v.g, g);
#pragma unroll
    for (int j = 0; j < COLS; ++j) {
      const float gf = HAS_F ? w1[k][j] * f[j] * (ELEMENT ? g[j] : 1.0f) : 0.0f;
      if (NEXT) {
        const float wy = w2[k][j] * y[j];
        p[0] = fmaf(o[j], o[j], p[0]);
        p[1] = fmaf(wy, o[j], p[1]);
        if (HAS_F) {
          p[AT_YF] = fmaf(wy, gf, p[AT_YF]);
          p[AT_OF] = fmaf(o[j], gf, p[AT_OF]);
        }
      }
      if (HAS_F) {
        p[AT_FF] = fmaf(f[j], f[j], p[AT_FF]);
        p[AT_DF] = fmaf(d[j], gf, p[AT_DF]);
      }
    }
  };
  // A row's factors from its sums, and its results.
  struct Factors {
    float r2, m2, b, bm;
  };
  auto factors_of = [&](uint32_t t, const float (&p)[N], float gt) {
    Factors x;
    x.r2 = NEXT ? rsqrtf(fmaf(p[0], inv_h, a.eps)) : 0.0f;
    x.m2 = NEXT ? x.r2 * x.r2 * (p[1] * inv_h) : 0.0f;              // r2^2 S2 / H
    const float r1 = post ? rsqrtf(fmaf(p[AT_FF], inv_h, a.eps)) : 1.0f;
    const float q = HAS_F && NEXT ? p[AT_DF] + x.r2 * (p[AT_YF] - x.m2 * p[AT_OF]) : p[AT_DF];
    const float b = a.beta * r1;
    x.b = b * gt;                                                   // beta r1 and a token's gate
    x.bm = post ? x.b * (r1 * r1 * (q * inv_h)) : 0.0f;             // times r1^2 Q / H
    if (token && t < rows && threadIdx.x == 0 && rank == 0) static_cast<float*>(a.dgate)[t] = b * q;
    return x;
  };
  auto finish = [&](Part& v, uint32_t t, int k, const Factors& x) {
    const int64_t to = static_cast<int64_t>(t) * a.H;
    float d[COLS];
    unpack8(v.d, d);
    if (NEXT) {
      float o[COLS], y[COLS];
      unpack8(v.o, o);
      unpack8(v.y, y);
#pragma unroll
      for (int j = 0; j < COLS; ++j) {
        d[j] = fmaf(x.r2, fmaf(-o[j], x.m2, w2[k][j] * y[j]), d[j]);   // dO
        s2[k][j] = fmaf(y[j], o[j] * x.r2, s2[k][j]);
      }
    }
    if (HAS_F) {
      float f[COLS], g[COLS];
      unpack8(v.f, f);
      if (ELEMENT) unpack8(v.g, g);
#pragma unroll
      for (int j = 0; j < COLS; ++j) {
        const float bd = x.b * d[j];
        s1[k][j] = fmaf(ELEMENT ? bd * g[j] : bd, f[j], s1[k][j]);
        const float dg = bd * f[j] * w1[k][j];
        f[j] = fmaf(ELEMENT ? w1[k][j] * g[j] : w1[k][j], bd, -f[j] * x.bm);
        if (ELEMENT) g[j] = dg;
      }
      pack8<T>(f, v.f);
      store8<T, VEC>(static_cast<T*>(a.dbranch) + to, c[k], v.f);
      if (ELEMENT) {
        pack8<T>(g, v.g);
        store8<T, VEC>(static_cast<T*>(a.dgate) + to, c[k], v.g);
      }
    }
    if (a.alpha != 1.0f)
#pragma unroll
      for (int j = 0; j < COLS; ++j) d[j] *= a.alpha;
    pack8<T>(d, v.d);
    store8<T, VEC>(static_cast<T*>(a.dresidual) + to, c[k], v.d);
  };
  if (BULK && VEC) {
    Turn turn{0, 0u};   // of the sums; the results are one turn behind
    uint32_t t = first_row + threadIdx.y;
    float share = 0.0f, gate_next = gate_of(t);
    bool behind = false;
    for (uint32_t t0 = first_row; t0 < rows || behind; t0 += step, t += step) {
      const bool ahead = t0 < rows;
      const float share_before = share, gt = gate_next;
      const int slot_before = turn.slot == 0 ? stages - 1 : turn.slot - 1;
      if (ahead) {
        issue_only_after(ring_wait(ring, turn, a.status), issue_t0, rows);
        float p[N];
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
          Part v;
          load_part(t, k, turn.slot, v);
          if (k > 0 && !c[k].any()) continue;   // (the first group is whole, or all of the thread is past the row)
          add_up(v, k, p);
        }
        if (!c[0].any())
#pragma unroll
          for (int i = 0; i < N; ++i) p[i] = 0.0f;
        share = post_sums<N>(p, &sums, half, tpr, cluster, rank);
        turn.next(stages);
      }
      if (behind) {
        float p[N];
        take_sums<N>(p, share_before, &sums, half ^ 1, tpr, cluster);
        gate_next = gate_of(t);
        const Factors x = factors_of(t - step, p, gt);
        if (t - step < rows) {
#pragma unroll
          for (int k = 0; k < CHUNKS; ++k) {
            Part v;
            load_part(t - step, k, slot_before, v);
            finish(v, t - step, k, x);
          }
        }
      }
      sums_barrier(cluster);
      if (behind && issuer) issue();   // the results' stage may be copied over
      behind = ahead;
      half ^= 1;
    }
    ring_end(ring, issued, stages, a.status);
  } else {
    // In one go: the narrow loads of a loose row, or memory's, are made once.
    Turn turn{0, 0u};
    uint32_t t = first_row + threadIdx.y;
    float gate_next = gate_of(t);
    for (uint32_t t0 = first_row; t0 < rows; t0 += step, t += step) {
      Part v;
      float p[N];
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] = 0.0f;
      const float gt = gate_next;
      gate_next = gate_of(t + step);
      if (BULK) issue_only_after(__all_sync(FULL_MASK, ring_wait(ring, turn, a.status)), issue_t0, rows);
      load_part(t, 0, turn.slot, v);
      add_up(v, 0, p);
      row_sum<N>(p, &sums, half, tpr, cluster, rank);
      if (BULK) {
        turn.next(stages);
        if (tpr == 32 && cluster == 1) __syncthreads();   // else the sums' barrier
        if (issuer) issue();
      }
      const Factors x = factors_of(t, p, gt);
      if (t < rows) finish(v, t, 0, x);
    }
    if (BULK) ring_end(ring, issued, stages, a.status);
  }
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
  auto put = [&](const float (&v)[CHUNKS][COLS], const void* times) {
    if (threadIdx.y == 0)
#pragma unroll
      for (int k = 0; k < CHUNKS; ++k) {
        float m[COLS];
        load_vector<T, VEC>(times, a.vec_f32, c[k], m);
        if (VEC) {
          if (c[k].any()) {
            float4* p = reinterpret_cast<float4*>(part + c[k].first);
            p[0] = make_float4(v[k][0] * m[0], v[k][1] * m[1], v[k][2] * m[2], v[k][3] * m[3]);
            p[1] = make_float4(v[k][4] * m[4], v[k][5] * m[5], v[k][6] * m[6], v[k][7] * m[7]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < COLS; ++j)
            if (c[k].col(j) < c[k].H) part[c[k].col(j)] = v[k][j] * m[j];
        }
      }
    part += a.H;
  };
  if (HAS_F && (post || channel)) {
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k) fold_rows(s1[k]);
    if (post) put(s1, channel ? a.gate : nullptr);
    if (channel) put(s1, a.norm_weight);
  }
  if (NEXT) {
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k) fold_rows(s2[k]);
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

// Shared memory of an SM, of which every block takes 1 KB and its static part.
constexpr size_t SM_SHARED = 228 * 1024, BLOCK_SHARED = 227 * 1024;

// `fixed`: at least the kernel's static shared memory.
template <typename K, typename A>
cudaError_t launch_rows(K kernel, const RowShape& s, int64_t units, size_t smem, size_t fixed, int stages, const A& args,
                        cudaStream_t stream) {
  if (smem > 32 * 1024) {   // with the static part possibly past the default of 48 KB
    // All that a block can have, not this call's size: the attribute is the
    // kernel's, and a call of another thread may come between it and the launch.
    const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(BLOCK_SHARED - fixed));
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

// Stages of a ring of `rounds` rounds with `resident` blocks on an SM, each with
// `fixed` bytes of static shared memory.
int ring_stages(size_t stage, int64_t resident, size_t fixed, int64_t rounds) {
  const size_t block = std::min(SM_SHARED / static_cast<size_t>(resident) - 1024, BLOCK_SHARED);
  const int64_t fit = block > fixed ? static_cast<int64_t>((block - fixed) / stage) : 0;
  return static_cast<int>(std::min<int64_t>(std::min<int64_t>(fit, MAX_STAGES), rounds));
}
// Bytes of a stage: `arrays` times a round's rows of a block's columns.
size_t stage_size(const RowShape& s, int64_t H, int cols, int rows, int64_t arrays, size_t size, bool vec) {
  const uint32_t row = static_cast<uint32_t>(std::min<int64_t>(H, s.tpr * cols) * static_cast<int64_t>(size));
  return static_cast<size_t>(arrays) * staged_rows(row, static_cast<uint32_t>(s.rows * rows), s.cluster, vec);
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
  // One wave: as many blocks as an SM's registers hold, each row after row.
  const int64_t resident = std::max(1, std::min(16, join_threads(sizeof(T), branch, element) / (s.tpr * s.rows)));
  const int64_t most = std::max<int64_t>(1, resident * num_sms / s.cluster);
  const int64_t arrays = 1 + (branch == 2 ? a.top_k : branch) + (element ? 1 : 0);
  constexpr size_t fixed = sizeof(RowSums<2>) + sizeof(Ring) + 256;
  auto rounds_of = [&](int rows, int64_t* units) {
    const int64_t groups = (a.T + s.rows * rows - 1) / (s.rows * rows);
    *units = std::min(groups, most);
    return (groups + *units - 1) / *units;
  };
  int64_t units = 0;
  int stages = 0;
  size_t smem = 0;
  if ((branch != 2 || a.top_k <= 32) && rounds_of(1, &units) > 1) {
    const int rows = join_rows(true, branch);
    const size_t stage = stage_size(s, a.H, COLS, rows, arrays, sizeof(T), vec);
    stages = ring_stages(stage, resident, fixed, rounds_of(rows, &units));
    if (stages < 2) stages = 0;
    smem = stage * stages;
  }
  if (stages == 0) {
    rounds_of(1, &units);
  } else {   // the only waits that may report
    const cudaError_t err = device_status_ptr(&a.status);
    if (err != cudaSuccess) return err;
  }
  return launch_rows(stages > 0 ? (vec ? pick_join<T, true, true>(branch, element)
                                       : pick_join<T, false, true>(branch, element))
                     : vec      ? pick_join<T, true, false>(branch, element)
                                : pick_join<T, false, false>(branch, element),
                     s, units, smem, fixed, stages, a, stream);
}

template <typename T, bool VEC, int CHUNKS, bool BULK>
auto pick_backward(bool has_f, bool next, bool element) {
  if (!has_f) return join_backward_kernel<T, VEC, CHUNKS, BULK, false, true, false>;
  if (next)
    return element ? join_backward_kernel<T, VEC, CHUNKS, BULK, true, true, true>
                   : join_backward_kernel<T, VEC, CHUNKS, BULK, true, true, false>;
  return element ? join_backward_kernel<T, VEC, CHUNKS, BULK, true, false, true>
                 : join_backward_kernel<T, VEC, CHUNKS, BULK, true, false, false>;
}

// Rows that share a block pay for two groups of columns a thread with idle
// lanes: from 1024 columns on.
int backward_chunks(int64_t H) { return H >= 1024 ? 2 : 1; }
// One wave of blocks that keep their column sums in registers: 512 threads of
// them fill an SM (of JOIN_BACKWARD_SMS).
int backward_resident(const RowShape& s) { return std::max(1, MAX_TPR / (s.tpr * s.rows)); }
int64_t backward_units(const RowShape& s, int64_t T, int64_t resident) {
  const int64_t groups = (T + s.rows - 1) / s.rows;
  return std::min<int64_t>(groups, std::max<int64_t>(1, JOIN_BACKWARD_SMS * resident / s.cluster));
}

// *units: the blocks (of clusters) that have left column sums.
template <typename T>
cudaError_t launch_join_backward_t(moe_dtype dtype, JoinBackwardArgs a, int64_t* units, cudaStream_t stream) {
  const bool vec = vec_ok(dtype, a.H, {a.dout, a.dnormed, a.f, a.joined, a.norm_weight, a.next_weight, a.dbranch,
                                       a.dresidual, a.gate_kind == MOE_GATE_TOKEN ? nullptr : a.gate,
                                       a.gate_kind == MOE_GATE_ELEMENT ? a.dgate : nullptr});
  const bool f = a.f != nullptr, next = a.next_weight != nullptr, element = a.gate_kind == MOE_GATE_ELEMENT;
  const int64_t arrays = 1 + (f ? 1 : 0) + (next ? 2 : 0) + (element ? 1 : 0);
  const int chunks = vec ? backward_chunks(a.H) : 1;
  RowShape s = row_shape(a.H, chunks);
  constexpr size_t fixed = sizeof(RowSums<6>) + sizeof(Ring) + 256;
  int stages = 0;
  size_t smem = 0;
  // Short loose rows of 16 bits that L2 holds gain nothing from the ring (16384 x
  // 518, join: 71 us with it, 64 without; 100000 x 385, past L2, norm: 144 and 182).
  constexpr int64_t L2_BYTES = int64_t{128} << 20;
  const bool in_l2 = arrays * a.T * a.H * static_cast<int64_t>(sizeof(T)) < L2_BYTES;
  if (vec || sizeof(T) == 4 || a.H >= 1024 || !in_l2) {
    // Three stages hold the rounds at work and one on its way; rather fewer blocks than fewer stages.
    const size_t stage = stage_size(s, a.H, COLS * chunks, 1, arrays, sizeof(T), vec);
    const int64_t groups = (a.T + s.rows - 1) / s.rows;
    for (int64_t resident = backward_resident(s); resident > 0; resident /= 2) {
      *units = backward_units(s, a.T, resident);
      const int64_t rounds = (groups + *units - 1) / *units;
      stages = rounds < 2 ? 0 : ring_stages(stage, resident, fixed, rounds);
      if (rounds < 2 || stages >= std::min<int64_t>(rounds, 3)) break;
    }
    if (stages < 2) stages = 0;
    smem = stage * stages;
  }
  if (stages == 0) {
    s = row_shape(a.H);
    *units = backward_units(s, a.T, backward_resident(s));
  } else {   // the only waits that may report
    const cudaError_t err = device_status_ptr(&a.status);
    if (err != cudaSuccess) return err;
  }
  smem = std::max(smem, static_cast<size_t>(s.rows - 1) * s.tpr * COLS * sizeof(float));   // the fold in the end
  return launch_rows(stages > 0 ? (!vec          ? pick_backward<T, false, 1, true>(f, next, element)
                                   : chunks == 2 ? pick_backward<T, true, 2, true>(f, next, element)
                                                 : pick_backward<T, true, 1, true>(f, next, element))
                     : vec ? pick_backward<T, true, 1, false>(f, next, element)
                           : pick_backward<T, false, 1, false>(f, next, element),
                     s, *units, smem, fixed, stages, a, stream);
}

}  // namespace

// An upper bound of the units of a backward, whatever its alignment.
int64_t join_backward_units(int64_t T, int64_t H) {
  const RowShape one = row_shape(H), more = row_shape(H, backward_chunks(H));
  return std::max(backward_units(one, T, backward_resident(one)), backward_units(more, T, backward_resident(more)));
}

cudaError_t launch_join(moe_dtype dtype, const JoinArgs& a, int branch, int num_sms, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  switch (dtype) {
    case MOE_F32: return launch_join_t<float>(dtype, a, branch, num_sms, stream);
    case MOE_F16: return launch_join_t<__half>(dtype, a, branch, num_sms, stream);
    default: return launch_join_t<__nv_bfloat16>(dtype, a, branch, num_sms, stream);
  }
}

cudaError_t launch_join_backward(moe_dtype dtype, const JoinBackwardArgs& a, float* dnorm_weight, float* dnext_weight,
                                 cudaStream_t stream) {
  int64_t units = 0;
  cudaError_t err = cudaSuccess;
  if (a.T > 0) {
    switch (dtype) {
      case MOE_F32: err = launch_join_backward_t<float>(dtype, a, &units, stream); break;
      case MOE_F16: err = launch_join_backward_t<__half>(dtype, a, &units, stream); break;
      default: err = launch_join_backward_t<__nv_bfloat16>(dtype, a, &units, stream); break;
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
