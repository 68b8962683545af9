// Global L2 norm over many gradient tensors, and clipping by it.
//
//   norm = sqrt(sum over tensors t, elements i of g_t[i]^2)
//   out_t[i] = g_t[i] * c,  c = max_norm / norm if norm is finite and larger
//   than max_norm, else 1
//
// Bound by HBM: the norm reads every element once, the clip reads and writes
// them (a second read: the factor is known only once every element has been
// seen). Both kernels cut the tensors into chunks of 32 KB; a persistent grid
// takes chunks blockIdx, blockIdx + grid, ... of the norm in order and of the
// clip in reverse, so that the clip starts on the bytes the norm left in L2.
//
// Sums. A thread adds the squares of the 16 (32) elements that it loads at a
// time in FP32 and carries the totals in FP64 (one FP64 addition per 16
// elements; FP64 throughout would be bound by the FP64 units). FP32 squares
// overflow above 1.8e19 and lose bits below 1e-19, so a group whose FP32 sum
// is above 2^100 or below 2^-60 and not of zeros alone is added again from its
// registers in FP64. Every sum has a fixed order: block b's chunks, its
// threads by a fixed tree, the blocks in order by the last block to finish;
// the result does not depend on timing.
#include <algorithm>

#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int GC_THREADS = 512;
constexpr int GC_CHUNK_BYTES = 32 * 1024;  // one round of GC_GROUP loads per thread
constexpr int GC_TABLE = 128;          // tensors per launch (the table travels in the kernel's parameters)
constexpr int GC_MAX_BLOCKS = 1024;    // partial sums per launch
constexpr int GC_GROUP = 4;            // 16-byte loads in flight per thread

struct GradEntry {
  const void* src;
  void* dst;
  int64_t numel;
  uint32_t first_chunk;
  int32_t dtype;
};
struct GradTable {
  GradEntry e[GC_TABLE];
  int n;
  uint32_t chunks;
};

// The tensor that owns a chunk.
__device__ __forceinline__ int find_entry(const GradTable& t, uint32_t chunk) {
  int lo = 0, hi = t.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.e[mid].first_chunk <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

// Elements of a chunk: [begin, end) of the tensor. Chunks start on 16-byte
// boundaries of src: the first also holds the elements before the first
// boundary (head), the last whatever is left.
struct ChunkRange {
  int64_t begin, vec, vec_end, end;  // scalar [begin, vec), 16-byte vectors [vec, vec_end), scalar [vec_end, end)
};
template <typename T>
__device__ __forceinline__ ChunkRange chunk_range(const GradEntry& e, uint32_t c) {
  constexpr int64_t PER = GC_CHUNK_BYTES / static_cast<int64_t>(sizeof(T));
  constexpr int64_t V = 16 / static_cast<int64_t>(sizeof(T));
  const int64_t mis = static_cast<int64_t>(reinterpret_cast<uintptr_t>(e.src) % 16 / sizeof(T));
  const int64_t head = min(mis == 0 ? int64_t{0} : V - mis, e.numel);
  ChunkRange r;
  r.vec = head + static_cast<int64_t>(c) * PER;
  r.begin = c == 0 ? 0 : r.vec;
  r.end = min(r.vec + PER, e.numel);
  r.vec_end = r.vec + (r.end - r.vec) / V * V;
  return r;
}

template <typename T>
__device__ __forceinline__ double chunk_sum(const GradEntry& e, uint32_t c) {
  const T* p = static_cast<const T*>(e.src);
  const ChunkRange r = chunk_range<T>(e, c);
  constexpr int V = 16 / static_cast<int>(sizeof(T));
  double acc = 0.0;
  for (int64_t i = r.begin + threadIdx.x; i < r.vec; i += GC_THREADS) {
    const double v = to_f32(p[i]);
    acc += v * v;
  }
  for (int64_t i = r.vec_end + threadIdx.x; i < r.end; i += GC_THREADS) {
    const double v = to_f32(p[i]);
    acc += v * v;
  }
  const int64_t n_vec = (r.vec_end - r.vec) / V;
  const uint4* q = reinterpret_cast<const uint4*>(p + r.vec);
  for (int64_t i0 = threadIdx.x; i0 < n_vec; i0 += GC_THREADS * GC_GROUP) {
    uint4 raw[GC_GROUP];
#pragma unroll
    for (int g = 0; g < GC_GROUP; ++g) {
      const int64_t i = i0 + static_cast<int64_t>(g) * GC_THREADS;
      raw[g] = i < n_vec ? q[i] : make_uint4(0u, 0u, 0u, 0u);
    }
    float s[GC_GROUP];
#pragma unroll
    for (int g = 0; g < GC_GROUP; ++g) {
      const T* x = reinterpret_cast<const T*>(&raw[g]);
      s[g] = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) s[g] = fmaf(to_f32(x[j]), to_f32(x[j]), s[g]);
    }
    const float sum = (s[0] + s[1]) + (s[2] + s[3]);
    if (sum >= 0x1p-60f && sum <= 0x1p100f) {
      acc += static_cast<double>(sum);
    } else {
      uint32_t any = 0;
#pragma unroll
      for (int g = 0; g < GC_GROUP; ++g) any |= raw[g].x | raw[g].y | raw[g].z | raw[g].w;
      // Signs alone (-0) take the slow path too; it adds their zeros.
      if (any != 0) {
#pragma unroll
        for (int g = 0; g < GC_GROUP; ++g) {
          const T* x = reinterpret_cast<const T*>(&raw[g]);
          for (int j = 0; j < V; ++j) {
            const double v = to_f32(x[j]);
            acc += v * v;
          }
        }
      }
    }
  }
  return acc;
}

__device__ __forceinline__ double block_sum(double v, double* sm) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(FULL_MASK, v, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = threadIdx.x < GC_THREADS / 32 ? sm[threadIdx.x] : 0.0;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(FULL_MASK, v, off);
  }
  return v;  // valid in warp 0
}

// partial[slot0 + b] = block b's sum. The launch with write_norm set also writes
// the norm: its last block to finish adds all n_partial sums in order.
__global__ void __launch_bounds__(GC_THREADS)
    grad_norm_kernel(const __grid_constant__ GradTable table, double* partial, uint32_t slot0, uint32_t n_partial,
                     uint32_t* ticket, int write_norm, float* norm) {
  __shared__ double sm[GC_THREADS / 32];
  __shared__ bool last;
  grid_dependency_wait();
  launch_dependents();
  double acc = 0.0;
  for (uint32_t c = blockIdx.x; c < table.chunks; c += gridDim.x) {
    const GradEntry& e = table.e[find_entry(table, c)];
    const uint32_t local = c - e.first_chunk;
    if (e.dtype == MOE_F32) acc += chunk_sum<float>(e, local);
    else if (e.dtype == MOE_F16) acc += chunk_sum<__half>(e, local);
    else acc += chunk_sum<__nv_bfloat16>(e, local);
  }
  acc = block_sum(acc, sm);
  if (threadIdx.x == 0) {
    partial[slot0 + blockIdx.x] = acc;
    last = false;
    if (write_norm) last = counter_acq_rel_add(ticket) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double total = 0.0;
  for (uint32_t i = threadIdx.x; i < n_partial; i += GC_THREADS) total += __ldcg(partial + i);
  total = block_sum(total, sm);
  if (threadIdx.x == 0) {
    *norm = static_cast<float>(sqrt(total));
    *ticket = 0;  // ready for the next call on this workspace
  }
}

template <typename T>
__device__ __forceinline__ void chunk_clip(const GradEntry& e, uint32_t c, float f) {
  const T* p = static_cast<const T*>(e.src);
  T* d = static_cast<T*>(e.dst);
  const ChunkRange r = chunk_range<T>(e, c);
  constexpr int V = 16 / static_cast<int>(sizeof(T));
  const bool vec = reinterpret_cast<uintptr_t>(e.src) % 16 == reinterpret_cast<uintptr_t>(e.dst) % 16;
  const int64_t v0 = vec ? r.vec : r.end;          // src and dst on different boundaries: all scalar
  const int64_t v1 = vec ? r.vec_end : r.end;
  for (int64_t i = r.begin + threadIdx.x; i < v0; i += GC_THREADS) d[i] = from_f32<T>(to_f32(p[i]) * f);
  for (int64_t i = v1 + threadIdx.x; i < r.end; i += GC_THREADS) d[i] = from_f32<T>(to_f32(p[i]) * f);
  if (!vec) return;
  const int64_t n_vec = (r.vec_end - r.vec) / V;
  const uint4* q = reinterpret_cast<const uint4*>(p + r.vec);
  uint4* o = reinterpret_cast<uint4*>(d + r.vec);
  for (int64_t i0 = threadIdx.x; i0 < n_vec; i0 += GC_THREADS * GC_GROUP) {
    uint4 raw[GC_GROUP];
#pragma unroll
    for (int g = 0; g < GC_GROUP; ++g) {
      const int64_t i = i0 + static_cast<int64_t>(g) * GC_THREADS;
      if (i < n_vec) raw[g] = q[i];
    }
#pragma unroll
    for (int g = 0; g < GC_GROUP; ++g) {
      const int64_t i = i0 + static_cast<int64_t>(g) * GC_THREADS;
      if (i < n_vec) {
        T* x = reinterpret_cast<T*>(&raw[g]);
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = from_f32<T>(to_f32(x[j]) * f);
        o[i] = raw[g];
      }
    }
  }
}

// Chunks in reverse order (see the file's comment). A factor of 1 copies the
// bits, and leaves tensors that are clipped in place untouched.
__global__ void __launch_bounds__(GC_THREADS)
    grad_clip_kernel(const __grid_constant__ GradTable table, const float* __restrict__ norm, float max_norm) {
  grid_dependency_wait();
  launch_dependents();
  const float n = *norm;
  const float f = (n > max_norm && n <= 3.402823466e38f) ? max_norm / n : 1.0f;
  for (uint32_t i = blockIdx.x; i < table.chunks; i += gridDim.x) {
    const uint32_t c = table.chunks - 1 - i;
    const GradEntry& e = table.e[find_entry(table, c)];
    if (f == 1.0f && e.dst == e.src) continue;
    const uint32_t local = c - e.first_chunk;
    if (e.dtype == MOE_F32) chunk_clip<float>(e, local, f);
    else if (e.dtype == MOE_F16) chunk_clip<__half>(e, local, f);
    else chunk_clip<__nv_bfloat16>(e, local, f);
  }
}

// Chunks of a tensor (at least one, so that a head without vectors is seen).
int64_t chunks_of(const moe_grad_tensor& t) {
  const int64_t bytes = t.numel * static_cast<int64_t>(dtype_size(static_cast<moe_dtype>(t.dtype)));
  return std::max<int64_t>(1, (bytes + GC_CHUNK_BYTES - 1) / GC_CHUNK_BYTES);
}

// The next launch's table: tensors i.. (empty ones left out). Returns the
// first tensor after it.
int64_t fill_table(const moe_grad_tensor* t, int64_t n, int64_t i, GradTable* table) {
  table->n = 0;
  int64_t chunks = 0;
  while (i < n && table->n < GC_TABLE) {
    if (t[i].numel > 0) {
      const int64_t c = chunks_of(t[i]);
      if (chunks > 0 && chunks + c > 0x7FFFFFFF) break;
      table->e[table->n++] = GradEntry{t[i].src, t[i].dst, t[i].numel, static_cast<uint32_t>(chunks), t[i].dtype};
      chunks += c;
    }
    ++i;
  }
  table->chunks = static_cast<uint32_t>(chunks);
  return i;
}

int grid_blocks(uint32_t chunks, int num_sms) {
  const int64_t want = std::min<int64_t>(static_cast<int64_t>(num_sms) * 4, GC_MAX_BLOCKS);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(chunks, want)));
}

}  // namespace

// The ticket, then GC_MAX_BLOCKS partial sums for each possible launch (a
// table may also end early on its chunk count: one more launch per 2^31
// chunks, 64 TB).
size_t grad_norm_scratch_bytes(int64_t n) {
  const int64_t launches = std::max<int64_t>(1, (n + GC_TABLE - 1) / GC_TABLE);
  return 256 + static_cast<size_t>(launches) * GC_MAX_BLOCKS * 8;
}

cudaError_t launch_grad_norm(const moe_grad_tensor* tensors, int64_t n, float* norm, void* scratch, int num_sms,
                             cudaStream_t stream) {
  uint32_t* ticket = static_cast<uint32_t*>(scratch);
  double* partial = reinterpret_cast<double*>(static_cast<uint8_t*>(scratch) + 256);
  cudaError_t err = cudaMemsetAsync(ticket, 0, 4, stream);
  if (err != cudaSuccess) return err;
  uint32_t slot = 0;
  int64_t i = 0;
  do {
    GradTable table;
    i = fill_table(tensors, n, i, &table);
    const int grid = grid_blocks(table.chunks, num_sms);
    const int write_norm = i >= n ? 1 : 0;
    err = launch_dependent(grad_norm_kernel, dim3(grid), dim3(GC_THREADS), 0, stream, table, partial, slot,
                           slot + static_cast<uint32_t>(grid), ticket, write_norm, norm);
    if (err != cudaSuccess) return err;
    slot += static_cast<uint32_t>(grid);
  } while (i < n);
  return cudaSuccess;
}

cudaError_t launch_grad_clip(const moe_grad_tensor* tensors, int64_t n, const float* norm, float max_norm, int num_sms,
                             cudaStream_t stream) {
  // The launches in reverse order too.
  for (int64_t hi = n; hi > 0;) {
    const int64_t lo = (hi - 1) / GC_TABLE * GC_TABLE;
    for (int64_t i = lo; i < hi;) {
      GradTable table;
      i = fill_table(tensors, hi, i, &table);
      if (table.chunks == 0) continue;
      const int grid = grid_blocks(table.chunks, num_sms);
      cudaError_t err = launch_dependent(grad_clip_kernel, dim3(grid), dim3(GC_THREADS), 0, stream, table, norm,
                                         max_norm);
      if (err != cudaSuccess) return err;
    }
    hi = lo;
  }
  return cudaSuccess;
}

}  // namespace moe
