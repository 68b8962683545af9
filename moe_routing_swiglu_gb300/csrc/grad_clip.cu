// Global L2 norm over many gradient tensors, and clipping by it.
//
//   norm = sqrt(sum over tensors t, elements i of g_t[i]^2)
//   out_t[i] = g_t[i] * c,  c = max_norm / norm if norm is finite and larger
//   than max_norm, else 1
//
// Bound by HBM: the norm reads every element once, the clip reads and writes
// them (a second read: the factor is known only once every element has been
// seen). The tensors are cut into units of 32 KB, one round of 16-byte loads
// of a block; two resident blocks per SM take units blockIdx, blockIdx + grid,
// ... (neighbouring blocks read neighbouring memory, no block is more than a
// unit behind) and issue a unit's loads before they use the one before. The
// clip walks the units backwards: it starts on the bytes that the norm has
// left in L2.
//
// Sums. A thread adds the squares of the 16 (32) elements of a unit that it
// loads in FP32 and carries the units' sums as a compensated pair of FP32 (the
// rounding error of each addition is kept in the second word; one FP64
// addition per unit kept the FP64 units busy for a third of the time: BF16
// norm of 300 MB 65 us, now 48 us = 6.2 TB/s, its clip 96 us = 6.3 TB/s).
// FP32 squares overflow above 1.8e19 and lose bits below 1e-19, so a unit whose
// sum FP32 does not hold (SUM_MIN, SUM_MAX below) and that is not of zeros alone
// is read and added again in FP64: 50M gradients of 1e-17 take 205 us in FP32
// and 257 in BF16, of any ordinary size 48 and 29. Threads and blocks are added
// in FP64. Every sum has a fixed order: block b's units, its threads by a fixed
// tree, the blocks by one last block; the result does not depend on timing.
#include <algorithm>
#include <type_traits>

#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int GC_THREADS = 512;
constexpr int GC_TABLE = 128;          // tensors per launch (the table travels in the kernel's parameters)
constexpr int GC_BLOCKS_PER_SM = 2;
constexpr int GC_MAX_BLOCKS = 1024;    // partial sums per launch
constexpr int GC_GROUP = 4;            // 16-byte loads per thread and round
constexpr int GC_UNIT_VECS = GC_THREADS * GC_GROUP;  // 32 KB

struct GradEntry {
  const void* src;
  void* dst;
  int64_t numel;
  uint32_t first_unit;
  int32_t dtype;
};
struct GradTable {
  GradEntry e[GC_TABLE];
  int n;
  uint32_t units;
};

// The tensor that owns a unit.
__device__ __forceinline__ int find_entry(const GradTable& t, uint32_t unit) {
  int lo = 0, hi = t.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.e[mid].first_unit <= unit) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ uint32_t entry_end(const GradTable& t, int i) {
  return i + 1 < t.n ? t.e[i + 1].first_unit : t.units;
}
__device__ __forceinline__ int elem_size(int dtype) { return dtype == MOE_F32 ? 4 : 2; }

// A tensor as bytes: `head` bytes before src's first 16-byte boundary, then
// `vecs` 16-byte vectors, then less than one vector. Unit u of it holds
// vectors GC_UNIT_VECS u ..; the first unit also the head, the last also the
// tail (fewer than 16 elements in all).
struct Span {
  int head;
  int64_t vecs;
};
__device__ __forceinline__ Span span_of(const GradEntry& e) {
  const int64_t bytes = e.numel * elem_size(e.dtype);
  Span s;
  s.head = static_cast<int>(min((16 - static_cast<int64_t>(reinterpret_cast<uintptr_t>(e.src) % 16)) % 16, bytes));
  s.vecs = (bytes - s.head) / 16;
  return s;
}

// A tensor's units as the table numbers them, and its vectors.
struct Cursor {
  int i;               // entry
  uint32_t first, end; // its units
  const uint4* q;      // its first vector
  int last_vecs;       // vectors of its last unit
  int dtype;
};
__device__ __forceinline__ void set_cursor(const GradTable& t, int i, Cursor& c) {
  const GradEntry& e = t.e[i];
  const Span s = span_of(e);
  c.i = i;
  c.first = e.first_unit;
  c.end = entry_end(t, i);
  c.q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(e.src) + s.head);
  c.last_vecs = static_cast<int>(s.vecs - static_cast<int64_t>(c.end - 1 - c.first) * GC_UNIT_VECS);
  c.dtype = e.dtype;
}

// This thread's vectors of unit u; those past the tensor's end read as zeros.
__device__ __forceinline__ void load_unit(const Cursor& c, uint32_t u, uint4 (&raw)[GC_GROUP]) {
  const uint4* q = c.q + static_cast<int64_t>(u - c.first) * GC_UNIT_VECS + threadIdx.x;
  if (u + 1 < c.end) {
#pragma unroll
    for (int g = 0; g < GC_GROUP; ++g) raw[g] = q[g * GC_THREADS];
  } else {
    const int t = static_cast<int>(threadIdx.x);
#pragma unroll
    for (int g = 0; g < GC_GROUP; ++g)
      raw[g] = t + g * GC_THREADS < c.last_vecs ? q[g * GC_THREADS] : make_uint4(0u, 0u, 0u, 0u);
  }
}

// Elements of unit u outside its vectors: the index of this thread's, or -1.
__device__ __forceinline__ int64_t odd_element(const GradEntry& e, uint32_t u, bool last) {
  const Span s = span_of(e);
  const int es = elem_size(e.dtype);
  const int n_head = u == 0 ? s.head / es : 0;
  const int t = static_cast<int>(threadIdx.x);
  if (t < n_head) return t;
  if (last) {
    const int64_t i = (s.head + s.vecs * 16) / es + (t - n_head);
    if (i < e.numel) return i;
  }
  return -1;
}

// The one or two elements of a 32-bit word (FP32: the second is 0).
template <typename T>
__device__ __forceinline__ float2 word_values(uint32_t w) {
  if (std::is_same<T, float>::value) return make_float2(__uint_as_float(w), 0.0f);
  if (std::is_same<T, __nv_bfloat16>::value)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return make_float2(__half2float(__ushort_as_half(static_cast<unsigned short>(w & 0xFFFFu))),
                     __half2float(__ushort_as_half(static_cast<unsigned short>(w >> 16))));
}

// The running sum: hi + lo in FP32, and what FP32 cannot hold in FP64.
struct Sum {
  float hi, lo;
  double wide;
};

template <typename T>
__device__ __forceinline__ float word_squares(uint32_t w, float s) {
  const float2 v = word_values<T>(w);
  s = fmaf(v.x, v.x, s);
  return std::is_same<T, float>::value ? s : fmaf(v.y, v.y, s);
}

// The squares of this thread's vectors of a unit in FP64, read again from
// memory (rare, and out of line: its registers are not the fast path's).
template <typename T>
__device__ double wide_vecs(const uint4* q, int vecs) {
  double acc = 0.0;
  for (int v = static_cast<int>(threadIdx.x); v < vecs; v += GC_THREADS) {
    const uint4 r = q[v];
    if ((r.x | r.y | r.z | r.w) == 0) continue;
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 v2 = word_values<T>(w[j]);
      acc += static_cast<double>(v2.x) * v2.x + static_cast<double>(v2.y) * v2.y;
    }
  }
  return acc;
}
__device__ __noinline__ double wide_unit(const uint4* q, int vecs, int dtype) {
  if (dtype == MOE_F32) return wide_vecs<float>(q, vecs);
  if (dtype == MOE_F16) return wide_vecs<__half>(q, vecs);
  return wide_vecs<__nv_bfloat16>(q, vecs);
}

// The sums of a thread's squares of a unit that FP32 holds. Each of the at most
// 32 fused multiply-adds whose result is a subnormal is off by at most 2^-150,
// all of them by 2^-145: 2^-45 of a sum of 2^-100, far under the 2^-24 of an
// ordinary rounding (RMS 2.2e-16 in FP32, 1.6e-16 in the 16-bit types). Above,
// 2^80 leaves the running sum room for 2^47 units.
constexpr float SUM_MIN = 0x1p-100f, SUM_MAX = 0x1p80f;

// Adds a unit's squares; false where FP32 does not hold them (nothing added).
template <typename T>
__device__ __forceinline__ bool add_unit(const uint4 (&raw)[GC_GROUP], Sum& acc) {
  float s[GC_GROUP];
#pragma unroll
  for (int g = 0; g < GC_GROUP; ++g)
    s[g] = word_squares<T>(raw[g].w, word_squares<T>(raw[g].z,
                           word_squares<T>(raw[g].y, word_squares<T>(raw[g].x, 0.0f))));
  const float sum = (s[0] + s[1]) + (s[2] + s[3]);
  // Two-sum: t + err is exactly hi + sum.
  const float t = acc.hi + sum;
  const float bb = t - acc.hi;
  const float err = (acc.hi - (t - bb)) + (sum - bb);
  if (!(sum >= SUM_MIN && sum <= SUM_MAX)) return false;
  acc.hi = t;
  acc.lo += err;
  return true;
}

__device__ __forceinline__ double element_of(const GradEntry& e, int64_t i) {
  if (e.dtype == MOE_F32) return static_cast<const float*>(e.src)[i];
  if (e.dtype == MOE_F16) return to_f32(static_cast<const __half*>(e.src)[i]);
  return to_f32(static_cast<const __nv_bfloat16*>(e.src)[i]);
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

// partial[slot0 + b] = block b's sum; with write_norm (a single block) the
// norm itself.
__global__ void __launch_bounds__(GC_THREADS, GC_BLOCKS_PER_SM)
    grad_norm_kernel(const __grid_constant__ GradTable table, double* partial, uint32_t slot0, int write_norm,
                     float* norm) {
  __shared__ double sm[GC_THREADS / 32];
  grid_dependency_wait();
  launch_dependents();
  Sum sum{0.0f, 0.0f, 0.0};
  uint32_t u = blockIdx.x;
  if (u < table.units) {
    Cursor c;
    set_cursor(table, find_entry(table, u), c);
    uint4 cur[GC_GROUP];
    load_unit(c, u, cur);
    while (true) {
      const uint32_t un = u + gridDim.x;
      const int i = c.i, dtype = c.dtype;
      const bool first = u == c.first, last = u + 1 == c.end;
      const int vecs = last ? c.last_vecs : GC_UNIT_VECS;
      const uint4* q = c.q + static_cast<int64_t>(u - c.first) * GC_UNIT_VECS;
      const uint32_t local = u - c.first;
      uint4 next[GC_GROUP];
      if (un < table.units) {
        if (un >= c.end) {
          int in = i + 1;
          while (un >= entry_end(table, in)) ++in;
          set_cursor(table, in, c);
        }
        load_unit(c, un, next);
      }
      const bool fits = dtype == MOE_F32   ? add_unit<float>(cur, sum)
                        : dtype == MOE_F16 ? add_unit<__half>(cur, sum)
                                           : add_unit<__nv_bfloat16>(cur, sum);
      if (!fits) {
        uint32_t any = 0;  // zeros alone (an expert without rows) need no second read
#pragma unroll
        for (int g = 0; g < GC_GROUP; ++g) any |= cur[g].x | cur[g].y | cur[g].z | cur[g].w;
        any &= dtype == MOE_F32 ? 0x7FFFFFFFu : 0x7FFF7FFFu;  // of either sign
        if (any != 0) sum.wide += wide_unit(q, vecs, dtype);
      }
      if (first || last) {
        const int64_t odd = odd_element(table.e[i], local, last);
        if (odd >= 0) {
          const double v = element_of(table.e[i], odd);
          sum.wide += v * v;
        }
      }
      if (un >= table.units) break;
#pragma unroll
      for (int g = 0; g < GC_GROUP; ++g) cur[g] = next[g];
      u = un;
    }
  }
  double acc = sum.wide + (static_cast<double>(sum.hi) + static_cast<double>(sum.lo));
  acc = block_sum(acc, sm);
  if (threadIdx.x == 0) {
    if (write_norm) *norm = static_cast<float>(sqrt(acc));
    else partial[slot0 + blockIdx.x] = acc;
  }
}

// One block: the norm from all partial sums.
__global__ void __launch_bounds__(GC_THREADS)
    grad_norm_finish_kernel(const double* partial, uint32_t n_partial, float* norm) {
  __shared__ double sm[GC_THREADS / 32];
  grid_dependency_wait();
  launch_dependents();
  double total = 0.0;
  for (uint32_t i = threadIdx.x; i < n_partial; i += GC_THREADS) total += partial[i];
  total = block_sum(total, sm);
  if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(total));
}

template <typename T>
__device__ __forceinline__ uint32_t scale_word(uint32_t w, float f) {
  const float2 v = word_values<T>(w);
  if constexpr (std::is_same<T, float>::value) return __float_as_uint(v.x * f);
  else return pack2<T>(v.x * f, v.y * f);
}
template <typename T>
__device__ __forceinline__ uint4 scale_vec(uint4 r, float f) {
  return make_uint4(scale_word<T>(r.x, f), scale_word<T>(r.y, f), scale_word<T>(r.z, f), scale_word<T>(r.w, f));
}

// Writes this thread's vectors of unit u (local: within its tensor), scaled; a
// factor of 1 copies the words (a product and a conversion would make one NaN
// of them all).
// dst on src's 16-byte phase takes 16-byte stores, on another one the vector's
// elements one by one.
template <typename T>
__device__ __forceinline__ void store_unit(const GradEntry& e, uint32_t local, int vecs, bool last, float f,
                                           const uint4 (&raw)[GC_GROUP]) {
  const int head = span_of(e).head;
  T* d = reinterpret_cast<T*>(static_cast<uint8_t*>(e.dst) + head);
  constexpr int V = 16 / static_cast<int>(sizeof(T));
  d += static_cast<int64_t>(local) * GC_UNIT_VECS * V;
  const bool aligned = reinterpret_cast<uintptr_t>(d) % 16 == 0;
#pragma unroll
  for (int g = 0; g < GC_GROUP; ++g) {
    const int v = static_cast<int>(threadIdx.x) + g * GC_THREADS;
    if (v >= vecs) continue;
    const uint4 o = f == 1.0f ? raw[g] : scale_vec<T>(raw[g], f);
    if (aligned) {
      reinterpret_cast<uint4*>(d)[v] = o;
    } else {
      const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if constexpr (V == 4) {
          d[v * V + j] = __uint_as_float(w[j]);
        } else {
          const uint16_t bits = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
          reinterpret_cast<uint16_t*>(d)[v * V + j] = bits;
        }
      }
    }
  }
  if (last || local == 0) {
    const int64_t odd = odd_element(e, local, last);
    if (odd >= 0) {
      const T v = static_cast<const T*>(e.src)[odd];
      static_cast<T*>(e.dst)[odd] = f == 1.0f ? v : from_f32<T>(to_f32(v) * f);
    }
  }
}

// A factor of 1 copies the bits, and leaves tensors that are clipped in place
// untouched.
__global__ void __launch_bounds__(GC_THREADS, GC_BLOCKS_PER_SM)
    grad_clip_kernel(const __grid_constant__ GradTable table, const float* __restrict__ norm, float max_norm) {
  grid_dependency_wait();
  launch_dependents();
  const float n = *norm;
  const float f = (n > max_norm && n <= 3.402823466e38f) ? max_norm / n : 1.0f;
  const uint32_t n_units = table.units;
  uint32_t k = blockIdx.x;  // the block's unit is n_units - 1 - k
  if (k >= n_units) return;
  Cursor c;
  set_cursor(table, find_entry(table, n_units - 1 - k), c);
  // In place with a factor of 1 nothing is read or written.
  bool idle = f == 1.0f && table.e[c.i].dst == table.e[c.i].src;
  uint4 cur[GC_GROUP];
  if (!idle) load_unit(c, n_units - 1 - k, cur);
  while (true) {
    const uint32_t u = n_units - 1 - k, kn = k + gridDim.x;
    const int i = c.i, dtype = c.dtype;
    const bool last = u + 1 == c.end, skip = idle;
    const int vecs = last ? c.last_vecs : GC_UNIT_VECS;
    const uint32_t local = u - c.first;
    uint4 next[GC_GROUP];
    if (kn < n_units) {
      const uint32_t un = n_units - 1 - kn;
      if (un < c.first) {
        int in = i - 1;
        while (un < table.e[in].first_unit) --in;
        set_cursor(table, in, c);
        idle = f == 1.0f && table.e[in].dst == table.e[in].src;
      }
      if (!idle) load_unit(c, un, next);
    }
    if (!skip) {
      if (dtype == MOE_F32) store_unit<float>(table.e[i], local, vecs, last, f, cur);
      else if (dtype == MOE_F16) store_unit<__half>(table.e[i], local, vecs, last, f, cur);
      else store_unit<__nv_bfloat16>(table.e[i], local, vecs, last, f, cur);
    }
    if (kn >= n_units) break;
#pragma unroll
    for (int g = 0; g < GC_GROUP; ++g) cur[g] = next[g];
    k = kn;
  }
}

// Units of a tensor: by its 16-byte vectors, at least one.
int64_t units_of(const moe_grad_tensor& t) {
  const int64_t bytes = t.numel * static_cast<int64_t>(dtype_size(static_cast<moe_dtype>(t.dtype)));
  const int64_t mis = static_cast<int64_t>(reinterpret_cast<uintptr_t>(t.src) % 16);
  const int64_t head = std::min<int64_t>((16 - mis) % 16, bytes);
  const int64_t vecs = (bytes - head) / 16;
  return std::max<int64_t>(1, (vecs + GC_UNIT_VECS - 1) / GC_UNIT_VECS);
}

// The next launch's table: tensors i .. (empty ones left out). Returns the
// first tensor after it.
int64_t fill_table(const moe_grad_tensor* t, int64_t n, int64_t i, GradTable* table) {
  table->n = 0;
  int64_t units = 0;
  while (i < n && table->n < GC_TABLE) {
    if (t[i].numel > 0) {
      const int64_t c = units_of(t[i]);
      if (units > 0 && units + c > 0x7FFFFFFF) break;
      table->e[table->n++] = GradEntry{t[i].src, t[i].dst, t[i].numel, static_cast<uint32_t>(units), t[i].dtype};
      units += c;
    }
    ++i;
  }
  table->units = static_cast<uint32_t>(units);
  return i;
}

int grid_blocks(uint32_t units, int num_sms) {
  const int64_t want = std::min<int64_t>(static_cast<int64_t>(num_sms) * GC_BLOCKS_PER_SM, GC_MAX_BLOCKS);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(units, want)));
}

}  // namespace

// GC_MAX_BLOCKS partial sums for each possible launch (a table may also end
// early on its unit count: one more launch per 2^31 units, 64 TB).
size_t grad_norm_scratch_bytes(int64_t n) {
  const int64_t launches = std::max<int64_t>(1, (n + GC_TABLE - 1) / GC_TABLE);
  return static_cast<size_t>(launches) * GC_MAX_BLOCKS * 8;
}

cudaError_t launch_grad_norm(const moe_grad_tensor* tensors, int64_t n, float* norm, void* scratch, int num_sms,
                             cudaStream_t stream) {
  double* partial = static_cast<double*>(scratch);
  uint32_t slot = 0;
  int64_t i = 0;
  do {
    GradTable table;
    i = fill_table(tensors, n, i, &table);
    const int grid = grid_blocks(table.units, num_sms);
    const int write_norm = i >= n && slot == 0 && grid == 1 ? 1 : 0;
    cudaError_t err = launch_dependent(grad_norm_kernel, dim3(grid), dim3(GC_THREADS), 0, stream, table, partial, slot,
                                       write_norm, norm);
    if (err != cudaSuccess || write_norm != 0) return err;
    slot += static_cast<uint32_t>(grid);
  } while (i < n);
  return launch_dependent(grad_norm_finish_kernel, dim3(1), dim3(GC_THREADS), 0, stream, partial, slot, norm);
}

cudaError_t launch_grad_clip(const moe_grad_tensor* tensors, int64_t n, const float* norm, float max_norm, int num_sms,
                             cudaStream_t stream) {
  // The launches in reverse order too.
  for (int64_t hi = n; hi > 0;) {
    const int64_t lo = (hi - 1) / GC_TABLE * GC_TABLE;
    for (int64_t i = lo; i < hi;) {
      GradTable table;
      i = fill_table(tensors, hi, i, &table);
      if (table.units == 0) continue;
      const int grid = grid_blocks(table.units, num_sms);
      cudaError_t err = launch_dependent(grad_clip_kernel, dim3(grid), dim3(GC_THREADS), 0, stream, table, norm,
                                         max_norm);
      if (err != cudaSuccess) return err;
    }
    hi = lo;
  }
  return cudaSuccess;
}

}  // namespace moe
