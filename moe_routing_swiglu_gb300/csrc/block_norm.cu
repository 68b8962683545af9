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

#include "moe_common.cuh"
#include "moe_internal.h"

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

// Every thread of a row gets the row's N sums. One barrier per call: the two
// halves of `sm` are used in turn, and a half is written again only after the
// barrier of the call between, which every reader of the half has passed.
template <int N>
struct RowSums {
  float v[2][MAX_CLUSTER * MAX_WARPS][N];   // [half][block of the cluster * warps + warp]
};

template <int N>
__device__ __forceinline__ void row_sum(float (&s)[N], RowSums<N>* sm, int& half, int tpr, int cluster, int rank) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s[i] += __shfl_xor_sync(FULL_MASK, s[i], off);
  if (tpr == 32 && cluster == 1) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = tpr >> 5;
  const int row_warp0 = static_cast<int>(threadIdx.y) * warps;   // rows side by side have slots of their own
  if (cluster == 1) {
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) sm->v[half][row_warp0 + warp][i] = s[i];
    __syncthreads();
  } else {
    cg::cluster_group cl = cg::this_cluster();
    if (lane < cluster) {
      float* dst = cl.map_shared_rank(&sm->v[half][rank * warps + warp][0], lane);
#pragma unroll
      for (int i = 0; i < N; ++i) dst[i] = s[i];
    }
    cl.sync();
  }
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = 0.0f;
  for (int w = lane; w < cluster * warps; w += 32)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += sm->v[half][row_warp0 + w][i];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s[i] += __shfl_xor_sync(FULL_MASK, s[i], off);
  half ^= 1;
}

__device__ __forceinline__ float weight_at(const void* p, int dtype, int64_t i) {
  if (dtype == MOE_F32) return static_cast<const float*>(p)[i];
  if (dtype == MOE_F16) return to_f32(static_cast<const __half*>(p)[i]);
  return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
}

// ---------------------------------------------------------------- forward

// BRANCH: 0 none (the norm alone), 1 rows of f, 2 the combine of expert rows.
template <typename T, bool VEC, int BRANCH>
__global__ void __launch_bounds__(MAX_TPR) join_kernel(const JoinArgs a, int cluster) {
  __shared__ RowSums<1> sums;
  const int tpr = blockDim.x;
  const int rank = cluster > 1 ? static_cast<int>(blockIdx.x) % cluster : 0;
  const int64_t unit = blockIdx.x / cluster, units = gridDim.x / cluster;
  const Cols<VEC> c(threadIdx.x, tpr, rank, a.H);
  const float inv_h = 1.0f / static_cast<float>(a.H);
  int half = 0;
  if (cluster > 1) cg::this_cluster().sync();   // every block runs before another one writes to its sums
  grid_dependency_wait();
  launch_dependents();
  float w1[COLS], w2[COLS], gc[COLS];
  if (BRANCH != 0) {
    load_vector<T, VEC>(a.norm_weight, a.vec_f32, c, w1);
    load_vector<T, VEC>(a.gate_kind == MOE_GATE_CHANNEL ? a.gate : nullptr, a.vec_f32, c, gc);
  }
  load_vector<T, VEC>(a.next_weight, a.vec_f32, c, w2);
  // Every thread of a block takes part in every round (the barriers), with a
  // row past the end as a row of zeros that is not stored.
  for (int64_t t0 = unit * blockDim.y; t0 < a.T; t0 += units * blockDim.y) {
    const int64_t t = t0 + threadIdx.y;
    const bool live = t < a.T;
    const int64_t at = (live ? t : t0) * a.H;
    Eight<T> x, gv;
    load8<T, VEC>(static_cast<const T*>(a.x) + at, c, x);
    float f[COLS], g = a.beta;
    if (BRANCH != 0) {
      if (a.gate_kind == MOE_GATE_ELEMENT) load8<T, VEC>(static_cast<const T*>(a.gate) + at, c, gv);
      if (a.gate_kind == MOE_GATE_TOKEN)
        g *= a.vec_f32 ? static_cast<const float*>(a.gate)[live ? t : t0]
                       : to_f32(static_cast<const T*>(a.gate)[live ? t : t0]);
    }
    if (BRANCH == 1) {
      Eight<T> fv;
      load8<T, VEC>(static_cast<const T*>(a.f) + at, c, fv);
#pragma unroll
      for (int j = 0; j < COLS; ++j) f[j] = to_f32(fv.e[j]);
    }
    if (BRANCH == 2) {
      // Slot order, as moe_combine; a bad row number makes the token NaN.
#pragma unroll
      for (int j = 0; j < COLS; ++j) f[j] = 0.0f;
      const int64_t slot0 = (live ? t : t0) * a.top_k;
      bool bad = false;
      constexpr int G = 4;   // rows whose loads are in flight together
      for (int k0 = 0; k0 < a.top_k; k0 += G) {
        Eight<T> v[G];
        float w[G];
#pragma unroll
        for (int i = 0; i < G; ++i) {
          w[i] = 0.0f;
          if (k0 + i < a.top_k) {
            uint32_t r = a.inv[slot0 + k0 + i];
            w[i] = weight_at(a.weights, a.weights_dtype, slot0 + k0 + i);
            if (r >= a.rows) {
              bad = true;
              r = 0;
            }
            load8<T, VEC>(static_cast<const T*>(a.f) + static_cast<int64_t>(r) * a.H, c, v[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < G; ++i)
          if (k0 + i < a.top_k)
#pragma unroll
            for (int j = 0; j < COLS; ++j) f[j] = fmaf(w[i], to_f32(v[i].e[j]), f[j]);
      }
      if (bad)
#pragma unroll
        for (int j = 0; j < COLS; ++j) f[j] = __int_as_float(0x7FC00000);
    }
    if (BRANCH != 0) {
      if (a.norm_weight != nullptr) {
        float s[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < COLS; ++j)
          if (VEC ? c.any() : c.col(j) < c.H) s[0] = fmaf(f[j], f[j], s[0]);
        row_sum<1>(s, &sums, half, tpr, cluster, rank);
        g *= 1.0f / sqrtf(fmaf(s[0], inv_h, a.eps));
      }
#pragma unroll
      for (int j = 0; j < COLS; ++j) {
        float b = f[j] * g * w1[j] * gc[j];
        if (a.gate_kind == MOE_GATE_ELEMENT) b *= to_f32(gv.e[j]);
        x.e[j] = from_f32<T>(fmaf(a.alpha, to_f32(x.e[j]), b));
      }
      if (live) store8<T, VEC>(static_cast<T*>(a.out) + at, c, x);
    }
    if (BRANCH == 0 || a.next_weight != nullptr) {
      float s[1] = {0.0f};
#pragma unroll
      for (int j = 0; j < COLS; ++j)
        if (VEC ? c.any() : c.col(j) < c.H) s[0] = fmaf(to_f32(x.e[j]), to_f32(x.e[j]), s[0]);
      row_sum<1>(s, &sums, half, tpr, cluster, rank);
      const float r = 1.0f / sqrtf(fmaf(s[0], inv_h, a.eps));
#pragma unroll
      for (int j = 0; j < COLS; ++j) x.e[j] = from_f32<T>(to_f32(x.e[j]) * r * w2[j]);
      if (live) store8<T, VEC>(static_cast<T*>(a.y) + at, c, x);
    }
  }
}

// ---------------------------------------------------------------- backward

// HAS_F: the join's branch is there; NEXT: the norm of out is there. Column
// sums go to partial[unit][column array][H], arrays in the order dw1, dgate
// (a channel gate's), dw2, those that are asked for.
template <typename T, bool VEC, bool HAS_F, bool NEXT>
__global__ void __launch_bounds__(MAX_TPR) join_backward_kernel(const JoinBackwardArgs a, int cluster) {
  __shared__ RowSums<6> sums;
  extern __shared__ float fold[];   // [rows of the block - 1][tpr * COLS]
  const int tpr = blockDim.x;
  const int rank = cluster > 1 ? static_cast<int>(blockIdx.x) % cluster : 0;
  const int64_t unit = blockIdx.x / cluster, units = gridDim.x / cluster;
  const Cols<VEC> c(threadIdx.x, tpr, rank, a.H);
  const float inv_h = 1.0f / static_cast<float>(a.H);
  const bool post = HAS_F && a.norm_weight != nullptr;
  const bool token = HAS_F && a.gate_kind == MOE_GATE_TOKEN;
  const bool element = HAS_F && a.gate_kind == MOE_GATE_ELEMENT;
  int half = 0;
  if (cluster > 1) cg::this_cluster().sync();   // every block runs before another one writes to its sums
  grid_dependency_wait();
  launch_dependents();
  float w1[COLS], w2[COLS], gc[COLS];
  float dw1[COLS], dw2[COLS], dgc[COLS];
#pragma unroll
  for (int j = 0; j < COLS; ++j) dw1[j] = dw2[j] = dgc[j] = 0.0f;
  if (HAS_F) {
    load_vector<T, VEC>(a.norm_weight, a.vec_f32, c, w1);
    load_vector<T, VEC>(a.gate_kind == MOE_GATE_CHANNEL ? a.gate : nullptr, a.vec_f32, c, gc);
  }
  if (NEXT) load_vector<T, VEC>(a.next_weight, a.vec_f32, c, w2);
  for (int64_t t0 = unit * blockDim.y; t0 < a.T; t0 += units * blockDim.y) {
    const int64_t t = t0 + threadIdx.y;
    const bool live = t < a.T;
    const int64_t at = (live ? t : t0) * a.H;
    Eight<T> dv, fv, ov, yv, gv;
    const bool has_d = a.dout != nullptr;
    if (has_d) load8<T, VEC>(static_cast<const T*>(a.dout) + at, c, dv);
    if (HAS_F) load8<T, VEC>(static_cast<const T*>(a.f) + at, c, fv);
    if (NEXT) {
      load8<T, VEC>(static_cast<const T*>(a.joined) + at, c, ov);
      load8<T, VEC>(static_cast<const T*>(a.dnormed) + at, c, yv);
    }
    if (element) load8<T, VEC>(static_cast<const T*>(a.gate) + at, c, gv);
    float gt = 1.0f;
    if (token)
      gt = a.vec_f32 ? static_cast<const float*>(a.gate)[live ? t : t0]
                     : to_f32(static_cast<const T*>(a.gate)[live ? t : t0]);
    float s[6] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < COLS; ++j) {
      const float d = has_d ? to_f32(dv.e[j]) : 0.0f;
      if (NEXT) {
        const float o = to_f32(ov.e[j]), wy = w2[j] * to_f32(yv.e[j]);
        s[0] = fmaf(o, o, s[0]);
        s[1] = fmaf(wy, o, s[1]);
        if (HAS_F) {
          const float f = to_f32(fv.e[j]);
          const float gf = w1[j] * gc[j] * (element ? to_f32(gv.e[j]) : 1.0f) * f;
          s[4] = fmaf(wy, gf, s[4]);
          s[5] = fmaf(o, gf, s[5]);
        }
      }
      if (HAS_F) {
        const float f = to_f32(fv.e[j]);
        const float gf = w1[j] * gc[j] * (element ? to_f32(gv.e[j]) : 1.0f) * f;
        s[2] = fmaf(f, f, s[2]);
        s[3] = fmaf(d, gf, s[3]);
      }
    }
    row_sum<6>(s, &sums, half, tpr, cluster, rank);
    const float r2 = NEXT ? 1.0f / sqrtf(fmaf(s[0], inv_h, a.eps)) : 0.0f;
    const float m2 = r2 * r2 * (s[1] * inv_h);                      // r2^2 S2 / H
    const float r1 = post ? 1.0f / sqrtf(fmaf(s[2], inv_h, a.eps)) : 1.0f;
    const float q = s[3] + r2 * (s[4] - m2 * s[5]);
    const float m1 = post ? r1 * r1 * (q * inv_h) : 0.0f;           // r1^2 Q / H
    const float b = a.beta * r1;
    if (token && live && threadIdx.x == 0 && rank == 0) static_cast<float*>(a.dgate)[t] = b * q;
    Eight<T> dx, df, dg;
#pragma unroll
    for (int j = 0; j < COLS; ++j) {
      float dO = has_d ? to_f32(dv.e[j]) : 0.0f;
      if (NEXT) {
        const float o = to_f32(ov.e[j]), y = to_f32(yv.e[j]);
        dO = fmaf(r2, fmaf(-o, m2, w2[j] * y), dO);
        if (live) dw2[j] = fmaf(y, o * r2, dw2[j]);
      }
      dx.e[j] = from_f32<T>(a.alpha * dO);
      if (HAS_F) {
        const float f = to_f32(fv.e[j]);
        const float g = gc[j] * (element ? to_f32(gv.e[j]) : 1.0f);
        const float bd = b * dO;                                    // beta r1 dO
        df.e[j] = from_f32<T>(gt * (fmaf(w1[j] * g, bd, -f * (b * m1))));
        const float bdf = bd * f;
        if (element) dg.e[j] = from_f32<T>(bdf * w1[j]);
        if (live) {
          dw1[j] = fmaf(bdf, g * gt, dw1[j]);
          dgc[j] = fmaf(bdf, w1[j], dgc[j]);
        }
      }
    }
    if (live) {
      store8<T, VEC>(static_cast<T*>(a.dresidual) + at, c, dx);
      if (HAS_F) store8<T, VEC>(static_cast<T*>(a.dbranch) + at, c, df);
      if (element) store8<T, VEC>(static_cast<T*>(a.dgate) + at, c, dg);
    }
  }
  // The block's rows side by side are added in order, then stored.
  float* part = a.partial + unit * a.arrays * static_cast<int64_t>(a.H);
  auto put = [&](float (&v)[COLS]) {
    if (blockDim.y > 1) {
      __syncthreads();
      if (threadIdx.y > 0)
#pragma unroll
        for (int j = 0; j < COLS; ++j) fold[((threadIdx.y - 1) * COLS + j) * tpr + threadIdx.x] = v[j];
      __syncthreads();
    }
    if (threadIdx.y == 0) {
      for (int y = 1; y < static_cast<int>(blockDim.y); ++y)
#pragma unroll
        for (int j = 0; j < COLS; ++j) v[j] += fold[((y - 1) * COLS + j) * tpr + threadIdx.x];
#pragma unroll
      for (int j = 0; j < COLS; ++j)
        if (VEC ? c.any() : c.col(j) < c.H) part[c.col(j)] = v[j];
    }
    part += a.H;
  };
  if (post) put(dw1);
  if (HAS_F && a.gate_kind == MOE_GATE_CHANNEL) put(dgc);
  if (NEXT) put(dw2);
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
  if (i < n)
    for (int u = slice; u < units; u += 8) s += partial[u * n + i];
  sm[slice][x] = s;
  __syncthreads();
  if (slice == 0 && i < n) {
    for (int k = 1; k < 8; ++k) s += sm[k][x];
    float* out = i < H ? out0 : i < 2 * static_cast<int64_t>(H) ? out1 : out2;
    out[i % H] = s;
  }
}

// ---------------------------------------------------------------- launches

template <typename K, typename A>
cudaError_t launch_rows(K kernel, const RowShape& s, int64_t units, size_t smem, const A& args, cudaStream_t stream) {
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
  return cudaLaunchKernelEx(&cfg, kernel, args, s.cluster);
}

bool vec_ok(moe_dtype dtype, int64_t H, std::initializer_list<const void*> ptrs) {
  if (H % COLS != 0) return false;
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
  return true;
}

template <typename T>
cudaError_t launch_join_t(moe_dtype dtype, const JoinArgs& a, int branch, int num_sms, cudaStream_t stream) {
  const RowShape s = row_shape(a.H);
  const bool vec = vec_ok(dtype, a.H, {a.f, a.x, a.out, a.y, a.norm_weight, a.next_weight,
                                       a.gate_kind == MOE_GATE_TOKEN ? nullptr : a.gate});
  const int64_t groups = (a.T + s.rows - 1) / s.rows;
  const int64_t units = std::min<int64_t>(groups, std::max<int64_t>(1, int64_t{8} * num_sms / s.cluster));
  auto pick = [&]() {
    if (branch == 0) return vec ? join_kernel<T, true, 0> : join_kernel<T, false, 0>;
    if (branch == 1) return vec ? join_kernel<T, true, 1> : join_kernel<T, false, 1>;
    return vec ? join_kernel<T, true, 2> : join_kernel<T, false, 2>;
  };
  return launch_rows(pick(), s, units, 0, a, stream);
}

template <typename T>
cudaError_t launch_join_backward_t(moe_dtype dtype, const JoinBackwardArgs& a, int64_t units, cudaStream_t stream) {
  const RowShape s = row_shape(a.H);
  const bool vec = vec_ok(dtype, a.H, {a.dout, a.dnormed, a.f, a.joined, a.norm_weight, a.next_weight, a.dbranch,
                                       a.dresidual, a.gate_kind == MOE_GATE_TOKEN ? nullptr : a.gate,
                                       a.gate_kind == MOE_GATE_ELEMENT ? a.dgate : nullptr});
  const size_t smem = static_cast<size_t>(s.rows - 1) * s.tpr * COLS * sizeof(float);
  const bool next = a.next_weight != nullptr;
  auto pick = [&]() {
    if (a.f == nullptr) return vec ? join_backward_kernel<T, true, false, true> : join_backward_kernel<T, false, false, true>;
    if (next) return vec ? join_backward_kernel<T, true, true, true> : join_backward_kernel<T, false, true, true>;
    return vec ? join_backward_kernel<T, true, true, false> : join_backward_kernel<T, false, true, false>;
  };
  return launch_rows(pick(), s, units, smem, a, stream);
}

}  // namespace

int64_t join_backward_units(int64_t T, int64_t H) {
  const RowShape s = row_shape(H);
  const int64_t groups = (T + s.rows - 1) / s.rows;
  return std::min<int64_t>(groups, std::max<int64_t>(1, JOIN_BACKWARD_BLOCKS / s.cluster));
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
  const int64_t units = join_backward_units(a.T, a.H);
  cudaError_t err = cudaSuccess;
  if (a.T > 0) {
    switch (dtype) {
      case MOE_F32: err = launch_join_backward_t<float>(dtype, a, units, stream); break;
      case MOE_F16: err = launch_join_backward_t<__half>(dtype, a, units, stream); break;
      default: err = launch_join_backward_t<__nv_bfloat16>(dtype, a, units, stream); break;
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
