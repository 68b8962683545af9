// MXFP4 quantisation and its inverse (the format and its rounding are in
// mxfp4.cuh), and the one-time layout of the expert weights' scales for the
// tensor cores.
#include "moe_common.cuh"
#include "moe_internal.h"
#include "mxfp4.cuh"

namespace moe {
namespace {

constexpr int MXQ_THREADS = 256;
constexpr int MXQ_UNROLL = 4;                           // 8-element units per thread and step
constexpr int MXQ_WARP_UNITS = 32 * MXQ_UNROLL;

// Eight consecutive elements as FP32, and the largest |x| bits among them.
template <typename T> struct Load8;
template <> struct Load8<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const uint4*>(p);
    b = *reinterpret_cast<const uint4*>(p + 4);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
  }
};
template <typename T> struct Load8 {
  uint4 a;
  __device__ __forceinline__ void load(const T* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const T* e = reinterpret_cast<const T*>(&a);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
  }
};

struct QuantArgs {
  const void* x;
  uint32_t rows;
  uint32_t upr;        // 8-element units per row, K / 8
  uint32_t upr_magic;  // ceil(2^32 / upr)
  uint32_t units;      // rows * upr
  const uint32_t* inv; // [rows * top_k] output row of each slot, or NULL (row r -> row r)
  int top_k;
  uint32_t rows_out;   // rows * top_k: entries of inv at or past it are skipped
  uint8_t* codes;      // [rows_out, K / 2]
  uint8_t* scales;     // [rows_out, pitch]
  int pitch;
};

// One thread quantises 8 elements, four lanes share a block: 16 (or 32)
// bytes in, 4 bytes of codes out, coalesced over the warp; the block's
// largest magnitude is exchanged by two shuffles. Row by row the units are
// contiguous, so a warp takes 128 consecutive units whatever K is. With inv
// each row's codes go to its top_k dispatched rows: x is read once and no
// dispatched copy of it in its own type is ever written.
template <typename T>
__global__ void __launch_bounds__(MXQ_THREADS) mx_quantize_kernel(const QuantArgs a) {
  grid_dependency_wait();
  launch_dependents();
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t warp = (blockIdx.x * MXQ_THREADS + threadIdx.x) >> 5;
  const uint32_t n_warps = gridDim.x * (MXQ_THREADS / 32);
  const T* __restrict__ x = static_cast<const T*>(a.x);
  const uint32_t n_seg = (a.units + MXQ_WARP_UNITS - 1) / MXQ_WARP_UNITS;
  const int64_t code_pitch = static_cast<int64_t>(a.upr) * 4;
  for (uint32_t seg = warp; seg < n_seg; seg += n_warps) {
    const uint32_t u0 = seg * MXQ_WARP_UNITS;
    Load8<T> in[MXQ_UNROLL];
#pragma unroll
    for (int i = 0; i < MXQ_UNROLL; ++i) {
      const uint32_t u = u0 + i * 32 + lane;
      if (u < a.units) in[i].load(x + static_cast<int64_t>(u) * 8);
    }
    const uint32_t row0 = u0 / a.upr;
    const uint32_t rem0 = u0 - row0 * a.upr;
#pragma unroll
    for (int i = 0; i < MXQ_UNROLL; ++i) {
      const uint32_t off = i * 32 + lane;
      const bool live = u0 + off < a.units;  // units is a multiple of 4: a block is all in or all out
      float v[8];
      uint32_t amax = 0;
      if (live) {
        in[i].get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7FFFFFFFu);
      }
      amax = max(amax, __shfl_xor_sync(FULL_MASK, amax, 1));
      amax = max(amax, __shfl_xor_sync(FULL_MASK, amax, 2));
      if (!live) continue;
      const uint32_t byte = mx_scale_byte(amax);
      const float s = mx_inv_scale(byte);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= s;
      const uint32_t codes = byte == 255u ? 0u : mx_pack8(v);
      const uint32_t local = rem0 + off;                      // < upr + 128
      const uint32_t dr = __umulhi(local, a.upr_magic);       // local / upr
      const uint32_t row = row0 + dr;
      const uint32_t unit = local - dr * a.upr;
      const uint32_t blk = unit >> 2;
      const bool head = (unit & 3u) == 0;
      const bool last = unit + 4 >= a.upr;                    // the row's last block also clears the row's pad bytes
      auto store = [&](uint32_t r) {
        *reinterpret_cast<uint32_t*>(a.codes + static_cast<int64_t>(r) * code_pitch + unit * 4) = codes;
        if (head) {
          uint8_t* sp = a.scales + static_cast<int64_t>(r) * a.pitch;
          sp[blk] = static_cast<uint8_t>(byte);
          if (last)
            for (int p = static_cast<int>(blk) + 1; p < a.pitch; ++p) sp[p] = 0;
        }
      };
      if (a.inv == nullptr) {
        store(row);
      } else {
        for (int j = 0; j < a.top_k; ++j) {
          const uint32_t r = a.inv[static_cast<int64_t>(row) * a.top_k + j];
          if (r < a.rows_out) store(r);
        }
      }
    }
  }
}

struct DequantArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  uint32_t upr;
  uint32_t upr_magic;
  uint32_t units;
  int pitch;
  void* out;
};

// One thread: 4 bytes of codes -> 8 values (one 16-byte store, two for FP32).
template <typename T>
__global__ void __launch_bounds__(MXQ_THREADS) mx_dequantize_kernel(const DequantArgs a) {
  grid_dependency_wait();
  launch_dependents();
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t warp = (blockIdx.x * MXQ_THREADS + threadIdx.x) >> 5;
  const uint32_t n_warps = gridDim.x * (MXQ_THREADS / 32);
  const uint32_t n_seg = (a.units + MXQ_WARP_UNITS - 1) / MXQ_WARP_UNITS;
  for (uint32_t seg = warp; seg < n_seg; seg += n_warps) {
    const uint32_t u0 = seg * MXQ_WARP_UNITS;
    const uint32_t row0 = u0 / a.upr;
    const uint32_t rem0 = u0 - row0 * a.upr;
    uint32_t c[MXQ_UNROLL], sb[MXQ_UNROLL];
#pragma unroll
    for (int i = 0; i < MXQ_UNROLL; ++i) {
      const uint32_t off = i * 32 + lane;
      if (u0 + off < a.units) {
        const uint32_t local = rem0 + off;
        const uint32_t dr = __umulhi(local, a.upr_magic);
        const uint32_t unit = local - dr * a.upr;
        c[i] = *reinterpret_cast<const uint32_t*>(a.codes + static_cast<int64_t>(u0 + off) * 4);
        sb[i] = a.scales[static_cast<int64_t>(row0 + dr) * a.pitch + (unit >> 2)];
      }
    }
#pragma unroll
    for (int i = 0; i < MXQ_UNROLL; ++i) {
      const uint32_t u = u0 + i * 32 + lane;
      if (u >= a.units) continue;
      uint32_t h[4];
      mx_unpack8(c[i], h);
      const float s = mx_scale(sb[i]);
      T o[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
        o[2 * j] = from_f32<T>(f.x * s);
        o[2 * j + 1] = from_f32<T>(f.y * s);
      }
      T* dst = static_cast<T*>(a.out) + static_cast<int64_t>(u) * 8;
      constexpr int VEC = static_cast<int>(sizeof(T) * 8 / 16);
#pragma unroll
      for (int q = 0; q < VEC; ++q) reinterpret_cast<uint4*>(dst)[q] = reinterpret_cast<const uint4*>(o)[q];
    }
  }
}

// Row-major scales [E, R, pitch] -> the tensor cores' order: for each expert,
// 128-row block and 256-element K block two atoms of 512 bytes, atom a
// holding the four scale bytes of K elements 128 a .. 128 a + 127 of row m at
// byte (m % 32) * 16 + (m / 32) * 4. Rows and blocks past the matrix get 0.
__global__ void mx_layout_scales_kernel(const uint8_t* __restrict__ src, uint32_t* __restrict__ dst, int64_t R,
                                        int64_t row_blocks, int64_t k_blocks, int64_t pitch, int64_t blocks_per_row,
                                        int64_t n_words) {
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; w < n_words;
       w += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int in = static_cast<int>(w & 127);          // word of the atom
    const int64_t atom = w >> 7;
    const int64_t kw = atom % (2 * k_blocks);          // which 128 K elements
    const int64_t rb = atom / (2 * k_blocks) % row_blocks;
    const int64_t e = atom / (2 * k_blocks * row_blocks);
    const int64_t m = rb * 128 + (in & 3) * 32 + (in >> 2);
    uint32_t v = 0;
    if (m < R) {
      const uint8_t* p = src + (e * R + m) * pitch;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (kw * 4 + b < blocks_per_row) v |= static_cast<uint32_t>(p[kw * 4 + b]) << (8 * b);
    }
    dst[w] = v;
  }
}

// Rows per launch so that the unit count stays below 2^31.
int64_t rows_per_launch(int64_t K) { return ((int64_t{1} << 31) - MXQ_WARP_UNITS) / (K / 8); }

int grid_for(uint32_t units, int num_sms) {
  const int64_t want = (static_cast<int64_t>(units) + MXQ_WARP_UNITS * (MXQ_THREADS / 32) - 1) /
                       (MXQ_WARP_UNITS * (MXQ_THREADS / 32));
  const int64_t cap = static_cast<int64_t>(num_sms) * 8;
  return static_cast<int>(want < cap ? want : cap);
}

uint32_t magic_for(uint32_t upr) { return static_cast<uint32_t>(((uint64_t{1} << 32) + upr - 1) / upr); }

}  // namespace

cudaError_t launch_mx_quantize(const void* x, moe_dtype dtype, int64_t rows, int64_t K, const uint32_t* inv, int top_k,
                               void* codes, void* scales, int num_sms, cudaStream_t stream) {
  const uint32_t upr = static_cast<uint32_t>(K / 8);
  const int64_t step = rows_per_launch(K);
  const int64_t pitch = mx_scale_pitch(K);
  for (int64_t r0 = 0; r0 < rows; r0 += step) {
    const int64_t n = rows - r0 < step ? rows - r0 : step;
    QuantArgs a{};
    a.x = static_cast<const uint8_t*>(x) + r0 * K * static_cast<int64_t>(dtype_size(dtype));
    a.rows = static_cast<uint32_t>(n);
    a.upr = upr;
    a.upr_magic = magic_for(upr);
    a.units = static_cast<uint32_t>(n * upr);
    a.inv = inv != nullptr ? inv + r0 * top_k : nullptr;
    a.top_k = top_k;
    a.rows_out = static_cast<uint32_t>(rows * top_k);
    a.codes = static_cast<uint8_t*>(codes) + (inv != nullptr ? 0 : r0 * (K / 2));
    a.scales = static_cast<uint8_t*>(scales) + (inv != nullptr ? 0 : r0 * pitch);
    a.pitch = static_cast<int>(pitch);
    const dim3 grid(grid_for(a.units, num_sms)), block(MXQ_THREADS);
    cudaError_t err;
    if (dtype == MOE_F32) err = launch_dependent(mx_quantize_kernel<float>, grid, block, 0, stream, a);
    else if (dtype == MOE_F16) err = launch_dependent(mx_quantize_kernel<__half>, grid, block, 0, stream, a);
    else err = launch_dependent(mx_quantize_kernel<__nv_bfloat16>, grid, block, 0, stream, a);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

cudaError_t launch_mx_dequantize(const void* codes, const void* scales, int64_t rows, int64_t K, void* out,
                                 moe_dtype dtype, int num_sms, cudaStream_t stream) {
  const uint32_t upr = static_cast<uint32_t>(K / 8);
  const int64_t step = rows_per_launch(K);
  const int64_t pitch = mx_scale_pitch(K);
  for (int64_t r0 = 0; r0 < rows; r0 += step) {
    const int64_t n = rows - r0 < step ? rows - r0 : step;
    DequantArgs a{};
    a.codes = static_cast<const uint8_t*>(codes) + r0 * (K / 2);
    a.scales = static_cast<const uint8_t*>(scales) + r0 * pitch;
    a.upr = upr;
    a.upr_magic = magic_for(upr);
    a.units = static_cast<uint32_t>(n * upr);
    a.pitch = static_cast<int>(pitch);
    a.out = static_cast<uint8_t*>(out) + r0 * K * static_cast<int64_t>(dtype_size(dtype));
    const dim3 grid(grid_for(a.units, num_sms)), block(MXQ_THREADS);
    cudaError_t err;
    if (dtype == MOE_F32) err = launch_dependent(mx_dequantize_kernel<float>, grid, block, 0, stream, a);
    else if (dtype == MOE_F16) err = launch_dependent(mx_dequantize_kernel<__half>, grid, block, 0, stream, a);
    else err = launch_dependent(mx_dequantize_kernel<__nv_bfloat16>, grid, block, 0, stream, a);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

cudaError_t launch_mx_layout_scales(const void* scales, void* dst, int64_t E, int64_t R, int64_t row_blocks, int64_t K,
                                    cudaStream_t stream) {
  const int64_t k_blocks = (K + 255) / 256;
  const int64_t n_words = E * row_blocks * k_blocks * 256;
  const int64_t want = (n_words + 255) / 256;
  mx_layout_scales_kernel<<<static_cast<unsigned>(want < 65535 ? want : 65535), 256, 0, stream>>>(
      static_cast<const uint8_t*>(scales), static_cast<uint32_t*>(dst), R, row_blocks, k_blocks, mx_scale_pitch(K),
      K / MX_BLOCK, n_words);
  return cudaGetLastError();
}

}  // namespace moe
