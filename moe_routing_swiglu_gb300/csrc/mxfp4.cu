// MXFP4 quantisation and its inverse (the format and its rounding are in
// mxfp4.cuh), and the one-time layout of the expert weights' scales for the
// tensor cores.
#include <type_traits>

#include "moe_common.cuh"
#include "moe_internal.h"
#include "mxfp4.cuh"

namespace moe {
namespace {

constexpr int MXQ_THREADS = 256;
constexpr int MXQ_UNROLL = 2;                           // 16-element units per thread and step
constexpr int MXQ_WARP_UNITS = 32 * MXQ_UNROLL;

// 32 bytes with one load or store (both addresses 32-byte aligned).
__device__ __forceinline__ void ld32(const void* p, uint32_t (&r)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st32(void* p, const uint32_t (&r)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// The same in two 16-byte halves, for bases that are only 16-byte aligned.
template <bool WIDE>
__device__ __forceinline__ void load32(const uint8_t* p, uint32_t (&r)[8]) {
  if (WIDE) {
    ld32(p, r);
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 16);
    r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w;
    r[4] = b.x; r[5] = b.y; r[6] = b.z; r[7] = b.w;
  }
}
template <bool WIDE>
__device__ __forceinline__ void store32(uint8_t* p, const uint32_t (&r)[8]) {
  if (WIDE) {
    st32(p, r);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(r[0], r[1], r[2], r[3]);
    *reinterpret_cast<uint4*>(p + 16) = make_uint4(r[4], r[5], r[6], r[7]);
  }
}

// 16 consecutive elements: raw words, the largest magnitude's FP32 bits
// (of this thread's 16), and the elements times a power of two.
template <typename T> struct Unit16 {  // F16, BF16
  uint32_t w[8];
  template <bool WIDE> __device__ __forceinline__ void load(const uint8_t* p) { load32<WIDE>(p, w); }
  __device__ __forceinline__ uint32_t amax_bits() const {
    // Magnitudes as pairs of 16-bit integers: integer order is the order of
    // the values, with infinities and NaNs on top.
    uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    const uint32_t h = max(m & 0xFFFFu, m >> 16);
    if (std::is_same<T, __nv_bfloat16>::value) return h << 16;
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(h))));
  }
  __device__ __forceinline__ void scaled8(int half, float s, float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const T* e = reinterpret_cast<const T*>(&w[half * 4 + i]);
      v[2 * i] = to_f32(e[0]) * s;
      v[2 * i + 1] = to_f32(e[1]) * s;
    }
  }
};
template <> struct Unit16<float> {
  uint32_t a[8], b[8];
  template <bool WIDE> __device__ __forceinline__ void load(const uint8_t* p) {
    load32<WIDE>(p, a);
    load32<WIDE>(p + 32, b);
  }
  __device__ __forceinline__ uint32_t amax_bits() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, max(a[i] & 0x7FFFFFFFu, b[i] & 0x7FFFFFFFu));
    return m;
  }
  __device__ __forceinline__ void scaled8(int half, float s, float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(half == 0 ? a[i] : b[i]) * s;
  }
};

struct QuantArgs {
  const uint8_t* x;
  uint32_t rows;
  uint32_t upr;        // 16-element units per row, K / 16
  uint32_t upr_magic;  // ceil(2^32 / upr)
  uint32_t units;      // rows * upr
  const uint32_t* inv; // [rows * top_k] output row of each slot, or NULL (row r -> row r)
  int top_k;
  uint32_t rows_out;   // rows * top_k: entries of inv at or past it are skipped
  uint8_t* codes;      // [rows_out, K / 2]
  uint8_t* scales;     // [rows_out, pitch]
  int pitch;
};

// One thread quantises 16 elements, two lanes share a block: 32 (or 64) bytes
// in, 8 bytes of codes out, coalesced over the warp; the block's largest
// magnitude takes one shuffle. Row by row the units are contiguous, so a warp
// takes 64 consecutive units whatever K is. With inv each row's codes go to
// its top_k dispatched rows: x is read once and no dispatched copy of it in
// its own type is ever written. Bound by HBM on large inputs: 98304 x 2048
// FP32 134 us (6.8 TB/s). 8192 x 4096 BF16 rows, two copies each, take 17.6 us in
// repeated calls, whose 102 MB fit L2 (27.4 with 8 elements a thread, whose issue
// slots were 60 % busy); 16 rows 1.8 us, a launch's latency.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(MXQ_THREADS) mx_quantize_kernel(const QuantArgs a) {
  grid_dependency_wait();
  launch_dependents();
  constexpr int UNIT_BYTES = 16 * static_cast<int>(sizeof(T));
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t warp = (blockIdx.x * MXQ_THREADS + threadIdx.x) >> 5;
  const uint32_t n_warps = gridDim.x * (MXQ_THREADS / 32);
  const uint32_t n_seg = (a.units + MXQ_WARP_UNITS - 1) / MXQ_WARP_UNITS;
  const int64_t code_pitch = static_cast<int64_t>(a.upr) * 8;
  for (uint32_t seg = warp; seg < n_seg; seg += n_warps) {
    const uint32_t u0 = seg * MXQ_WARP_UNITS;
    Unit16<T> in[MXQ_UNROLL];
#pragma unroll
    for (int i = 0; i < MXQ_UNROLL; ++i) {
      // units is even: a block's two lanes are both in or both out (those out read unit 0 and store nothing)
      const uint32_t u = u0 + i * 32 + lane;
      in[i].template load<WIDE>(a.x + static_cast<int64_t>(u < a.units ? u : 0) * UNIT_BYTES);
    }
    const uint32_t row0 = u0 / a.upr;
    const uint32_t rem0 = u0 - row0 * a.upr;
#pragma unroll
    for (int i = 0; i < MXQ_UNROLL; ++i) {
      const uint32_t off = i * 32 + lane;
      uint32_t amax = in[i].amax_bits();
      amax = max(amax, __shfl_xor_sync(FULL_MASK, amax, 1));
      if (u0 + off >= a.units) continue;
      const uint32_t byte = mx_scale_byte(amax);
      const float s = mx_inv_scale(byte);
      uint2 codes;
      float v[8];
      in[i].scaled8(0, s, v);
      codes.x = mx_pack8(v);
      in[i].scaled8(1, s, v);
      codes.y = mx_pack8(v);
      if (byte == 255u) codes = make_uint2(0u, 0u);
      const uint32_t local = rem0 + off;                      // < upr + 64
      const uint32_t dr = __umulhi(local, a.upr_magic);       // local / upr
      const uint32_t row = row0 + dr;
      const uint32_t unit = local - dr * a.upr;
      const uint32_t blk = unit >> 1;
      const bool head = (unit & 1u) == 0;
      auto store = [&](uint32_t r) {
        *reinterpret_cast<uint2*>(a.codes + static_cast<int64_t>(r) * code_pitch + unit * 8) = codes;
        if (head) {
          uint8_t* sp = a.scales + static_cast<int64_t>(r) * a.pitch;
          sp[blk] = static_cast<uint8_t>(byte);
          if (unit + 2 >= a.upr)  // the row's last block also clears the row's pad bytes
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
  uint8_t* out;
};

// One thread: 8 bytes of codes -> 16 values. Bound by HBM writes: 16384 x 4096
// to BF16 31 us in repeated calls (170 MB; 36.6 with a unit's two 16-byte
// halves stored in turn), 98304 x 2048 to BF16 89 us (5.7 TB/s).
template <typename T, bool WIDE>
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
    uint2 c[MXQ_UNROLL];
    uint32_t sb[MXQ_UNROLL];
#pragma unroll
    for (int i = 0; i < MXQ_UNROLL; ++i) {
      const uint32_t off = i * 32 + lane;
      if (u0 + off < a.units) {
        const uint32_t local = rem0 + off;
        const uint32_t dr = __umulhi(local, a.upr_magic);
        const uint32_t unit = local - dr * a.upr;
        c[i] = *reinterpret_cast<const uint2*>(a.codes + static_cast<int64_t>(u0 + off) * 8);
        sb[i] = a.scales[static_cast<int64_t>(row0 + dr) * a.pitch + (unit >> 1)];
      }
    }
#pragma unroll
    for (int i = 0; i < MXQ_UNROLL; ++i) {
      const uint32_t u = u0 + i * 32 + lane;
      if (u >= a.units) continue;
      const float s = mx_scale(sb[i]);
      uint8_t* dst = a.out + static_cast<int64_t>(u) * (16 * static_cast<int>(sizeof(T)));
      uint32_t o[8];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t h[4];
        mx_unpack8(half == 0 ? c[i].x : c[i].y, h);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
          if constexpr (std::is_same<T, float>::value) {
            o[2 * j] = __float_as_uint(f.x * s);
            o[2 * j + 1] = __float_as_uint(f.y * s);
          } else {
            o[half * 4 + j] = pack2<T>(f.x * s, f.y * s);
          }
        }
        if (std::is_same<T, float>::value) store32<WIDE>(dst + half * 32, o);
      }
      if (!std::is_same<T, float>::value) store32<WIDE>(dst, o);
    }
  }
}

// Row-major scales [E, R, pitch] -> the tensor cores' order: for each expert,
// weight block and 128 K elements two atoms of 512 bytes, of two 128-row tiles
// (gate and up rows of the same channels, or two halves of 256 down rows). An
// atom holds the four scale bytes of row m at byte (m % 32) * 16 + (m / 32) * 4.
// Rows and blocks past the matrix get 0.
__global__ void mx_layout_scales_kernel(const uint8_t* __restrict__ s0, const uint8_t* __restrict__ s1,
                                        uint32_t* __restrict__ dst, int64_t R, int64_t w_blocks, int64_t k_words,
                                        int64_t pitch, int64_t blocks_per_row, int64_t n_words) {
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; w < n_words;
       w += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int in = static_cast<int>(w & 127);          // word of the atom
    const int half = static_cast<int>((w >> 7) & 1);   // tile of the block
    const int64_t kw = (w >> 8) % k_words;             // which 128 K elements
    const int64_t wb = (w >> 8) / k_words % w_blocks;
    const int64_t e = (w >> 8) / k_words / w_blocks;
    const int64_t m = (s1 != nullptr ? wb : 2 * wb + half) * 128 + (in & 3) * 32 + (in >> 2);
    uint32_t v = 0;
    if (m < R) {
      const uint8_t* p = (s1 != nullptr && half != 0 ? s1 : s0) + (e * R + m) * pitch;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (kw * 4 + b < blocks_per_row) v |= static_cast<uint32_t>(p[kw * 4 + b]) << (8 * b);
    }
    dst[w] = v;
  }
}

// Rows per launch so that the unit count stays below 2^31.
int64_t rows_per_launch(int64_t K) { return ((int64_t{1} << 31) - MXQ_WARP_UNITS) / (K / 16); }

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
  const uint32_t upr = static_cast<uint32_t>(K / 16);
  const int64_t step = rows_per_launch(K);
  const int64_t pitch = mx_scale_pitch(K);
  for (int64_t r0 = 0; r0 < rows; r0 += step) {
    const int64_t n = rows - r0 < step ? rows - r0 : step;
    QuantArgs a{};
    a.x = static_cast<const uint8_t*>(x) + r0 * K * static_cast<int64_t>(dtype_size(dtype));
    const bool wide = reinterpret_cast<uintptr_t>(a.x) % 32 == 0;
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
    auto kern = dtype == MOE_F32   ? (wide ? mx_quantize_kernel<float, true> : mx_quantize_kernel<float, false>)
                : dtype == MOE_F16 ? (wide ? mx_quantize_kernel<__half, true> : mx_quantize_kernel<__half, false>)
                                   : (wide ? mx_quantize_kernel<__nv_bfloat16, true>
                                           : mx_quantize_kernel<__nv_bfloat16, false>);
    const cudaError_t err = launch_dependent(kern, grid, block, 0, stream, a);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

cudaError_t launch_mx_dequantize(const void* codes, const void* scales, int64_t rows, int64_t K, void* out,
                                 moe_dtype dtype, int num_sms, cudaStream_t stream) {
  const uint32_t upr = static_cast<uint32_t>(K / 16);
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
    const bool wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
    const dim3 grid(grid_for(a.units, num_sms)), block(MXQ_THREADS);
    auto kern = dtype == MOE_F32   ? (wide ? mx_dequantize_kernel<float, true> : mx_dequantize_kernel<float, false>)
                : dtype == MOE_F16 ? (wide ? mx_dequantize_kernel<__half, true> : mx_dequantize_kernel<__half, false>)
                                   : (wide ? mx_dequantize_kernel<__nv_bfloat16, true>
                                           : mx_dequantize_kernel<__nv_bfloat16, false>);
    const cudaError_t err = launch_dependent(kern, grid, block, 0, stream, a);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

cudaError_t launch_mx_layout_scales(const void* s0, const void* s1, void* dst, int64_t E, int64_t R, int64_t K,
                                    cudaStream_t stream) {
  const int64_t k_words = (K + 127) / 128;
  const int64_t w_blocks = mx_weight_blocks(s1 != nullptr, R);
  const int64_t n_words = E * w_blocks * k_words * 256;
  const int64_t want = (n_words + 255) / 256;
  mx_layout_scales_kernel<<<static_cast<unsigned>(want < 65535 ? want : 65535), 256, 0, stream>>>(
      static_cast<const uint8_t*>(s0), static_cast<const uint8_t*>(s1), static_cast<uint32_t*>(dst), R, w_blocks,
      k_words, mx_scale_pitch(K), K / MX_BLOCK, n_words);
  return cudaGetLastError();
}

}  // namespace moe
