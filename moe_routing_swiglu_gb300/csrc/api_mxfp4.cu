// C ABI of the MXFP4 experts: argument checks on the host, then kernel
// launches on the caller's stream (contracts in include/moe.h).
#include <algorithm>
#include <new>

#include "moe_common.cuh"
#include "moe_internal.h"
#include "mxfp4.cuh"

using moe::align_up;
using moe::api_cuda_fail;
using moe::api_fail;
using moe::api_ok;
using moe::dtype_size;
using moe::dtype_valid;

struct moe_experts_mxfp4 {
  int device;
  int num_sms;
  int64_t E, H, I;
  moe::MxWeights w;
};

namespace {

constexpr int64_t MX_MAX_K = 262144;
// Dispatched rows of the products: tensor-map coordinates are signed 32-bit.
constexpr int64_t MX_MAX_ROWS = (int64_t{1} << 31) - 1024;

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool k_valid(int64_t K) { return K >= 32 && K <= MX_MAX_K && K % 32 == 0; }
bool rows_valid(int64_t rows) { return rows >= 0 && rows < int64_t{0xFFFFFFFF}; }

moe_status device_sms(int* sms) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess) err = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return err == cudaSuccess ? MOE_OK : api_cuda_fail(err, "device query");
}

moe_status check_device(const moe_experts_mxfp4* ex) {
  int dev = -1;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return api_cuda_fail(err, "cudaGetDevice");
  if (dev != ex->device)
    return api_fail(MOE_ERR_UNSUPPORTED, "the current device is not the device the experts were created on");
  return MOE_OK;
}

// Codes and scales of an MXFP4 matrix.
moe_status check_mx(const void* codes, const void* scales, const char* null_msg, const char* align_msg) {
  if (codes == nullptr || scales == nullptr) return api_fail(MOE_ERR_NULL, null_msg);
  if (!aligned(codes, 16) || !aligned(scales, 4)) return api_fail(MOE_ERR_ALIGNMENT, align_msg);
  return MOE_OK;
}

constexpr char MX_ALIGN[] = "MXFP4 codes must be 16-byte and scales 4-byte aligned";

moe_status check_stage(const moe_experts_mxfp4* ex, const void* codes, const void* scales, const uint32_t* offsets,
                       int64_t rows, int dtype) {
  if (ex == nullptr || offsets == nullptr) return api_fail(MOE_ERR_NULL, "experts and offsets must be non-NULL");
  if (!dtype_valid(dtype)) return api_fail(MOE_ERR_DTYPE, "output dtype must be MOE_F32, MOE_F16 or MOE_BF16");
  if (rows < 0 || rows > MX_MAX_ROWS) return api_fail(MOE_ERR_SHAPE, "rows must be in 0 .. 2^31 - 1024");
  if (rows > 0) {
    const moe_status st = check_mx(codes, scales, "input codes and scales must be non-NULL", MX_ALIGN);
    if (st != MOE_OK) return st;
  }
  return check_device(ex);
}

moe_status run_stage(const moe_experts_mxfp4* ex, bool gate_up, const void* codes, const void* scales,
                     const uint32_t* offsets, int64_t rows, moe_dtype dtype, void* out, void* q_codes, void* q_scales,
                     cudaStream_t s) {
  const char* why = nullptr;
  const cudaError_t err =
      moe::launch_experts_mx(ex->w, gate_up, codes, scales, offsets, static_cast<int>(ex->E), rows, ex->H, ex->I, dtype,
                             out, q_codes, q_scales, ex->num_sms, s, &why);
  if (err != cudaSuccess)
    return api_cuda_fail(err, gate_up ? "MXFP4 gate/up launch" : "MXFP4 down launch", why);
  return MOE_OK;
}

// h as MXFP4 [rows, I]: codes, then scales.
struct HiddenLayout {
  size_t scales, total;
};
HiddenLayout hidden_layout(const moe_experts_mxfp4* ex, int64_t rows) {
  const size_t n = static_cast<size_t>(rows);
  HiddenLayout h{};
  h.scales = align_up(n * static_cast<size_t>(ex->I / 2) + 1, 256);
  h.total = h.scales + align_up(n * static_cast<size_t>(moe::mx_scale_pitch(ex->I)) + 1, 256);
  return h;
}

struct ForwardMxLayout {
  size_t indices, weights, counts, offsets, row_src, inv, scratch, xq, xs, h, y, total;
};
ForwardMxLayout forward_mx_layout(const moe_experts_mxfp4* ex, int64_t T, int top_k, moe_dtype dtype) {
  const size_t n = static_cast<size_t>(T) * static_cast<size_t>(top_k);
  ForwardMxLayout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align_up(bytes > 0 ? bytes : 1, 256);
    return at;
  };
  L.indices = take(n * 4);
  L.weights = take(n * 4);  // room for any logits dtype
  L.counts = take(static_cast<size_t>(ex->E) * 4);
  L.offsets = take(static_cast<size_t>(ex->E + 1) * 4);
  L.row_src = take(n * 4);
  L.inv = take(n * 4);
  L.scratch = take(moe::route_dispatch_scratch_bytes(T, ex->E));
  L.xq = take(n * static_cast<size_t>(ex->H / 2));
  L.xs = take(n * static_cast<size_t>(moe::mx_scale_pitch(ex->H)));
  L.h = take(hidden_layout(ex, static_cast<int64_t>(n)).total);
  L.y = take(n * static_cast<size_t>(ex->H) * dtype_size(dtype));
  L.total = off;
  return L;
}

bool slots_fit(int64_t T, int64_t k) { return T >= 0 && k >= 1 && T <= int64_t{0xFFFFFFFE} / k; }

}  // namespace

extern "C" {

int64_t moe_mxfp4_scale_pitch(int64_t K) { return K > 0 && K % 32 == 0 ? moe::mx_scale_pitch(K) : 0; }

moe_status moe_mxfp4_quantize(const void* x, moe_dtype dtype, int64_t rows, int64_t K, const uint32_t* inv,
                              int32_t top_k, void* codes, void* scales, void* stream) {
  if (!dtype_valid(dtype)) return api_fail(MOE_ERR_DTYPE, "x dtype must be MOE_F32, MOE_F16 or MOE_BF16");
  if (!k_valid(K)) return api_fail(MOE_ERR_SHAPE, "K must be a multiple of 32 in 32 .. 262144");
  if (top_k < 1 || (inv == nullptr && top_k != 1))
    return api_fail(MOE_ERR_TOP_K, "top_k must be >= 1, and 1 without inv");
  if (!slots_fit(rows, top_k)) return api_fail(MOE_ERR_SHAPE, "rows must be >= 0 and rows*top_k < 2^32-1");
  if (rows == 0) return api_ok();
  if (x == nullptr) return api_fail(MOE_ERR_NULL, "x must be non-NULL");
  if (!aligned(x, 16) || !aligned(inv, 4))
    return api_fail(MOE_ERR_ALIGNMENT, "x must be 16-byte and inv 4-byte aligned");
  moe_status st = check_mx(codes, scales, "codes and scales must be non-NULL", MX_ALIGN);
  if (st != MOE_OK) return st;
  int sms = 0;
  st = device_sms(&sms);
  if (st != MOE_OK) return st;
  const cudaError_t err = moe::launch_mx_quantize(x, dtype, rows, K, inv, top_k, codes, scales, sms,
                                                  static_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return api_cuda_fail(err, "moe_mxfp4_quantize launch");
  return api_ok();
}

moe_status moe_mxfp4_dequantize(const void* codes, const void* scales, int64_t rows, int64_t K, void* out,
                                moe_dtype dtype, void* stream) {
  if (!dtype_valid(dtype)) return api_fail(MOE_ERR_DTYPE, "out dtype must be MOE_F32, MOE_F16 or MOE_BF16");
  if (!k_valid(K)) return api_fail(MOE_ERR_SHAPE, "K must be a multiple of 32 in 32 .. 262144");
  if (!rows_valid(rows)) return api_fail(MOE_ERR_SHAPE, "rows must be in 0 .. 2^32-2");
  if (rows == 0) return api_ok();
  moe_status st = check_mx(codes, scales, "codes and scales must be non-NULL", MX_ALIGN);
  if (st != MOE_OK) return st;
  if (out == nullptr) return api_fail(MOE_ERR_NULL, "out must be non-NULL");
  if (!aligned(out, 16)) return api_fail(MOE_ERR_ALIGNMENT, "out must be 16-byte aligned");
  int sms = 0;
  st = device_sms(&sms);
  if (st != MOE_OK) return st;
  const cudaError_t err =
      moe::launch_mx_dequantize(codes, scales, rows, K, out, dtype, sms, static_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return api_cuda_fail(err, "moe_mxfp4_dequantize launch");
  return api_ok();
}

size_t moe_experts_mxfp4_storage_size(int64_t E, int64_t H, int64_t I) {
  if (E < 1 || E > moe::ROUTE_MAX_E || !k_valid(H) || !k_valid(I)) return 0;
  return moe::mx_weight_scale_bytes(true, E, I, H) + moe::mx_weight_scale_bytes(false, E, H, I);
}

moe_status moe_experts_mxfp4_create(const void* gate_codes, const void* gate_scales, const void* up_codes,
                                    const void* up_scales, const void* down_codes, const void* down_scales, int64_t E,
                                    int64_t H, int64_t I, void* storage, size_t storage_bytes, void* stream,
                                    moe_experts_mxfp4** out) {
  if (out == nullptr) return api_fail(MOE_ERR_NULL, "out must be non-NULL");
  *out = nullptr;
  if (E < 1 || E > moe::ROUTE_MAX_E) return api_fail(MOE_ERR_SHAPE, "E must satisfy 1 <= E <= 1024");
  if (!k_valid(H) || !k_valid(I)) return api_fail(MOE_ERR_SHAPE, "H and I must be multiples of 32 in 32 .. 262144");
  const void* const pairs[3][2] = {{gate_codes, gate_scales}, {up_codes, up_scales}, {down_codes, down_scales}};
  for (const auto& p : pairs) {
    const moe_status st = check_mx(p[0], p[1], "gate, up and down codes and scales must be non-NULL", MX_ALIGN);
    if (st != MOE_OK) return st;
  }
  if (storage == nullptr || storage_bytes < moe_experts_mxfp4_storage_size(E, H, I))
    return api_fail(MOE_ERR_WORKSPACE, "storage smaller than moe_experts_mxfp4_storage_size()");
  if (!aligned(storage, 256)) return api_fail(MOE_ERR_ALIGNMENT, "storage must be 256-byte aligned");
  moe_experts_mxfp4* ex = new (std::nothrow) moe_experts_mxfp4{};
  if (ex == nullptr) return api_fail(MOE_ERR_WORKSPACE, "no host memory for the handle");
  ex->E = E;
  ex->H = H;
  ex->I = I;
  cudaError_t err = cudaGetDevice(&ex->device);
  if (err == cudaSuccess) err = cudaDeviceGetAttribute(&ex->num_sms, cudaDevAttrMultiProcessorCount, ex->device);
  if (err != cudaSuccess) {
    delete ex;
    return api_cuda_fail(err, "moe_experts_mxfp4_create device query");
  }
  ex->w.gate = gate_codes;
  ex->w.up = up_codes;
  ex->w.down = down_codes;
  uint8_t* sf = static_cast<uint8_t*>(storage);
  uint8_t* sf_down = sf + moe::mx_weight_scale_bytes(true, E, I, H);
  ex->w.gate_up_sf = sf;
  ex->w.down_sf = sf_down;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  err = moe::launch_mx_layout_scales(gate_scales, up_scales, sf, E, I, H, s);
  if (err == cudaSuccess) err = moe::launch_mx_layout_scales(down_scales, nullptr, sf_down, E, H, I, s);
  if (err != cudaSuccess) {
    delete ex;
    return api_cuda_fail(err, "moe_experts_mxfp4_create scale layout");
  }
  *out = ex;
  return api_ok();
}

void moe_experts_mxfp4_destroy(moe_experts_mxfp4* experts) { delete experts; }

moe_status moe_experts_mxfp4_gate_up(const moe_experts_mxfp4* ex, const void* x_codes, const void* x_scales,
                                     const uint32_t* offsets, int64_t rows, moe_dtype dtype, void* h, void* h_codes,
                                     void* h_scales, void* stream) {
  moe_status st = check_stage(ex, x_codes, x_scales, offsets, rows, dtype);
  if (st != MOE_OK) return st;
  if (rows == 0) return api_ok();
  if ((h_codes == nullptr) != (h_scales == nullptr))
    return api_fail(MOE_ERR_NULL, "h_codes and h_scales must both be given or both be NULL");
  if (h == nullptr && h_codes == nullptr) return api_fail(MOE_ERR_NULL, "h, or h_codes and h_scales, must be non-NULL");
  if (!aligned(h, 16) || !aligned(h_codes, 16) || !aligned(h_scales, 4))
    return api_fail(MOE_ERR_ALIGNMENT, "h and h_codes must be 16-byte, h_scales 4-byte aligned");
  st = run_stage(ex, true, x_codes, x_scales, offsets, rows, dtype, h, h_codes, h_scales,
                 static_cast<cudaStream_t>(stream));
  return st != MOE_OK ? st : api_ok();
}

moe_status moe_experts_mxfp4_down(const moe_experts_mxfp4* ex, const void* h_codes, const void* h_scales,
                                  const uint32_t* offsets, int64_t rows, moe_dtype dtype, void* y, void* stream) {
  moe_status st = check_stage(ex, h_codes, h_scales, offsets, rows, dtype);
  if (st != MOE_OK) return st;
  if (rows == 0) return api_ok();
  if (y == nullptr) return api_fail(MOE_ERR_NULL, "y must be non-NULL");
  if (!aligned(y, 16)) return api_fail(MOE_ERR_ALIGNMENT, "y must be 16-byte aligned");
  st = run_stage(ex, false, h_codes, h_scales, offsets, rows, dtype, y, nullptr, nullptr,
                 static_cast<cudaStream_t>(stream));
  return st != MOE_OK ? st : api_ok();
}

size_t moe_experts_mxfp4_forward_dispatched_workspace_size(const moe_experts_mxfp4* ex, int64_t rows) {
  if (ex == nullptr || rows < 0 || rows > MX_MAX_ROWS) return 0;
  return hidden_layout(ex, rows).total;
}

moe_status moe_experts_mxfp4_forward_dispatched(const moe_experts_mxfp4* ex, const void* x_codes, const void* x_scales,
                                                const uint32_t* offsets, int64_t rows, moe_dtype dtype, void* y,
                                                void* workspace, size_t workspace_bytes, void* stream) {
  moe_status st = check_stage(ex, x_codes, x_scales, offsets, rows, dtype);
  if (st != MOE_OK) return st;
  if (rows > 0 && y == nullptr) return api_fail(MOE_ERR_NULL, "y must be non-NULL");
  if (!aligned(y, 16)) return api_fail(MOE_ERR_ALIGNMENT, "y must be 16-byte aligned");
  const HiddenLayout hl = hidden_layout(ex, rows);
  if (workspace == nullptr || workspace_bytes < hl.total)
    return api_fail(MOE_ERR_WORKSPACE, "workspace smaller than moe_experts_mxfp4_forward_dispatched_workspace_size()");
  if (!aligned(workspace, 256)) return api_fail(MOE_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  if (rows == 0) return api_ok();
  uint8_t* hq = static_cast<uint8_t*>(workspace);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = run_stage(ex, true, x_codes, x_scales, offsets, rows, dtype, nullptr, hq, hq + hl.scales, s);
  if (st != MOE_OK) return st;
  st = run_stage(ex, false, hq, hq + hl.scales, offsets, rows, dtype, y, nullptr, nullptr, s);
  return st != MOE_OK ? st : api_ok();
}

size_t moe_forward_mxfp4_workspace_size(const moe_experts_mxfp4* ex, int64_t T, int32_t top_k, moe_dtype dtype) {
  if (ex == nullptr || T < 0 || top_k < 1 || T > MX_MAX_ROWS / top_k || !dtype_valid(dtype)) return 0;
  return forward_mx_layout(ex, T, top_k, dtype).total;
}

moe_status moe_forward_mxfp4(const moe_experts_mxfp4* ex, const void* x, moe_dtype dtype, const void* logits,
                             moe_dtype logits_dtype, int64_t T, int32_t top_k, int32_t renormalize, void* out,
                             uint32_t* indices_opt, void* weights_opt, void* workspace, size_t workspace_bytes,
                             void* stream) {
  if (ex == nullptr) return api_fail(MOE_ERR_NULL, "experts must be non-NULL");
  if (!dtype_valid(dtype) || !dtype_valid(logits_dtype))
    return api_fail(MOE_ERR_DTYPE, "dtypes must be MOE_F32, MOE_F16 or MOE_BF16");
  if (top_k < 1 || top_k > ex->E) return api_fail(MOE_ERR_TOP_K, "top_k must satisfy 1 <= top_k <= E");
  if (T < 0 || T > MX_MAX_ROWS / top_k) return api_fail(MOE_ERR_SHAPE, "T must be >= 0 and T*top_k <= 2^31 - 1024");
  if (T > 0 && (x == nullptr || logits == nullptr || out == nullptr))
    return api_fail(MOE_ERR_NULL, "x, logits and out must be non-NULL");
  if (!aligned(x, 16) || !aligned(out, 16)) return api_fail(MOE_ERR_ALIGNMENT, "x and out must be 16-byte aligned");
  const ForwardMxLayout L = forward_mx_layout(ex, T, top_k, dtype);
  if (workspace == nullptr || workspace_bytes < L.total)
    return api_fail(MOE_ERR_WORKSPACE, "workspace smaller than moe_forward_mxfp4_workspace_size()");
  if (!aligned(workspace, 256)) return api_fail(MOE_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  moe_status st = check_device(ex);
  if (st != MOE_OK) return st;
  if (T == 0) return api_ok();

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint32_t* indices = indices_opt != nullptr ? indices_opt : reinterpret_cast<uint32_t*>(ws + L.indices);
  void* weights = weights_opt != nullptr ? weights_opt : static_cast<void*>(ws + L.weights);
  uint32_t* offsets = reinterpret_cast<uint32_t*>(ws + L.offsets);
  uint32_t* inv = reinterpret_cast<uint32_t*>(ws + L.inv);
  const int64_t rows = T * top_k;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t err = moe::launch_route_dispatch(
      logits, logits_dtype, T, static_cast<int>(ex->E), top_k, renormalize != 0, indices, weights, nullptr, nullptr,
      dtype, ex->H, reinterpret_cast<uint32_t*>(ws + L.counts), offsets, reinterpret_cast<uint32_t*>(ws + L.row_src),
      inv, nullptr, ws + L.scratch, ex->num_sms, s);
  if (err != cudaSuccess) return api_cuda_fail(err, "moe_forward_mxfp4 route + dispatch launch");
  err = moe::launch_mx_quantize(x, dtype, T, ex->H, inv, top_k, ws + L.xq, ws + L.xs, ex->num_sms, s);
  if (err != cudaSuccess) return api_cuda_fail(err, "moe_forward_mxfp4 quantisation launch");
  uint8_t* hq = ws + L.h;
  uint8_t* hs = hq + hidden_layout(ex, rows).scales;
  st = run_stage(ex, true, ws + L.xq, ws + L.xs, offsets, rows, dtype, nullptr, hq, hs, s);
  if (st != MOE_OK) return st;
  st = run_stage(ex, false, hq, hs, offsets, rows, dtype, ws + L.y, nullptr, nullptr, s);
  if (st != MOE_OK) return st;
  err = moe::launch_combine(ws + L.y, dtype, inv, weights, logits_dtype, T, top_k, ex->H, out, s);
  if (err != cudaSuccess) return api_cuda_fail(err, "moe_forward_mxfp4 combine launch");
  return api_ok();
}

}  // extern "C"
