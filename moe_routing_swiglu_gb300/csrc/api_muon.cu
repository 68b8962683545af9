// C ABI of the orthogonalised updates (contracts in include/moe.h).
#include <cmath>

#include "moe_common.cuh"
#include "moe_internal.h"

using moe::api_cuda_fail;
using moe::api_fail;
using moe::api_ok;
using moe::dtype_size;
using moe::dtype_valid;

namespace {

constexpr int64_t MAX_SIDE = 65536, MAX_MATRICES = 65535;

bool shape_ok(int64_t E, int64_t rows, int64_t cols) {
  if (E < 0 || rows < 0 || cols < 0 || E > MAX_MATRICES || rows > MAX_SIDE || cols > MAX_SIDE) return false;
  return moe::newton_schulz_tiles(E, rows, cols) <= 0x7FFFFFFF;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && na > 0 && nb > 0 && x < y + nb && y < x + na;
}

moe_status check_common(int64_t E, int64_t rows, int64_t cols, int32_t steps, float eps, const void* ws, size_t have) {
  if (!shape_ok(E, rows, cols))
    return api_fail(MOE_ERR_SHAPE, "need 0 <= E <= 65535, 0 <= rows, cols <= 65536 and fewer than 2^31 tiles");
  if (steps < 1 || steps > 100) return api_fail(MOE_ERR_SHAPE, "steps must be in 1 .. 100");
  if (!(eps > 0.0f) || !std::isfinite(eps)) return api_fail(MOE_ERR_SHAPE, "eps must be finite and > 0");
  if (E * rows * cols == 0) return MOE_OK;
  if (ws == nullptr || have < moe::newton_schulz_scratch_bytes(E, rows, cols))
    return api_fail(MOE_ERR_WORKSPACE, "workspace smaller than moe_orthogonalize_workspace_size()");
  if (reinterpret_cast<uintptr_t>(ws) % 256 != 0)
    return api_fail(MOE_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  return MOE_OK;
}

bool misaligned(const void* p, int dtype) {
  return reinterpret_cast<uintptr_t>(p) % dtype_size(static_cast<moe_dtype>(dtype)) != 0;
}

moe_status launch(const moe::NewtonSchulz& o, void* ws, void* stream, const char* where) {
  const char* why = nullptr;
  const cudaError_t err = moe::launch_newton_schulz(o, ws, static_cast<cudaStream_t>(stream), &why);
  if (err != cudaSuccess) return api_cuda_fail(err, where, why);
  return api_ok();
}

}  // namespace

extern "C" {

size_t moe_orthogonalize_workspace_size(int64_t E, int64_t rows, int64_t cols) {
  if (!shape_ok(E, rows, cols) || E * rows * cols == 0) return 0;
  return moe::newton_schulz_scratch_bytes(E, rows, cols);
}

moe_status moe_orthogonalize(const void* matrices, moe_dtype dtype, int64_t E, int64_t rows, int64_t cols,
                             int32_t steps, float eps, void* out, moe_dtype out_dtype, void* workspace,
                             size_t workspace_bytes, void* stream) {
  if (!dtype_valid(dtype)) return api_fail(MOE_ERR_DTYPE, "dtype must be MOE_F32, MOE_F16 or MOE_BF16");
  if (out_dtype != MOE_F16 && out_dtype != MOE_BF16)
    return api_fail(MOE_ERR_DTYPE, "out_dtype must be MOE_F16 or MOE_BF16");
  moe_status st = check_common(E, rows, cols, steps, eps, workspace, workspace_bytes);
  if (st != MOE_OK) return st;
  const size_t n = static_cast<size_t>(E * rows * cols);
  if (n == 0) return api_ok();
  if (matrices == nullptr || out == nullptr) return api_fail(MOE_ERR_NULL, "matrices and out must be non-NULL");
  if (misaligned(matrices, dtype) || misaligned(out, out_dtype))
    return api_fail(MOE_ERR_ALIGNMENT, "tensors must be aligned to their element size");
  const size_t in_bytes = n * dtype_size(dtype), out_bytes = n * dtype_size(out_dtype);
  const size_t ws_bytes = moe::newton_schulz_scratch_bytes(E, rows, cols);
  if (overlap(workspace, ws_bytes, matrices, in_bytes) || overlap(workspace, ws_bytes, out, out_bytes))
    return api_fail(MOE_ERR_SHAPE, "the workspace overlaps a tensor");
  // The matrices are read before the first product: out may be their own memory.
  moe::NewtonSchulz o{};
  o.grad = matrices;
  o.grad_dtype = dtype;
  o.E = E;
  o.rows = rows;
  o.cols = cols;
  o.steps = steps;
  o.eps = eps;
  o.result = out;
  o.result_dtype = out_dtype;
  return launch(o, workspace, stream, "moe_orthogonalize launch");
}

moe_status moe_muon_step(void* weight, moe_dtype weight_dtype, const void* grad, moe_dtype grad_dtype, float* momentum,
                         int64_t E, int64_t rows, int64_t cols, const moe_muon_params* p, void* workspace,
                         size_t workspace_bytes, void* stream) {
  if (!dtype_valid(weight_dtype) || !dtype_valid(grad_dtype))
    return api_fail(MOE_ERR_DTYPE, "dtypes must be MOE_F32, MOE_F16 or MOE_BF16");
  if (p == nullptr) return api_fail(MOE_ERR_NULL, "params must be non-NULL");
  if (!std::isfinite(p->lr) || !std::isfinite(p->weight_decay) || !std::isfinite(p->update_scale) ||
      !(p->momentum_decay >= 0.0f && p->momentum_decay < 1.0f))
    return api_fail(MOE_ERR_SHAPE, "lr, weight_decay and update_scale must be finite, momentum_decay in [0, 1)");
  const float keep = static_cast<float>(1.0 - static_cast<double>(p->lr) * p->weight_decay);
  const float rate = static_cast<float>(static_cast<double>(p->lr) * p->update_scale);
  if (!std::isfinite(keep) || !std::isfinite(rate))
    return api_fail(MOE_ERR_SHAPE, "lr * weight_decay and lr * update_scale must be in FP32's range");
  moe_status st = check_common(E, rows, cols, p->steps, p->eps, workspace, workspace_bytes);
  if (st != MOE_OK) return st;
  const size_t n = static_cast<size_t>(E * rows * cols);
  if (n == 0) return api_ok();
  if (weight == nullptr || grad == nullptr || momentum == nullptr)
    return api_fail(MOE_ERR_NULL, "weight, grad and momentum must be non-NULL");
  if (misaligned(weight, weight_dtype) || misaligned(grad, grad_dtype) || misaligned(momentum, MOE_F32))
    return api_fail(MOE_ERR_ALIGNMENT, "tensors must be aligned to their element size");
  const size_t wb = n * dtype_size(weight_dtype), gb = n * dtype_size(grad_dtype), mb = n * 4;
  const size_t sb = moe::newton_schulz_scratch_bytes(E, rows, cols);
  if (overlap(weight, wb, grad, gb) || overlap(weight, wb, momentum, mb) || overlap(grad, gb, momentum, mb) ||
      overlap(workspace, sb, weight, wb) || overlap(workspace, sb, grad, gb) || overlap(workspace, sb, momentum, mb))
    return api_fail(MOE_ERR_SHAPE, "two of weight, grad, momentum and workspace overlap");
  moe::NewtonSchulz o{};
  o.grad = grad;
  o.grad_dtype = grad_dtype;
  o.momentum = momentum;
  o.momentum_decay = p->momentum_decay;
  o.nesterov = p->nesterov != 0;
  o.E = E;
  o.rows = rows;
  o.cols = cols;
  o.steps = p->steps;
  o.eps = p->eps;
  o.result = weight;
  o.result_dtype = weight_dtype;
  o.update = 1;
  o.keep = keep;
  o.rate = rate;
  return launch(o, workspace, stream, "moe_muon_step launch");
}

}  // extern "C"
