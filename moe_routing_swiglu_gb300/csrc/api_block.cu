// C ABI of the norms around a block (contracts in include/moe.h).
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "moe_common.cuh"
#include "moe_internal.h"

using moe::api_cuda_fail;
using moe::api_fail;
using moe::api_ok;
using moe::dtype_size;
using moe::dtype_valid;

namespace {

// A buffer of a call. Two buffers of the same rows (`rows` set: [T, H] in the
// call's dtype) may be one and the same: a thread reads its elements of a row
// before it writes them. Every other overlap with a written buffer is an error.
struct Range {
  const void* p;
  size_t bytes;
  bool rows;
};

moe_status check_overlap(std::initializer_list<Range> written, std::initializer_list<Range> read) {
  auto clash = [](const Range& a, const Range& b) {
    if (a.p == nullptr || b.p == nullptr || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.bytes && y < x + a.bytes;
  };
  for (auto w = written.begin(); w != written.end(); ++w) {
    for (auto o = written.begin(); o != w; ++o)
      if (clash(*w, *o)) return api_fail(MOE_ERR_SHAPE, "two outputs overlap");
    for (const Range& r : read)
      if (clash(*w, r) && !(w->rows && r.rows && w->p == r.p))
        return api_fail(MOE_ERR_SHAPE, "an output overlaps an input that is not the same tensor");
  }
  return MOE_OK;
}

moe_status check_rows(int dtype, int64_t T, int64_t H) {
  if (!dtype_valid(dtype)) return api_fail(MOE_ERR_DTYPE, "dtype must be MOE_F32, MOE_F16 or MOE_BF16");
  if (H < 1 || H > moe::BLOCK_NORM_MAX_H) return api_fail(MOE_ERR_SHAPE, "H must be in 1 .. 32768");
  if (T < 0 || T > 0x7FFFFFFF) return api_fail(MOE_ERR_SHAPE, "T must be in 0 .. 2^31 - 1");
  return MOE_OK;
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

moe_status check_eps(float eps) {
  if (!(eps > 0.0f) || !std::isfinite(eps)) return api_fail(MOE_ERR_SHAPE, "eps must be finite and > 0");
  return MOE_OK;
}

// The backward's factors hold up to the cube of 1 / sqrt(mean + eps) times the
// gradients, 2^120 of them from this eps on. Below about 2^-128 the square alone
// is infinite, and the gradient of a row of zeros was NaN.
moe_status check_backward_eps(float eps) {
  if (eps < 0x1p-80f) return api_fail(MOE_ERR_SHAPE, "eps must be at least 2^-80 in a backward call");
  return MOE_OK;
}

moe_status check_vector(const void* p, int vec_dtype, int dtype) {
  if (vec_dtype != MOE_F32 && vec_dtype != dtype)
    return api_fail(MOE_ERR_DTYPE, "weight vectors must be MOE_F32 or of the rows' dtype");
  if (misaligned(p, dtype_size(static_cast<moe_dtype>(vec_dtype))))
    return api_fail(MOE_ERR_ALIGNMENT, "weight vectors must be aligned to their element size");
  return MOE_OK;
}

moe_status check_params(const moe_block_join_params* p, int dtype, int64_t T) {
  if (p == nullptr) return api_fail(MOE_ERR_NULL, "params must be non-NULL");
  if (p->gate_kind < MOE_GATE_NONE || p->gate_kind > MOE_GATE_ELEMENT)
    return api_fail(MOE_ERR_SHAPE, "unknown gate kind");
  if (p->gate_kind != MOE_GATE_NONE && p->gate == nullptr && (T > 0 || p->gate_kind == MOE_GATE_CHANNEL))
    return api_fail(MOE_ERR_NULL, "gate must be non-NULL");
  if (!std::isfinite(p->residual_scale) || !std::isfinite(p->branch_scale))
    return api_fail(MOE_ERR_SHAPE, "residual_scale and branch_scale must be finite");
  moe_status st = check_eps(p->eps);
  if (st != MOE_OK) return st;
  const bool gate_vector = p->gate_kind == MOE_GATE_CHANNEL || p->gate_kind == MOE_GATE_TOKEN;
  for (const void* v : {p->norm_weight, p->next_weight, gate_vector ? p->gate : nullptr})
    if (v != nullptr && (st = check_vector(v, p->vec_dtype, dtype)) != MOE_OK) return st;
  return MOE_OK;
}

moe_status device_sms(int* sms) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess) err = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return err == cudaSuccess ? MOE_OK : api_cuda_fail(err, "device query");
}

size_t vector_bytes(const moe_block_join_params* p, int64_t n) {
  return static_cast<size_t>(n) * dtype_size(static_cast<moe_dtype>(p->vec_dtype));
}
Range gate_range(const moe_block_join_params* p, moe_dtype dtype, int64_t T, int64_t H) {
  switch (p->gate_kind) {
    case MOE_GATE_CHANNEL: return {p->gate, vector_bytes(p, H), false};
    case MOE_GATE_TOKEN: return {p->gate, vector_bytes(p, T), false};
    case MOE_GATE_ELEMENT: return {p->gate, static_cast<size_t>(T * H) * dtype_size(dtype), true};
    default: return {nullptr, 0, false};
  }
}

bool rows_misaligned(moe_dtype dtype, std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (misaligned(p, dtype_size(dtype))) return true;
  return false;
}

// Forward with either kind of branch (combine: rows of expert outputs).
moe_status join(const void* branch, size_t branch_bytes, bool combine, const uint32_t* inv, const void* weights,
                moe_dtype weights_dtype, int32_t top_k, const void* residual, moe_dtype dtype,
                const moe_block_join_params* p, int64_t T, int64_t H, void* out, void* normed, void* stream,
                const char* where) {
  moe_status st = check_params(p, dtype, T);
  if (st != MOE_OK) return st;
  if (T == 0) return api_ok();
  if (branch == nullptr || residual == nullptr || out == nullptr)
    return api_fail(MOE_ERR_NULL, "the branch, residual and out must be non-NULL");
  if ((p->next_weight != nullptr) != (normed != nullptr))
    return api_fail(MOE_ERR_NULL, "normed and next_weight go together");
  if (rows_misaligned(dtype, {branch, residual, out, normed, p->gate_kind == MOE_GATE_ELEMENT ? p->gate : nullptr}))
    return api_fail(MOE_ERR_ALIGNMENT, "rows must be aligned to their element size");
  const size_t bytes = static_cast<size_t>(T * H) * dtype_size(dtype);
  const size_t slots = combine ? static_cast<size_t>(T) * top_k : 0;
  st = check_overlap({{out, bytes, true}, {normed, bytes, true}},
                     {{branch, branch_bytes, !combine},
                      {residual, bytes, true},
                      {p->norm_weight, vector_bytes(p, H), false},
                      {p->next_weight, vector_bytes(p, H), false},
                      gate_range(p, dtype, T, H),
                      {inv, slots * 4, false},
                      {weights, combine ? slots * dtype_size(weights_dtype) : 0, false}});
  if (st != MOE_OK) return st;
  int sms = 0;
  st = device_sms(&sms);
  if (st != MOE_OK) return st;
  const moe::JoinArgs a{branch, residual, out, normed, p->norm_weight, p->next_weight, p->gate, inv, weights, T,
                        static_cast<int>(H), p->gate_kind, p->vec_dtype == MOE_F32, weights_dtype, top_k,
                        static_cast<uint32_t>(slots), p->residual_scale, p->branch_scale, p->eps, nullptr};
  const cudaError_t err = moe::launch_join(dtype, a, combine ? 2 : 1, sms, static_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return api_cuda_fail(err, where);
  return api_ok();
}

// Bytes of `arrays` column sums of every unit.
size_t partial_bytes(int64_t T, int64_t H, int arrays) {
  if (T < 0 || T > 0x7FFFFFFF || H < 1 || H > moe::BLOCK_NORM_MAX_H) return 0;
  return moe::align_up(static_cast<size_t>(std::max<int64_t>(1, moe::join_backward_units(T, H)) * arrays * H) * 4, 256);
}

moe_status check_workspace(const void* ws, size_t have, size_t need) {
  if (ws == nullptr || have < need) return api_fail(MOE_ERR_WORKSPACE, "workspace smaller than its size function says");
  if (misaligned(ws, 256)) return api_fail(MOE_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_block_norm(const void* x, moe_dtype dtype, const void* weight, moe_dtype weight_dtype, float eps,
                          int64_t T, int64_t H, void* y, void* stream) {
  moe_status st = check_rows(dtype, T, H);
  if (st == MOE_OK) st = check_eps(eps);
  if (st != MOE_OK) return st;
  if (weight == nullptr) return api_fail(MOE_ERR_NULL, "weight must be non-NULL");
  st = check_vector(weight, weight_dtype, dtype);
  if (st != MOE_OK) return st;
  if (T == 0) return api_ok();
  if (x == nullptr || y == nullptr) return api_fail(MOE_ERR_NULL, "x and y must be non-NULL");
  if (rows_misaligned(dtype, {x, y})) return api_fail(MOE_ERR_ALIGNMENT, "rows must be aligned to their element size");
  const size_t bytes = static_cast<size_t>(T * H) * dtype_size(dtype);
  st = check_overlap({{y, bytes, true}},
                     {{x, bytes, true}, {weight, static_cast<size_t>(H) * dtype_size(weight_dtype), false}});
  if (st != MOE_OK) return st;
  int sms = 0;
  st = device_sms(&sms);
  if (st != MOE_OK) return st;
  moe::JoinArgs a{};
  a.x = x;
  a.y = y;
  a.next_weight = weight;
  a.T = T;
  a.H = static_cast<int>(H);
  a.vec_f32 = weight_dtype == MOE_F32;
  a.eps = eps;
  const cudaError_t err = moe::launch_join(dtype, a, 0, sms, static_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return api_cuda_fail(err, "moe_block_norm launch");
  return api_ok();
}

size_t moe_block_norm_backward_workspace_size(int64_t T, int64_t H) { return partial_bytes(T, H, 1); }

moe_status moe_block_norm_backward(const void* dy, const void* x, moe_dtype dtype, const void* weight,
                                   moe_dtype weight_dtype, const void* dresidual, float eps, int64_t T, int64_t H,
                                   void* dx, float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
  moe_status st = check_rows(dtype, T, H);
  if (st == MOE_OK) st = check_eps(eps);
  if (st == MOE_OK) st = check_backward_eps(eps);
  if (st != MOE_OK) return st;
  if (weight == nullptr || dweight == nullptr) return api_fail(MOE_ERR_NULL, "weight and dweight must be non-NULL");
  st = check_vector(weight, weight_dtype, dtype);
  if (st != MOE_OK) return st;
  if (T > 0 && (dy == nullptr || x == nullptr || dx == nullptr))
    return api_fail(MOE_ERR_NULL, "dy, x and dx must be non-NULL");
  if (rows_misaligned(dtype, {dy, x, dresidual, dx}) || misaligned(dweight, 4))
    return api_fail(MOE_ERR_ALIGNMENT, "tensors must be aligned to their element size");
  const size_t need = partial_bytes(T, H, 1);
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != MOE_OK) return st;
  const size_t bytes = static_cast<size_t>(T * H) * dtype_size(dtype);
  st = check_overlap({{dx, bytes, true}, {dweight, static_cast<size_t>(H) * 4, false}, {workspace, need, false}},
                     {{dy, bytes, true},
                      {x, bytes, true},
                      {dresidual, bytes, true},
                      {weight, static_cast<size_t>(H) * dtype_size(weight_dtype), false}});
  if (st != MOE_OK) return st;
  moe::JoinBackwardArgs a{};
  a.dout = dresidual;
  a.dnormed = dy;
  a.joined = x;
  a.next_weight = weight;
  a.dresidual = dx;
  a.partial = static_cast<float*>(workspace);
  a.T = T;
  a.H = static_cast<int>(H);
  a.vec_f32 = weight_dtype == MOE_F32;
  a.arrays = 1;
  a.alpha = 1.0f;
  a.eps = eps;
  const cudaError_t err =
      moe::launch_join_backward(dtype, a, nullptr, dweight, static_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return api_cuda_fail(err, "moe_block_norm_backward launch");
  return api_ok();
}

moe_status moe_block_join(const void* branch, const void* residual, moe_dtype dtype, const moe_block_join_params* params,
                          int64_t T, int64_t H, void* out, void* normed, void* stream) {
  const moe_status st = check_rows(dtype, T, H);
  if (st != MOE_OK) return st;
  return join(branch, static_cast<size_t>(T * H) * dtype_size(dtype), false, nullptr, nullptr, MOE_F32, 0, residual,
              dtype, params, T, H, out, normed, stream, "moe_block_join launch");
}

moe_status moe_combine_join(const void* y_dispatched, moe_dtype dtype, const uint32_t* inv, const void* weights,
                            moe_dtype weights_dtype, const void* residual, const moe_block_join_params* params,
                            int64_t T, int32_t top_k, int64_t H, void* out, void* normed, void* stream) {
  const moe_status st = check_rows(dtype, T, H);
  if (st != MOE_OK) return st;
  if (!dtype_valid(weights_dtype)) return api_fail(MOE_ERR_DTYPE, "weights_dtype must be MOE_F32, MOE_F16 or MOE_BF16");
  if (top_k < 1) return api_fail(MOE_ERR_TOP_K, "top_k must be >= 1");
  if (T > int64_t{0xFFFFFFFE} / top_k) return api_fail(MOE_ERR_SHAPE, "need T*top_k < 2^32-1");
  if (T > 0 && (inv == nullptr || weights == nullptr))
    return api_fail(MOE_ERR_NULL, "inv and weights must be non-NULL");
  if (misaligned(inv, 4) || misaligned(weights, dtype_size(weights_dtype)))
    return api_fail(MOE_ERR_ALIGNMENT, "inv and weights must be aligned to their element size");
  return join(y_dispatched, static_cast<size_t>(T * H) * top_k * dtype_size(dtype), true, inv, weights, weights_dtype,
              top_k, residual, dtype, params, T, H, out, normed, stream, "moe_combine_join launch");
}

size_t moe_block_join_backward_workspace_size(int64_t T, int64_t H) { return partial_bytes(T, H, 3); }

moe_status moe_block_join_backward(const void* dout, const void* dnormed, const void* branch, const void* joined,
                                   moe_dtype dtype, const moe_block_join_params* p, int64_t T, int64_t H,
                                   void* dbranch, void* dresidual, float* dnorm_weight, void* dgate,
                                   float* dnext_weight, void* workspace, size_t workspace_bytes, void* stream) {
  moe_status st = check_rows(dtype, T, H);
  if (st == MOE_OK) st = check_params(p, dtype, T);
  if (st == MOE_OK) st = check_backward_eps(p->eps);
  if (st != MOE_OK) return st;
  const bool next = p->next_weight != nullptr, gated = p->gate_kind != MOE_GATE_NONE;
  const bool element = p->gate_kind == MOE_GATE_ELEMENT;
  if (T > 0 && (branch == nullptr || dbranch == nullptr || dresidual == nullptr))
    return api_fail(MOE_ERR_NULL, "branch, dbranch and dresidual must be non-NULL");
  if (T > 0 && next && (dnormed == nullptr || joined == nullptr))
    return api_fail(MOE_ERR_NULL, "dnormed and joined must be non-NULL with next_weight");
  if (T > 0 && !next && dout == nullptr) return api_fail(MOE_ERR_NULL, "dout must be non-NULL without next_weight");
  if ((dnorm_weight != nullptr) != (p->norm_weight != nullptr) || (dnext_weight != nullptr) != next ||
      ((dgate != nullptr) != gated && (T > 0 || p->gate_kind == MOE_GATE_CHANNEL)))
    return api_fail(MOE_ERR_NULL, "dnorm_weight, dgate and dnext_weight go with norm_weight, gate and next_weight");
  if (!next) dnormed = joined = nullptr;
  if (rows_misaligned(dtype, {dout, dnormed, branch, joined, dbranch, dresidual, element ? p->gate : nullptr,
                              element ? dgate : nullptr}) ||
      misaligned(dnorm_weight, 4) || misaligned(dnext_weight, 4) || (gated && !element && misaligned(dgate, 4)))
    return api_fail(MOE_ERR_ALIGNMENT, "tensors must be aligned to their element size");
  const size_t need = partial_bytes(T, H, 3);
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != MOE_OK) return st;
  const size_t bytes = static_cast<size_t>(T * H) * dtype_size(dtype), col = static_cast<size_t>(H) * 4;
  const size_t dgate_bytes = element ? bytes : p->gate_kind == MOE_GATE_TOKEN ? static_cast<size_t>(T) * 4 : col;
  st = check_overlap({{dbranch, bytes, true},
                      {dresidual, bytes, true},
                      {dnorm_weight, col, false},
                      {dnext_weight, col, false},
                      {gated ? dgate : nullptr, dgate_bytes, element},
                      {workspace, need, false}},
                     {{dout, bytes, true},
                      {dnormed, bytes, true},
                      {branch, bytes, true},
                      {joined, bytes, true},
                      {p->norm_weight, vector_bytes(p, H), false},
                      {p->next_weight, vector_bytes(p, H), false},
                      gate_range(p, dtype, T, H)});
  if (st != MOE_OK) return st;
  if (T == 0 && branch == nullptr) branch = workspace;   // not read: only says that the join has a branch
  const int arrays = (p->norm_weight != nullptr) + (p->gate_kind == MOE_GATE_CHANNEL) + next;
  const moe::JoinBackwardArgs a{dout, dnormed, branch, joined, p->norm_weight, p->next_weight, p->gate, dbranch,
                                dresidual, dgate, static_cast<float*>(workspace), T, static_cast<int>(H), p->gate_kind,
                                p->vec_dtype == MOE_F32, arrays, p->residual_scale, p->branch_scale, p->eps,
                                nullptr};
  const cudaError_t err =
      moe::launch_join_backward(dtype, a, dnorm_weight, dnext_weight, static_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return api_cuda_fail(err, "moe_block_join_backward launch");
  return api_ok();
}

}  // extern "C"
