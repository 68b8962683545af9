// C ABI of the gradient norm and clipping (contracts in include/moe.h).
#include <algorithm>
#include <limits>
#include <vector>

#include "moe_common.cuh"
#include "moe_internal.h"

using moe::api_cuda_fail;
using moe::api_fail;
using moe::api_ok;

namespace {

moe_status check_tensors(const moe_grad_tensor* t, int64_t n, bool with_dst) {
  if (n < 0 || n > (int64_t{1} << 24)) return api_fail(MOE_ERR_SHAPE, "n must be in 0 .. 2^24");
  if (n > 0 && t == nullptr) return api_fail(MOE_ERR_NULL, "tensors must be non-NULL");
  for (int64_t i = 0; i < n; ++i) {
    if (!moe::dtype_valid(t[i].dtype)) return api_fail(MOE_ERR_DTYPE, "gradient dtype must be F32, F16 or BF16");
    if (t[i].numel < 0 || t[i].numel > (int64_t{1} << 46)) return api_fail(MOE_ERR_SHAPE, "numel must be >= 0");
    if (t[i].numel == 0) continue;
    if (t[i].src == nullptr || (with_dst && t[i].dst == nullptr))
      return api_fail(MOE_ERR_NULL, "gradient pointers must be non-NULL");
    const uintptr_t es = moe::dtype_size(static_cast<moe_dtype>(t[i].dtype));
    if (reinterpret_cast<uintptr_t>(t[i].src) % es != 0 ||
        (with_dst && reinterpret_cast<uintptr_t>(t[i].dst) % es != 0))
      return api_fail(MOE_ERR_ALIGNMENT, "gradients must be aligned to their element size");
  }
  return MOE_OK;
}

// No written range overlaps any other range (an in-place entry is one range),
// nor the norm, which blocks still read while others write.
moe_status check_overlap(const moe_grad_tensor* t, int64_t n, const float* norm) {
  struct Range {
    uintptr_t lo, hi;
    bool written;
  };
  const uintptr_t norm_lo = reinterpret_cast<uintptr_t>(norm), norm_hi = norm_lo + sizeof(float);
  try {
    std::vector<Range> r;
    r.reserve(static_cast<size_t>(2 * n));
    for (int64_t i = 0; i < n; ++i) {
      if (t[i].numel == 0) continue;
      const uintptr_t bytes =
          static_cast<uintptr_t>(t[i].numel) * moe::dtype_size(static_cast<moe_dtype>(t[i].dtype));
      const uintptr_t d = reinterpret_cast<uintptr_t>(t[i].dst), s = reinterpret_cast<uintptr_t>(t[i].src);
      if (norm_lo < d + bytes && d < norm_hi) return api_fail(MOE_ERR_SHAPE, "norm lies in a dst");
      r.push_back({d, d + bytes, true});
      if (s != d) r.push_back({s, s + bytes, false});
    }
    std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    uintptr_t hi_any = 0, hi_written = 0;  // ends of the ranges so far
    for (const Range& x : r) {
      if (x.lo < hi_written || (x.written && x.lo < hi_any))
        return api_fail(MOE_ERR_SHAPE, "a dst overlaps another gradient");
      hi_any = std::max(hi_any, x.hi);
      if (x.written) hi_written = std::max(hi_written, x.hi);
    }
  } catch (...) {
    return api_fail(MOE_ERR_WORKSPACE, "no host memory for the overlap check");
  }
  return MOE_OK;
}

moe_status device_sms(int* sms) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess) err = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return err == cudaSuccess ? MOE_OK : api_cuda_fail(err, "device query");
}

}  // namespace

extern "C" {

size_t moe_grad_norm_workspace_size(int64_t n) { return n < 0 ? 0 : moe::grad_norm_scratch_bytes(n); }

moe_status moe_grad_norm(const moe_grad_tensor* tensors, int64_t n, float* norm, void* workspace,
                         size_t workspace_bytes, void* stream) {
  moe_status st = check_tensors(tensors, n, false);
  if (st != MOE_OK) return st;
  if (norm == nullptr) return api_fail(MOE_ERR_NULL, "norm must be non-NULL");
  if (reinterpret_cast<uintptr_t>(norm) % 4 != 0) return api_fail(MOE_ERR_ALIGNMENT, "norm must be 4-byte aligned");
  if (workspace == nullptr || workspace_bytes < moe::grad_norm_scratch_bytes(n))
    return api_fail(MOE_ERR_WORKSPACE, "workspace smaller than moe_grad_norm_workspace_size()");
  if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
    return api_fail(MOE_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  int sms = 0;
  st = device_sms(&sms);
  if (st != MOE_OK) return st;
  const cudaError_t err =
      moe::launch_grad_norm(tensors, n, norm, workspace, sms, static_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return api_cuda_fail(err, "moe_grad_norm launch");
  return api_ok();
}

moe_status moe_grad_clip(const moe_grad_tensor* tensors, int64_t n, const float* norm, float max_norm, void* stream) {
  moe_status st = check_tensors(tensors, n, true);
  if (st != MOE_OK) return st;
  if (!(max_norm >= 0.0f) || !(max_norm <= std::numeric_limits<float>::max()))
    return api_fail(MOE_ERR_SHAPE, "max_norm must be finite and >= 0");
  if (norm == nullptr) return api_fail(MOE_ERR_NULL, "norm must be non-NULL");
  if (reinterpret_cast<uintptr_t>(norm) % 4 != 0) return api_fail(MOE_ERR_ALIGNMENT, "norm must be 4-byte aligned");
  st = check_overlap(tensors, n, norm);
  if (st != MOE_OK) return st;
  int sms = 0;
  st = device_sms(&sms);
  if (st != MOE_OK) return st;
  const cudaError_t err =
      moe::launch_grad_clip(tensors, n, norm, max_norm, sms, static_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return api_cuda_fail(err, "moe_grad_clip launch");
  return api_ok();
}

}  // extern "C"
