// A long sum of rounds' sums, mostly in FP32: 16 of them are added in FP32, then
// go into FP64, of which the SMs have little. Against the exact sum of positive
// terms: a round's own additions, then at most 16 roundings of 2^-24 of it,
// whatever the number of rounds and their sizes.
//
// No CUDA header: a host test compiles this file alone.
#pragma once

#if defined(__CUDACC__)
#define MOE_SUM_FN __device__ __forceinline__
#else
#define MOE_SUM_FN inline
#endif

namespace moe {

struct RoundSums {
  static constexpr int NEAR = 16;
  float near = 0.0f;   // what is not in far yet
  double far = 0.0;
  int rounds = 0;

  MOE_SUM_FN void add(float sum) {
    near += sum;
    if (++rounds == NEAR) {
      far += near;
      near = 0.0f;
      rounds = 0;
    }
  }
};

}  // namespace moe
