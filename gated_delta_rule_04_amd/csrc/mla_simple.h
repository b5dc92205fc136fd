// One wavefront's share of a softmax-weighted sum, the simplest form: 64 keys
// at a time, a key a lane for the scores, a channel a lane for the sums.
#pragma once

#include "mla_launch.h"

namespace mla {

__device__ __forceinline__ float wave_sum(float x) {
  for (int m = 32; m; m >>= 1) x += __shfl_xor(x, m);
  return x;
}
__device__ __forceinline__ float wave_max(float x) {
  for (int m = 32; m; m >>= 1) x = fmaxf(x, __shfl_xor(x, m));
  return x;
}
__device__ __forceinline__ float dot(const bf16* a, const bf16* b, int n) {
  float s = 0.f;
  for (int i = 0; i < n; ++i) s += (float)a[i] * (float)b[i];
  return s;
}

// Document of token i (counted through the batch); false for padding.
__device__ __forceinline__ bool token_document(const AttnArgs& a, int i, int& begin, int& end) {
  int n;
  if (a.cu) {
    int lo = 0, hi = a.N;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.cu[mid] <= i) lo = mid; else hi = mid;
    }
    n = lo;
  } else {
    n = i / a.T;
  }
  document(a.cu, a.T, n, begin, end);
  return i >= begin && i < end;
}

}  // namespace mla
