// Absorbed latent attention over the paged cache: a wavefront a query row,
// 64 cache rows at a time with the running maximum and sum of the softmax.

#include <math.h>

#include "mla_simple.h"

namespace mla {
namespace {

template <int R, int DR>
__global__ __launch_bounds__(64) void paged_kernel(PagedArgs a) {
  constexpr int D = R + DR;
  const int i = blockIdx.x, h = blockIdx.y, lane = threadIdx.x;
  // sequence of query row i: the last n with cu[n] <= i
  int n = i, first = i, last = i + 1;
  if (a.cu) {
    int lo = 0, hi = a.N;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.cu[mid] <= i) lo = mid; else hi = mid;
    }
    n = lo;
    document(a.cu, a.Tq, n, first, last);
    if (i < first || i >= last) return;
  }
  const int L = min(max(a.lens[n], 0), a.max_pages * a.page_size);
  const int end = min(L, L - (last - i) + 1);
  const long long row = (long long)i * a.H + h;
  const bf16* q = a.q + row * D;
  __shared__ float p[64];
  __shared__ const bf16* rows[64];
  float m = -INFINITY, l = 0.f, acc[R / 64] = {};
  for (int j0 = 0; j0 < end; j0 += 64) {
    const int j = j0 + lane;
    const bf16* k = nullptr;
    if (j < end) {
      const int page = a.table[(long long)n * a.max_pages + j / a.page_size];
      if ((unsigned)page < (unsigned)a.num_pages)
        k = a.cache + ((long long)page * a.page_size + j % a.page_size) * D;
    }
    const float s = k ? dot(q, k, D) * a.scale : -INFINITY;
    const float mx = fmaxf(m, wave_max(s));
    const float at = mx == -INFINITY ? 0.f : mx;  // nothing but masked rows (or NaN, which the maximum passes over)
    const float c = expf(m - at), e = k ? expf(s - at) : 0.f;
    m = mx;
    l = l * c + wave_sum(e);
    __syncthreads();
    p[lane] = e;
    rows[lane] = k;
    __syncthreads();
    for (int d = 0; d < R / 64; ++d) acc[d] *= c;
    for (int t = 0; t < 64; ++t) {
      if (!rows[t]) continue;
      for (int d = 0; d < R / 64; ++d) acc[d] += p[t] * (float)rows[t][d * 64 + lane];
    }
  }
  for (int d = 0; d < R / 64; ++d) a.o[row * R + d * 64 + lane] = (bf16)(l > 0.f || l != l ? acc[d] / l : 0.f);
  if (a.lse && lane == 0) a.lse[row] = l > 0.f || l != l ? (m == -INFINITY ? 0.f : m) + logf(l) : -INFINITY;
}

template <int R, int DR>
hipError_t launch(const PagedArgs& a, hipStream_t stream) {
  paged_kernel<R, DR><<<dim3(a.Tq, a.H), dim3(64), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t paged_workspace(int, int, int, int, int, long long) { return 0; }

hipError_t launch_paged(int R, int Dr, const PagedArgs& a, hipStream_t stream) {
  switch (R + Dr) {
    case 128: return launch<128, 0>(a, stream);
    case 192: return launch<128, 64>(a, stream);
    case 256: return launch<256, 0>(a, stream);
    case 320: return launch<256, 64>(a, stream);
    case 512: return launch<512, 0>(a, stream);
    case 576: return launch<512, 64>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace mla
