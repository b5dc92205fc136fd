// Expanded latent attention, forward: a wavefront a query row, 64 keys at a
// time with the running maximum and sum of the softmax.

#include <math.h>

#include "mla_simple.h"

namespace mla {
namespace {

template <int DN, int DR>
__global__ __launch_bounds__(64) void fwd_kernel(AttnArgs a) {
  constexpr int DQ = DN + DR;
  const int i = blockIdx.x, h = blockIdx.y, lane = threadIdx.x;
  int begin, end;
  if (!token_document(a, i, begin, end)) return;
  const long long row = (long long)i * a.H + h;
  const bf16* q = a.q + row * DQ;
  __shared__ float p[64];
  float m = -INFINITY, l = 0.f, acc[DN / 64] = {};
  for (int j0 = begin; j0 <= i; j0 += 64) {
    const int j = j0 + lane;
    float s = -INFINITY;
    if (j <= i) {
      s = dot(q, a.kv + ((long long)j * a.H + h) * (2 * DN), DN);
      if (DR) s += dot(q + DN, a.k_pe + (long long)j * DR, DR);
      s *= a.scale;
    }
    const float mx = fmaxf(m, wave_max(s));
    const float at = mx == -INFINITY ? 0.f : mx;  // the maximum passes over NaN
    const float c = expf(m - at), e = expf(s - at);
    m = mx;
    l = l * c + wave_sum(e);
    __syncthreads();
    p[lane] = e;
    __syncthreads();
    for (int d = 0; d < DN / 64; ++d) acc[d] *= c;
    for (int t = 0; t < 64 && j0 + t <= i; ++t)
      for (int d = 0; d < DN / 64; ++d)
        acc[d] += p[t] * (float)a.kv[((long long)(j0 + t) * a.H + h) * (2 * DN) + DN + d * 64 + lane];
  }
  for (int d = 0; d < DN / 64; ++d) a.o[row * DN + d * 64 + lane] = (bf16)(acc[d] / l);
  if (a.lse && lane == 0) a.lse[row] = m + logf(l);
}

template <int DN, int DR>
hipError_t launch(const AttnArgs& a, hipStream_t stream) {
  fwd_kernel<DN, DR><<<dim3(a.tokens, a.H), dim3(64), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_fwd(int Dn, int Dr, const AttnArgs& a, hipStream_t stream) {
  if (Dn == 64) return Dr ? launch<64, 64>(a, stream) : launch<64, 0>(a, stream);
  return Dr ? launch<128, 64>(a, stream) : launch<128, 0>(a, stream);
}

}  // namespace mla
