// Expanded latent attention, backward: a wavefront a query row for dq, a
// wavefront a key row for dk and dv, 64 partners at a time.
//
//   p = exp(s - lse), dp = do v^T, ds = p (dp - <do, o>)
//   dq = scale ds k, dk = scale ds^T q, dv = p^T do

#include <math.h>

#include "mla_simple.h"

namespace mla {
namespace {

template <int DN, int DR>
__device__ __forceinline__ float score(const AttnArgs& a, int i, int j, int h) {
  const bf16* q = a.q + ((long long)i * a.H + h) * (DN + DR);
  float s = dot(q, a.kv + ((long long)j * a.H + h) * (2 * DN), DN);
  if (DR) s += dot(q + DN, a.k_pe + (long long)j * DR, DR);
  return s * a.scale;
}

template <int DN, int DR>
__global__ __launch_bounds__(64) void dq_kernel(AttnArgs a) {
  constexpr int DQ = DN + DR;
  const int i = blockIdx.x, h = blockIdx.y, lane = threadIdx.x;
  int begin, end;
  if (!token_document(a, i, begin, end)) return;
  const long long row = (long long)i * a.H + h;
  float dl = 0.f;
  for (int d = lane; d < DN; d += 64) dl += (float)a.o_in[row * DN + d] * (float)a.dout[row * DN + d];
  dl = wave_sum(dl);
  if (lane == 0) a.delta[row] = dl;
  __shared__ float ds[64];
  float acc[DQ / 64] = {};
  for (int j0 = begin; j0 <= i; j0 += 64) {
    const int j = j0 + lane;
    float x = 0.f;
    if (j <= i) {
      const float p = expf(score<DN, DR>(a, i, j, h) - a.lse[row]);
      x = p * (dot(a.dout + row * DN, a.kv + ((long long)j * a.H + h) * (2 * DN) + DN, DN) - dl) * a.scale;
    }
    __syncthreads();
    ds[lane] = x;
    __syncthreads();
    for (int t = 0; t < 64 && j0 + t <= i; ++t)
      for (int d = 0; d < DQ / 64; ++d) {
        const int c = d * 64 + lane;
        const bf16* k = c < DN ? a.kv + ((long long)(j0 + t) * a.H + h) * (2 * DN) + c
                               : a.k_pe + (long long)(j0 + t) * DR + c - DN;
        acc[d] += ds[t] * (float)*k;
      }
  }
  for (int d = 0; d < DQ / 64; ++d) a.dq[row * DQ + d * 64 + lane] = (bf16)acc[d];
}

template <int DN, int DR>
__global__ __launch_bounds__(64) void dkv_kernel(AttnArgs a) {
  constexpr int DQ = DN + DR;
  const int j = blockIdx.x, h = blockIdx.y, lane = threadIdx.x;
  int begin, end;
  if (!token_document(a, j, begin, end)) return;
  const long long col = (long long)j * a.H + h;
  __shared__ float ds[64], ps[64];
  float dk[DQ / 64] = {}, dv[DN / 64] = {};
  for (int i0 = j; i0 < end; i0 += 64) {
    const int i = i0 + lane;
    float x = 0.f, p = 0.f;
    if (i < end) {
      const long long row = (long long)i * a.H + h;
      p = expf(score<DN, DR>(a, i, j, h) - a.lse[row]);
      x = p * (dot(a.dout + row * DN, a.kv + col * (2 * DN) + DN, DN) - a.delta[row]) * a.scale;
    }
    __syncthreads();
    ds[lane] = x;
    ps[lane] = p;
    __syncthreads();
    for (int t = 0; t < 64 && i0 + t < end; ++t) {
      const long long row = (long long)(i0 + t) * a.H + h;
      for (int d = 0; d < DQ / 64; ++d) dk[d] += ds[t] * (float)a.q[row * DQ + d * 64 + lane];
      for (int d = 0; d < DN / 64; ++d) dv[d] += ps[t] * (float)a.dout[row * DN + d * 64 + lane];
    }
  }
  for (int d = 0; d < DN / 64; ++d) {
    a.dkv[col * (2 * DN) + d * 64 + lane] = (bf16)dk[d];
    a.dkv[col * (2 * DN) + DN + d * 64 + lane] = (bf16)dv[d];
  }
  if (DR) a.pe_part[((long long)h * a.tokens + j) * DR + lane] = dk[DQ / 64 - 1];
}

// Sum of the heads' shares of dk_pe, in head order.
__global__ __launch_bounds__(64) void pe_kernel(AttnArgs a, int DR) {
  const int j = blockIdx.x;
  int begin, end;
  if (!token_document(a, j, begin, end)) return;
  float s = 0.f;
  for (int h = 0; h < a.H; ++h) s += a.pe_part[((long long)h * a.tokens + j) * DR + threadIdx.x];
  a.dk_pe[(long long)j * DR + threadIdx.x] = (bf16)s;
}

template <int DN, int DR>
hipError_t launch(const AttnArgs& a, hipStream_t stream) {
  const dim3 grid(a.tokens, a.H);
  dq_kernel<DN, DR><<<grid, dim3(64), 0, stream>>>(a);
  dkv_kernel<DN, DR><<<grid, dim3(64), 0, stream>>>(a);
  if (DR) pe_kernel<<<dim3(a.tokens), dim3(DR), 0, stream>>>(a, DR);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_bwd(int Dn, int Dr, const AttnArgs& a, hipStream_t stream) {
  if (Dn == 64) return Dr ? launch<64, 64>(a, stream) : launch<64, 0>(a, stream);
  return Dr ? launch<128, 64>(a, stream) : launch<128, 0>(a, stream);
}

}  // namespace mla
