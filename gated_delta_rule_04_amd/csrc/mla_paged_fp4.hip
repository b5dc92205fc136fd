// Absorbed latent attention over the paged 4-bit cache: one wavefront a row of
// queries, the cache rows one after the other, float32.

#include <float.h>
#include <math.h>

#include "mla_fp4.h"

namespace mla {
namespace {

template <int R, int DR>
__global__ __launch_bounds__(256) void paged_fp4_kernel(PagedArgs a) {
  constexpr int kRow = fp4_row_bytes(R, DR), kPer = R / 64;  // channels a lane
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (row >= (long long)a.Tq * a.H) return;
  const int token = (int)(row / a.H);
  int n = token, first = token, last = token + 1;
  if (a.cu) {
    if (token >= min(max(a.cu[a.N], 0), a.Tq)) return;
    int lo = 0, hi = a.N;
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2;
      if (min(max(a.cu[mid], 0), a.Tq) <= token)
        lo = mid;
      else
        hi = mid;
    }
    n = lo;
    document(a.cu, a.Tq, n, first, last);
  }
  const int L = min(max(a.lens[n], 0), a.max_pages * a.page_size);
  const int sees = min(L - (last - first) + (token - first) + 1, L);
  const bf16* q = a.q + row * (R + DR);
  float qv[kPer], qr = DR ? (float)q[R + lane] : 0.f, acc[kPer] = {}, m = -FLT_MAX, l = 0.f;
  for (int i = 0; i < kPer; ++i) qv[i] = (float)q[lane * kPer + i];
  for (int j = 0; j < sees; ++j) {
    const int page = a.table[(long long)n * a.max_pages + j / a.page_size];
    if ((unsigned)page >= (unsigned)a.num_pages) continue;
    const unsigned char* c = a.cache4 + ((long long)page * a.page_size + j % a.page_size) * kRow;
    unsigned codes = 0;
    for (int i = 0; i < kPer / 2; ++i) codes |= (unsigned)c[lane * kPer / 2 + i] << (8 * i);
    const u32x4 v = fp4_values(codes, __builtin_bit_cast(float, (unsigned)c[R / 2 + 2 * DR + lane * kPer / 32] << 23));
    float x[kPer], s = DR ? qr * (float)((const bf16*)(c + R / 2))[lane] : 0.f;
    for (int i = 0; i < kPer; ++i) {
      x[i] = __builtin_bit_cast(float, i % 2 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
      s += qv[i] * x[i];
    }
    for (int k = 1; k < 64; k <<= 1) s += __shfl_xor(s, k);
    s *= a.scale * kda::kLog2e;
    const float mn = fmaxf(m, s), f = kda::fast_exp2(m - mn), p = kda::fast_exp2(s - mn);
    m = mn;
    l = l * f + p;
    for (int i = 0; i < kPer; ++i) acc[i] = acc[i] * f + p * x[i];
  }
  const float r = l == 0.f ? 0.f : 1.f / l;
  for (int i = 0; i < kPer; ++i) a.o[row * R + lane * kPer + i] = (bf16)(acc[i] * r);
  if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * (1.f / kda::kLog2e);
}

template <int R, int DR>
hipError_t launch(const PagedArgs& a, hipStream_t stream) {
  const long long rows = (long long)a.Tq * a.H;
  paged_fp4_kernel<R, DR><<<dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t paged_fp4_workspace(int, int, int, int, int, long long) { return 0; }

hipError_t launch_paged_fp4(int R, int Dr, const PagedArgs& a, hipStream_t stream) {
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
