// Expanded latent attention, forward, causal, one pass over the keys.
//
// A workgroup takes 128 queries of a head, 32 a wavefront, and goes through
// the keys they see 64 at a time: S^T = K Q^T (the queries are B operands in
// registers), the softmax's running maximum and sum a query a lane, then
// O^T += V^T P^T, P from the accumulators of S^T without leaving the lane.
// Sums and statistics are float32; P is rounded to bf16 as an operand, the row
// sum is taken before that.

#include <math.h>

#include "mla_tile.h"

namespace mla {
namespace {

constexpr int kQ = 128, kK = 64;  // queries of a workgroup, keys of a tile

template <int DN, int DR>
__global__ __launch_bounds__(256, 2) void fwd_kernel(AttnArgs a, TileMap map) {
  constexpr int DQ = DN + DR, KP = DQ + kPad, VP = DN + kPad;
  constexpr int kKv = 2 * DN / 8, kPe = DR / 8;             // 16-byte pieces of a row
  constexpr int nKv = kK * kKv / 256, nPe = kK * kPe / 256;  // pieces a thread
  __shared__ __align__(16) bf16 ks[kK * KP];
  __shared__ __align__(16) bf16 vs[kK * VP];
  int h, len, q0;
  long long t0;
  if (!tile_place<kQ>(a, map, true, h, t0, len, q0)) return;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, w0 = q0 + (tid >> 6) * 32;
  const int qi = w0 + (lane & 31);  // this lane's query
  const int keys = min(len, q0 + kQ);
  const bf16* kv = a.kv + (t0 * a.H + h) * (2 * DN);
  const bf16* pe = a.k_pe + t0 * DR;

  bf16x8 qf[DQ / 16];
#pragma unroll
  for (int s = 0; s < DQ / 16; ++s) {
    qf[s] = bf16x8{};
    if (qi < len) qf[s] = row_frag(a.q + ((t0 + qi) * a.H + h) * DQ, s, half);
  }
  u32x4 rkv[nKv], rpe[nPe ? nPe : 1];
  auto load = [&](int j0) {
#pragma unroll
    for (int p = 0; p < nKv; ++p) {
      const int row = (p * 256 + tid) / kKv, c = (p * 256 + tid) % kKv;
      rkv[p] = u32x4{};
      if (j0 + row < len) rkv[p] = *(const u32x4*)(kv + (long long)j0 * (a.H * 2 * DN) + row * (a.H * 2 * DN) + c * 8);
    }
    if constexpr (DR > 0) {
#pragma unroll
      for (int p = 0; p < nPe; ++p) {
        const int row = (p * 256 + tid) / kPe, c = (p * 256 + tid) % kPe;
        rpe[p] = u32x4{};
        if (j0 + row < len) rpe[p] = *(const u32x4*)(pe + (long long)(j0 + row) * DR + c * 8);
      }
    }
  };
  auto store = [&]() {
#pragma unroll
    for (int p = 0; p < nKv; ++p) {
      const int row = (p * 256 + tid) / kKv, c = (p * 256 + tid) % kKv;
      *(u32x4*)(c < DN / 8 ? ks + row * KP + c * 8 : vs + row * VP + (c - DN / 8) * 8) = rkv[p];
    }
    if constexpr (DR > 0) {
#pragma unroll
      for (int p = 0; p < nPe; ++p)
        *(u32x4*)(ks + ((p * 256 + tid) / kPe) * KP + DN + ((p * 256 + tid) % kPe) * 8) = rpe[p];
    }
  };

  f32x16 acc[DN / 32] = {};
  float m = -FLT_MAX, l = 0.f;  // running maximum of the scaled scores in log2 units; this lane's half of the sum
  const float c = a.scale * kda::kLog2e;
  load(0);
  for (int j0 = 0; j0 < keys; j0 += kK) {
    __syncthreads();
    store();
    __syncthreads();
    if (j0 + kK < keys) load(j0 + kK);
    if (j0 > w0 + 31) continue;  // all of it is past this wavefront's queries
    f32x16 s[2] = {};
#pragma unroll
    for (int k = 0; k < DQ / 16; ++k)
#pragma unroll
      for (int u = 0; u < 2; ++u) s[u] = mma(row_frag(ks + (32 * u + (lane & 31)) * KP, k, half), qf[k], s[u]);
    if (j0 + kK - 1 > w0) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (j0 + 32 * u + acc_row(i, half) > qi) s[u][i] = -INFINITY;
    }
    float mx = -INFINITY;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[u][i]);
    mx = halves_max(mx) * c;
    // The sums keep their reference while the maximum rises by less than 2^8:
    // the weights stay far inside float32 and bf16 keeps its relative step.
    if (__any(mx > m + 8.f)) {
      const float mn = fmaxf(m, mx), f = kda::fast_exp2(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int d = 0; d < DN / 32; ++d) acc[d] *= f;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[u][i] = kda::fast_exp2(__builtin_fmaf(s[u][i], c, -m));
        l += s[u][i];
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bf16x8 pf = acc_frag(s[u], k);
#pragma unroll
        for (int d = 0; d < DN / 32; ++d) acc[d] = mma(tr_frag<VP>(vs, 32 * u + 16 * k, 32 * d, lane), pf, acc[d]);
      }
    }
  }
  l = halves_sum(l);
  if (qi >= len) return;
  const long long row = (t0 + qi) * a.H + h;
  const float r = l == 0.f ? 0.f : 1.f / l;  // 0: every score was -infinity
#pragma unroll
  for (int d = 0; d < DN / 32; ++d)
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *(u32x2*)(a.o + row * DN + 32 * d + acc_row(i, half)) =
          u32x2{kda::pk_bf16(acc[d][i] * r, acc[d][i + 1] * r), kda::pk_bf16(acc[d][i + 2] * r, acc[d][i + 3] * r)};
  if (a.lse && half == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * (1.f / kda::kLog2e);
}

template <int DN, int DR>
hipError_t launch(const AttnArgs& a, hipStream_t stream) {
  const TileMap map = tile_map<kQ>(a);
  fwd_kernel<DN, DR><<<dim3((unsigned)map.blocks()), dim3(256), 0, stream>>>(a, map);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_fwd(int Dn, int Dr, const AttnArgs& a, hipStream_t stream) {
  if (Dn == 64) return Dr ? launch<64, 64>(a, stream) : launch<64, 0>(a, stream);
  return Dr ? launch<128, 64>(a, stream) : launch<128, 0>(a, stream);
}

}  // namespace mla
