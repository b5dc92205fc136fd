// Expanded latent attention, forward, causal, one pass over the keys.
//
// A workgroup takes 128 queries of a head, 32 a wavefront, and goes through
// the keys they see 64 at a time: S^T = K Q^T (the queries are B operands in
// registers), the softmax's running maximum and sum a query a lane, then
// O^T += V^T P^T, P from the accumulators of S^T without leaving the lane.
// Keys and values go from memory straight into LDS, the next tile during a
// tile; two workgroups a CU (2 x 80 KB of LDS at 128 / 64 channels) keep the
// matrix units busy during the other's softmax.
// Sums and statistics are float32; P is rounded to bf16 as an operand, the row
// sum is taken before that.
// B1 T16384 H12 128/64: 0.95 to 1.04 ms by GPU, 990 to 1,090 TFLOP/s, a large
// bf16 matrix product reaching 1,551; T4096 H96: 0.55 ms.  The matrix units are busy 53 to 61% of
// the time; the rest is the softmax's vector work.  Before the next tile's
// scores were formed beside the weights: 1.11 ms.

#include <math.h>

#include "mla_tile.h"

namespace mla {
namespace {

constexpr int kQ = 128, kK = 64;  // queries of a workgroup, keys of a tile

template <int DN, int DR>
__global__ __launch_bounds__(256, 2) void fwd_kernel(AttnArgs a, TileMap map) {
  constexpr int DQ = DN + DR;
  constexpr unsigned kKey = kK * DN * 2, kRot = kK * DR * 2;  // bytes of a tile's parts: keys, values, rotary keys
  __shared__ __align__(1024) char lds[2 * (2 * kKey + kRot)];  // keys of 2 tiles, values of 2
  int h, len, q0;
  long long t0;
  if (!tile_place<kQ>(a, map, true, h, t0, len, q0)) return;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w0 = q0 + wave * 32;
  const int qi = w0 + (lane & 31);  // this lane's query
  const int keys = min(len, q0 + kQ);
  const bf16* kv = a.kv + (t0 * a.H + h) * (2 * DN);
  const bf16* pe = a.k_pe + t0 * DR;
  const unsigned base = lds_address(lds);
  const LaneAt<DN> at(lane);
  const LaneAt<64> at_rot(lane);

  bf16x8 qf[DQ / 16];
#pragma unroll
  for (int s = 0; s < DQ / 16; ++s) {
    qf[s] = bf16x8{};
    if (qi < len) qf[s] = row_frag(a.q + ((t0 + qi) * a.H + h) * DQ, s, half);
  }
  // A tile's keys are needed a tile before its values.
  constexpr unsigned kTileKey = kKey + kRot;
  auto fetch_keys = [&](int t) {
    const unsigned to = base + (t & 1) * kTileKey;
    const long long j0 = (long long)t * kK;
    fetch_rows<kK, DN>(kv + j0 * (a.H * 2 * DN), a.H * 2 * DN, (int)(len - 1 - j0), to, wave, lane);
    if constexpr (DR > 0) fetch_rows<kK, DR>(pe + j0 * DR, DR, (int)(len - 1 - j0), to + kKey, wave, lane);
  };
  auto fetch_values = [&](int t) {
    const long long j0 = (long long)t * kK;
    fetch_rows<kK, DN>(kv + j0 * (a.H * 2 * DN) + DN, a.H * 2 * DN, (int)(len - 1 - j0),
                       base + 2 * kTileKey + (t & 1) * kKey, wave, lane);
  };
  auto scores = [&](int t, f32x16* s) {
    const unsigned ks = base + (t & 1) * kTileKey, rs = ks + kKey;
    s[0] = s[1] = f32x16{};
#pragma unroll
    for (int k = 0; k < DN / 16; ++k)
#pragma unroll
      for (int u = 0; u < 2; ++u) s[u] = mma(row_frag(ks, at, 32 * u, k), qf[k], s[u]);
#pragma unroll
    for (int k = 0; k < DR / 16; ++k)
#pragma unroll
      for (int u = 0; u < 2; ++u) s[u] = mma(row_frag(rs, at_rot, 32 * u, k), qf[DN / 16 + k], s[u]);
  };

  f32x16 acc[DN / 32] = {}, s[2];
  float m = -FLT_MAX, l = 0.f;  // running maximum of the scaled scores in log2 units; this lane's half of the sum
  const float c = a.scale * kda::kLog2e;
  const int tiles = (keys + kK - 1) / kK;
  constexpr int kLoads = (2 * kKey + kRot) / 4096;  // a wavefront's share of a tile's keys and values
  fetch_keys(0);
  if (tiles > 1) fetch_keys(1);
  fetch_values(0);
  if (tiles > 1)
    tile_barrier<kLoads>();
  else
    tile_barrier<kKey / 4096>();
  scores(0, s);
  for (int t = 0; t < tiles; ++t) {
    const int j0 = t * kK;
    tile_barrier<0>();  // these values and the next keys are there, and all are done with the tile before
    if (t + 2 < tiles) fetch_keys(t + 2);
    if (t + 1 < tiles) fetch_values(t + 1);
    if (j0 > w0 + 31) continue;  // all of it is past this wavefront's queries
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
    // The next tile's scores are formed beside this tile's weights, so that
    // matrix and vector work overlap (after the last tile: of what is there,
    // and not used).
    f32x16 s1[2];
    scores(t + 1, s1);
    const unsigned vs = base + 2 * kTileKey + (t & 1) * kKey;
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
        for (int d = 0; d < DN / 32; ++d) acc[d] = mma(tr_frag(vs, at, 32 * u + 16 * k, d), pf, acc[d]);
      }
    }
    s[0] = s1[0];
    s[1] = s1[1];
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
