// Expanded latent attention, backward, causal.
//
//   p = exp(s - lse), dp = do v^T, ds = p (dp - delta), delta = <do, o> = sum_j p dp
//   dq = scale ds k, dk = scale ds^T q, dv = p^T do
//
// Three passes, so that no sum needs atomics: delta_kernel and dq_kernel go along
// the keys of 128 queries, dkv_kernel along the queries of 128 keys.  Each forms
// s and dp again (9 products in all where one pass over saved deltas has 5; a
// pass over both directions would add dq in an order that changes from run to
// run, or keep it in a workspace of float32 tiles).  p and ds are rounded to
// bf16 as operands; sums are float32.
// B1 T16384 H12 128/64: delta 0.89 to 0.93 ms by GPU (three workgroups a CU,
// matrix units 70% busy; tiles of 64 keys at two a CU 1.07), dq 1.51 to 1.57 ms
// (57%), dk and dv 2.2 to 2.6 ms (39%: the sums and operands of 32 keys are 339
// registers, so one wavefront a SIMD; a fifth more before the next tile's scores
// were formed beside the weights), dk_pe's sum 9 us.

#include <math.h>

#include "mla_tile.h"

namespace mla {
namespace {

constexpr int kRows = 128;  // queries (or keys) of a workgroup, 32 a wavefront
constexpr int kK = 32;      // keys of a tile of the delta and dq kernels
constexpr int kI = 32;      // queries of a tile of the dk, dv kernel

// Tiles of kK keys of a head: keys, values and rotary keys one after another.
template <int DN, int DR>
struct KeyTiles {
  static constexpr unsigned kKey = kK * DN * 2;
  const bf16 *kv, *pe;
  int ld, len;
  __device__ __forceinline__ KeyTiles(const AttnArgs& a, long long t0, int h, int len)
      : kv(a.kv + (t0 * a.H + h) * (2 * DN)), pe(a.k_pe + t0 * DR), ld(a.H * 2 * DN), len(len) {}
  __device__ __forceinline__ void fetch(int j0, unsigned to, int wave, int lane) const {
    const bf16* from = kv + (long long)j0 * ld;
    fetch_rows<kK, DN>(from, ld, len - 1 - j0, to, wave, lane);
    fetch_rows<kK, DN>(from + DN, ld, len - 1 - j0, to + kKey, wave, lane);
    if constexpr (DR > 0) fetch_rows<kK, DR>(pe + (long long)j0 * DR, DR, len - 1 - j0, to + 2 * kKey, wave, lane);
  }
};

// Each query's log-sum-exp in log2 units and its delta, for the two kernels
// after it: delta = sum_j p dp in float32, along the keys of 128 queries.  The
// rounded o would be at hand, but <do, o> carries its rounding as one term in
// all of a row's ds; where a row attends to few keys, p (dp - delta) is small
// beside that term, and dq mostly rounding (scores of standard deviation 8: a
// row's dq off by 65% at the 95th percentile, by 0.3% with this sum).
template <int DN, int DR>
__global__ __launch_bounds__(256, 2) void delta_kernel(AttnArgs a, TileMap map) {
  constexpr int DQ = DN + DR;
  constexpr unsigned kKey = kK * DN * 2, kRot = kK * DR * 2;  // bytes of a tile's parts: keys, values, rotary keys
  __shared__ __align__(1024) char lds[2][2 * kKey + kRot];
  int h, len, q0;
  long long t0;
  if (!tile_place<kRows>(a, map, true, h, t0, len, q0)) return;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w0 = q0 + wave * 32;
  const int qi = w0 + (lane & 31);
  const int keys = min(len, q0 + kRows);
  const long long row = (t0 + qi) * a.H + h;
  const bool on = qi < len;

  bf16x8 qf[DQ / 16], df[DN / 16];
#pragma unroll
  for (int s = 0; s < DQ / 16; ++s) qf[s] = on ? row_frag(a.q + row * DQ, s, half) : bf16x8{};
#pragma unroll
  for (int s = 0; s < DN / 16; ++s) df[s] = on ? row_frag(a.dout + row * DN, s, half) : bf16x8{};
  const float lse = on ? a.lse[row] * kda::kLog2e : 0.f;
  const float c = a.scale * kda::kLog2e;

  const unsigned base = lds_address(&lds[0][0]);
  const LaneAt<DN> at(lane);
  const LaneAt<64> at_rot(lane);
  const KeyTiles<DN, DR> tiles(a, t0, h, len);
  float delta = 0.f;  // this lane's half of sum_j p dp
  tiles.fetch(0, base, wave, lane);
  for (int j0 = 0; j0 < keys; j0 += kK) {
    const unsigned b = (j0 / kK) & 1, ks = base + b * (2 * kKey + kRot), vs = ks + kKey, rs = vs + kKey;
    tile_barrier<0>();  // this tile is there, and all are done with the one before
    if (j0 + kK < keys) tiles.fetch(j0 + kK, base + (b ^ 1) * (2 * kKey + kRot), wave, lane);
    if (j0 > w0 + 31) continue;
    f32x16 s = {}, dp = {};
#pragma unroll
    for (int k = 0; k < DN / 16; ++k) {
      s = mma(row_frag(ks, at, 0, k), qf[k], s);
      dp = mma(row_frag(vs, at, 0, k), df[k], dp);
    }
#pragma unroll
    for (int k = 0; k < DR / 16; ++k) s = mma(row_frag(rs, at_rot, 0, k), qf[DN / 16 + k], s);
    if (j0 + kK - 1 > w0) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (j0 + acc_row(i, half) > qi) s[i] = -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
      delta = __builtin_fmaf(kda::fast_exp2(__builtin_fmaf(s[i], c, -lse)), dp[i], delta);
  }
  delta = halves_sum(delta);
  if (on && half == 0) *(f32x2*)(a.delta + 2 * row) = f32x2{lse, delta};
}

// dq.
template <int DN, int DR>
__global__ __launch_bounds__(256, 2) void dq_kernel(AttnArgs a, TileMap map) {
  constexpr int DQ = DN + DR;
  constexpr unsigned kKey = kK * DN * 2, kRot = kK * DR * 2;  // bytes of a tile's parts: keys, values, rotary keys
  __shared__ __align__(1024) char lds[2][2 * kKey + kRot];
  int h, len, q0;
  long long t0;
  if (!tile_place<kRows>(a, map, true, h, t0, len, q0)) return;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w0 = q0 + wave * 32;
  const int qi = w0 + (lane & 31);
  const int keys = min(len, q0 + kRows);
  const long long row = (t0 + qi) * a.H + h;
  const bool on = qi < len;

  bf16x8 qf[DQ / 16], df[DN / 16];
#pragma unroll
  for (int s = 0; s < DQ / 16; ++s) qf[s] = on ? row_frag(a.q + row * DQ, s, half) : bf16x8{};
#pragma unroll
  for (int s = 0; s < DN / 16; ++s) df[s] = on ? row_frag(a.dout + row * DN, s, half) : bf16x8{};
  const f32x2 stat = on ? *(const f32x2*)(a.delta + 2 * row) : f32x2{};
  const float lse = stat[0], delta = stat[1];
  const float c = a.scale * kda::kLog2e;

  const unsigned base = lds_address(&lds[0][0]);
  const LaneAt<DN> at(lane);
  const LaneAt<64> at_rot(lane);
  const KeyTiles<DN, DR> tiles(a, t0, h, len);
  f32x16 acc[DQ / 32] = {};
  tiles.fetch(0, base, wave, lane);
  for (int j0 = 0; j0 < keys; j0 += kK) {
    const unsigned b = (j0 / kK) & 1, ks = base + b * (2 * kKey + kRot), vs = ks + kKey, rs = vs + kKey;
    tile_barrier<0>();  // this tile is there, and all are done with the one before
    if (j0 + kK < keys) tiles.fetch(j0 + kK, base + (b ^ 1) * (2 * kKey + kRot), wave, lane);
    if (j0 > w0 + 31) continue;
    f32x16 s = {}, dp = {};
#pragma unroll
    for (int k = 0; k < DN / 16; ++k) {
      s = mma(row_frag(ks, at, 0, k), qf[k], s);
      dp = mma(row_frag(vs, at, 0, k), df[k], dp);
    }
#pragma unroll
    for (int k = 0; k < DR / 16; ++k) s = mma(row_frag(rs, at_rot, 0, k), qf[DN / 16 + k], s);
    if (j0 + kK - 1 > w0) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (j0 + acc_row(i, half) > qi) s[i] = -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = kda::fast_exp2(__builtin_fmaf(s[i], c, -lse)) * (dp[i] - delta);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const bf16x8 sf = acc_frag(s, k);
#pragma unroll
      for (int d = 0; d < DN / 32; ++d) acc[d] = mma(tr_frag(ks, at, 16 * k, d), sf, acc[d]);
#pragma unroll
      for (int d = 0; d < DR / 32; ++d)
        acc[DN / 32 + d] = mma(tr_frag(rs, at_rot, 16 * k, d), sf, acc[DN / 32 + d]);
    }
  }
  if (!on) return;
#pragma unroll
  for (int d = 0; d < DQ / 32; ++d) {
    acc[d] *= a.scale;
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *(u32x2*)(a.dq + row * DQ + 32 * d + acc_row(i, half)) =
          u32x2{kda::pk_bf16(acc[d][i], acc[d][i + 1]), kda::pk_bf16(acc[d][i + 2], acc[d][i + 3])};
  }
}

// dk and dv: S = Q K^T with the wavefront's 32 keys as B operands in registers,
// so that P and dS come as B operands over the queries; dV^T += dO^T P and
// dK^T += Q^T dS.  The rotary part of dk is this head's share of dk_pe.
// Up to 128 channels two wavefronts a SIMD (B4 T4096 H16 128/0: backward 1.15 ms
// where one takes 1.20, though 12 of their 256 registers spill); at 128 / 64 too
// many do (3.8 -> 6.6 ms at T16384 H12; both before delta had its own kernel).
template <int DN, int DR>
__global__ __launch_bounds__(256, DN + DR <= 128 ? 2 : 1) void dkv_kernel(AttnArgs a, TileMap map) {
  constexpr int DQ = DN + DR;
  // bytes of a tile's parts: queries, dout, the queries' rotary parts, and each wavefront's (lse, delta) rows
  constexpr unsigned kQry = kI * DN * 2, kRot = kI * DR * 2, kStat = kI * 8, kTileBytes = 2 * kQry + kRot + 4 * kStat;
  constexpr int kLoads = (2 * kQry + kRot) / 4096 + 1;  // a wavefront's share of a tile
  __shared__ __align__(1024) char lds[3][kTileBytes];
  int h, len, k0;
  long long t0;
  if (!tile_place<kRows>(a, map, false, h, t0, len, k0)) return;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w0 = k0 + wave * 32;
  const int kj = w0 + (lane & 31);  // this lane's key
  const bool on = kj < len;
  const long long col = (t0 + kj) * a.H + h;
  const long long first = t0 * a.H + h;

  bf16x8 kf[DQ / 16], vf[DN / 16];
#pragma unroll
  for (int s = 0; s < DN / 16; ++s) {
    kf[s] = on ? row_frag(a.kv + col * (2 * DN), s, half) : bf16x8{};
    vf[s] = on ? row_frag(a.kv + col * (2 * DN) + DN, s, half) : bf16x8{};
  }
#pragma unroll
  for (int s = 0; s < DR / 16; ++s) kf[DN / 16 + s] = on ? row_frag(a.k_pe + (t0 + kj) * DR, s, half) : bf16x8{};
  const float c = a.scale * kda::kLog2e;

  const unsigned base = lds_address(&lds[0][0]);
  const LaneAt<DN> at(lane);
  const LaneAt<64> at_rot(lane);
  auto fetch = [&](int i0, int b) {
    const unsigned to = base + b * kTileBytes;
    const int last = len - 1 - i0;
    const long long row = first + (long long)i0 * a.H;
    fetch_rows<kI, DN>(a.q + row * DQ, a.H * DQ, last, to, wave, lane);
    fetch_rows<kI, DN>(a.dout + row * DN, a.H * DN, last, to + kQry, wave, lane);
    if constexpr (DR > 0) fetch_rows<kI, DR>(a.q + row * DQ + DN, a.H * DQ, last, to + 2 * kQry, wave, lane);
    load_lds4(a.delta + 2 * row, (unsigned)(min(lane / 2, last) * (2 * a.H) + (lane & 1)) * 4,
              to + 2 * kQry + kRot + wave * kStat);
  };
  f32x16 dk[DQ / 32] = {}, dv[DN / 32] = {};
  // The scores of the next tile are formed beside the weights of this one, so
  // that matrix and vector work of one wavefront overlap.
  auto scores = [&](int b, f32x16& s, f32x16& dp) {
    const unsigned qs = base + b * kTileBytes, os = qs + kQry, rs = os + kQry;
    s = f32x16{};
    dp = f32x16{};
#pragma unroll
    for (int k = 0; k < DN / 16; ++k) {
      s = mma(row_frag(qs, at, 0, k), kf[k], s);
      dp = mma(row_frag(os, at, 0, k), vf[k], dp);
    }
#pragma unroll
    for (int k = 0; k < DR / 16; ++k) s = mma(row_frag(rs, at_rot, 0, k), kf[DN / 16 + k], s);
  };
  const int tiles = (len - k0 + kI - 1) / kI;
  f32x16 s, dp;
  fetch(k0, 0);
  if (tiles > 1) fetch(k0 + kI, 1);
  if (tiles > 1)
    tile_barrier<kLoads>();
  else
    tile_barrier<0>();
  scores(0, s, dp);
  int b = 0;  // buffer of tile t, of 3
  for (int t = 0; t < tiles; ++t) {
    const int i0 = k0 + t * kI, b1 = b == 2 ? 0 : b + 1, b2 = b1 == 2 ? 0 : b1 + 1;
    const unsigned qs = base + b * kTileBytes, os = qs + kQry, rs = os + kQry, st = rs + kRot + wave * kStat;
    tile_barrier<0>();  // the next tile is there, and all are done with the one before
    if (t + 2 < tiles) fetch(i0 + 2 * kI, b2);
    if (i0 < w0 + 31 || i0 + kI > len) {  // queries before the key, and past the document
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int qi = i0 + acc_row(i, half);
        if (qi < kj || qi >= len) s[i] = -INFINITY;
      }
    }
    f32x16 s1, dp1;
    scores(t + 1 < tiles ? b1 : b, s1, dp1);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
      const f32x4 stat = *(const lds_f32x4*)(st + acc_row(i, half) * 8);  // lse, delta of two queries
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[i + e] = kda::fast_exp2(__builtin_fmaf(s[i + e], c, -stat[2 * e]));
        dp[i + e] = s[i + e] * (dp[i + e] - stat[2 * e + 1]);
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const bf16x8 pf = acc_frag(s, k), sf = acc_frag(dp, k);
#pragma unroll
      for (int d = 0; d < DN / 32; ++d) dv[d] = mma(tr_frag(os, at, 16 * k, d), pf, dv[d]);
#pragma unroll
      for (int d = 0; d < DN / 32; ++d) dk[d] = mma(tr_frag(qs, at, 16 * k, d), sf, dk[d]);
#pragma unroll
      for (int d = 0; d < DR / 32; ++d)
        dk[DN / 32 + d] = mma(tr_frag(rs, at_rot, 16 * k, d), sf, dk[DN / 32 + d]);
    }
    s = s1;
    dp = dp1;
    b = b1;
  }
  if (!on) return;
#pragma unroll
  for (int d = 0; d < DN / 32; ++d) {
    dk[d] *= a.scale;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      bf16* to_k = a.dkv + col * (2 * DN) + 32 * d + acc_row(i, half);
      *(u32x2*)to_k = u32x2{kda::pk_bf16(dk[d][i], dk[d][i + 1]), kda::pk_bf16(dk[d][i + 2], dk[d][i + 3])};
      *(u32x2*)(to_k + DN) = u32x2{kda::pk_bf16(dv[d][i], dv[d][i + 1]), kda::pk_bf16(dv[d][i + 2], dv[d][i + 3])};
    }
  }
#pragma unroll
  for (int d = DN / 32; d < DQ / 32; ++d) {
    dk[d] *= a.scale;
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *(f32x4*)(a.pe_part + ((long long)h * a.tokens + t0 + kj) * DR + 32 * d - DN + acc_row(i, half)) =
          f32x4{dk[d][i], dk[d][i + 1], dk[d][i + 2], dk[d][i + 3]};
  }
}

// dk_pe: the heads' shares summed in head order, 4 channels a thread.  Tokens
// behind the last document have no shares and are left as they were.
template <int DR>
__global__ __launch_bounds__(256) void pe_kernel(AttnArgs a) {
  constexpr int kQuads = DR / 4;
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long t = id / kQuads;
  const int end = a.cu ? min(max(a.cu[a.N], 0), a.T) : a.tokens;
  if (t >= end) return;
  const float* from = a.pe_part + t * DR + (id % kQuads) * 4;
  f32x4 s = {};
#pragma unroll 4
  for (int h = 0; h < a.H; ++h) s += *(const f32x4*)(from + (long long)h * a.tokens * DR);
  *(u32x2*)(a.dk_pe + t * DR + (id % kQuads) * 4) = u32x2{kda::pk_bf16(s[0], s[1]), kda::pk_bf16(s[2], s[3])};
}

template <int DN, int DR>
hipError_t launch(const AttnArgs& a, hipStream_t stream) {
  const TileMap map = tile_map<kRows>(a);
  const dim3 grid((unsigned)map.blocks()), block(256);
  delta_kernel<DN, DR><<<grid, block, 0, stream>>>(a, map);
  dq_kernel<DN, DR><<<grid, block, 0, stream>>>(a, map);
  dkv_kernel<DN, DR><<<grid, block, 0, stream>>>(a, map);
  if constexpr (DR > 0)
    pe_kernel<DR><<<dim3((unsigned)(((long long)a.tokens * (DR / 4) + 255) / 256)), block, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_bwd(int Dn, int Dr, const AttnArgs& a, hipStream_t stream) {
  if (Dn == 64) return Dr ? launch<64, 64>(a, stream) : launch<64, 0>(a, stream);
  return Dr ? launch<128, 64>(a, stream) : launch<128, 0>(a, stream);
}

}  // namespace mla
