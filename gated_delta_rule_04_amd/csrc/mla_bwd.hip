// Expanded latent attention, backward, causal.
//
//   p = exp(s - lse), dp = do v^T, ds = p (dp - delta), delta = <do, o> = sum_j p dp
//   dq = scale ds k, dk = scale ds^T q, dv = p^T do
//
// Two passes, so that no sum needs atomics: dq_kernel goes along the keys of
// 128 queries, dkv_kernel along the queries of 128 keys.  Each forms s and dp
// again (7 products in all where one pass has 5; a pass over both would add
// dq in an order that changes from run to run, or keep it in a workspace of
// float32 tiles).  p and ds are rounded to bf16 as operands; sums are float32.

#include <math.h>

#include "mla_tile.h"

namespace mla {
namespace {

constexpr int kRows = 128;  // queries (or keys) of a workgroup, 32 a wavefront
constexpr int kK = 32;      // keys of a tile of the dq kernel
constexpr int kI = 32;      // queries of a tile of the dk, dv kernel

// A tile of ROWS tokens, LDS row stride P: a strided [token][H][W] tensor's
// channels, or the shared rotary key's.  Pieces of 16 bytes, kept in registers
// between load and store so that the next tile is on its way during a tile.
template <int ROWS, int W, int P>
struct Tile {
  static constexpr int kPiece = W / 8, kN = ROWS * kPiece / 256;
  static_assert(W == 0 || (ROWS * kPiece) % 256 == 0, "pieces");
  u32x4 r[kN ? kN : 1];
  __device__ __forceinline__ void load(const bf16* base, int stride, int rows, int tid) {
#pragma unroll
    for (int p = 0; p < kN; ++p) {
      const int row = (p * 256 + tid) / kPiece, c = (p * 256 + tid) % kPiece;
      r[p] = u32x4{};
      if (row < rows) r[p] = *(const u32x4*)(base + row * stride + c * 8);
    }
  }
  __device__ __forceinline__ void store(bf16* lds, int tid) const {
#pragma unroll
    for (int p = 0; p < kN; ++p)
      *(u32x4*)(lds + ((p * 256 + tid) / (kPiece ? kPiece : 1)) * P + ((p * 256 + tid) % (kPiece ? kPiece : 1)) * 8) = r[p];
  }
};

// dq.  Also writes delta for the other kernel, summed as sum_j p dp in float32
// (the rounded o would put half a bf16 step of o into every ds).  A workgroup
// that starts a document takes delta from a pass of its own over its 128 keys
// first: there rows see few keys, and the rounding of o would show in dq.
// Further rows use <do, o> of the rounded o, whose error their many keys
// average down.
template <int DN, int DR>
__global__ __launch_bounds__(256, 2) void dq_kernel(AttnArgs a, TileMap map) {
  constexpr int DQ = DN + DR, KP = DQ + kPad, VP = DN + kPad;
  __shared__ __align__(16) bf16 ks[kK * KP];
  __shared__ __align__(16) bf16 vs[kK * VP];
  int h, len, q0;
  long long t0;
  if (!tile_place<kRows>(a, map, true, h, t0, len, q0)) return;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, w0 = q0 + (tid >> 6) * 32;
  const int qi = w0 + (lane & 31);
  const int keys = min(len, q0 + kRows);
  const int ld = a.H * 2 * DN;
  const bf16* kv = a.kv + (t0 * a.H + h) * (2 * DN);
  const bf16* pe = a.k_pe + t0 * DR;
  const long long row = (t0 + qi) * a.H + h;
  const bool on = qi < len;

  bf16x8 qf[DQ / 16], df[DN / 16];
  float lse = 0.f, delta = 0.f;
#pragma unroll
  for (int s = 0; s < DQ / 16; ++s) qf[s] = on ? row_frag(a.q + row * DQ, s, half) : bf16x8{};
#pragma unroll
  for (int s = 0; s < DN / 16; ++s) {
    df[s] = on ? row_frag(a.dout + row * DN, s, half) : bf16x8{};
    const bf16x8 of = on ? row_frag(a.o_in + row * DN, s, half) : bf16x8{};
#pragma unroll
    for (int i = 0; i < 8; ++i) delta += (float)of[i] * (float)df[s][i];
  }
  delta = halves_sum(delta);
  if (on) lse = a.lse[row] * kda::kLog2e;
  const float c = a.scale * kda::kLog2e;

  Tile<kK, DN, KP> tk;
  Tile<kK, DN, VP> tv;
  Tile<kK, DR, KP> tp;
  f32x16 acc[DQ / 32] = {};
  float sum = 0.f;  // this lane's half of sum_j p dp
  for (int pass = q0 == 0 ? 0 : 1; pass < 2; ++pass) {
    auto load = [&](int j0) {
      const bf16* at = kv + (long long)j0 * ld;
      tk.load(at, ld, len - j0, tid);
      tv.load(at + DN, ld, len - j0, tid);
      if constexpr (DR > 0) tp.load(pe + (long long)j0 * DR, DR, len - j0, tid);
    };
    sum = 0.f;
    load(0);
    for (int j0 = 0; j0 < keys; j0 += kK) {
      __syncthreads();
      tk.store(ks, tid);
      tv.store(vs, tid);
      if constexpr (DR > 0) tp.store(ks + DN, tid);
      __syncthreads();
      if (j0 + kK < keys) load(j0 + kK);
      if (j0 > w0 + 31) continue;
      f32x16 s = {}, dp = {};
#pragma unroll
      for (int k = 0; k < DQ / 16; ++k) s = mma(row_frag(ks + (lane & 31) * KP, k, half), qf[k], s);
#pragma unroll
      for (int k = 0; k < DN / 16; ++k) dp = mma(row_frag(vs + (lane & 31) * VP, k, half), df[k], dp);
      const bool edge = j0 + kK - 1 > w0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float p = kda::fast_exp2(__builtin_fmaf(s[i], c, -lse));
        if (edge && j0 + acc_row(i, half) > qi) p = 0.f;
        sum = __builtin_fmaf(p, dp[i], sum);
        s[i] = p * (dp[i] - delta);
      }
      if (pass == 0) continue;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bf16x8 sf = acc_frag(s, k);
#pragma unroll
        for (int d = 0; d < DQ / 32; ++d) acc[d] = mma(tr_frag<KP>(ks, 16 * k, 32 * d, lane), sf, acc[d]);
      }
    }
    sum = halves_sum(sum);
    if (pass == 0) delta = sum;
  }
  if (!on) return;
  if (half == 0) a.delta[row] = sum;
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
template <int DN, int DR>
__global__ __launch_bounds__(256, 1) void dkv_kernel(AttnArgs a, TileMap map) {
  constexpr int DQ = DN + DR, QP = DQ + kPad, OP = DN + kPad;
  __shared__ __align__(16) bf16 qs[kI * QP];
  __shared__ __align__(16) bf16 os[kI * OP];
  __shared__ __align__(16) float ls[kI], ds[kI];
  int h, len, k0;
  long long t0;
  if (!tile_place<kRows>(a, map, false, h, t0, len, k0)) return;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, w0 = k0 + (tid >> 6) * 32;
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

  Tile<kI, DQ, QP> tq;
  Tile<kI, DN, OP> to;
  float rl = 0.f, rd = 0.f;
  auto load = [&](int i0) {
    tq.load(a.q + (first + (long long)i0 * a.H) * DQ, a.H * DQ, len - i0, tid);
    to.load(a.dout + (first + (long long)i0 * a.H) * DN, a.H * DN, len - i0, tid);
    if (tid < kI) {
      rl = rd = 0.f;  // past the document: q and do are zero, and so is what p weighs
      if (i0 + tid < len) {
        rl = a.lse[first + (long long)(i0 + tid) * a.H] * kda::kLog2e;
        rd = a.delta[first + (long long)(i0 + tid) * a.H];
      }
    }
  };
  f32x16 dk[DQ / 32] = {}, dv[DN / 32] = {};
  load(k0);
  for (int i0 = k0; i0 < len; i0 += kI) {
    __syncthreads();
    tq.store(qs, tid);
    to.store(os, tid);
    if (tid < kI) {
      ls[tid] = rl;
      ds[tid] = rd;
    }
    __syncthreads();
    if (i0 + kI < len) load(i0 + kI);
    if (i0 + kI - 1 < w0) continue;  // all of it is before this wavefront's keys
    f32x16 s = {}, dp = {};
#pragma unroll
    for (int k = 0; k < DQ / 16; ++k) s = mma(row_frag(qs + (lane & 31) * QP, k, half), kf[k], s);
#pragma unroll
    for (int k = 0; k < DN / 16; ++k) dp = mma(row_frag(os + (lane & 31) * OP, k, half), vf[k], dp);
    const bool edge = i0 < w0 + 31;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const f32x4 lse = *(const f32x4*)(ls + acc_row(i, half)), del = *(const f32x4*)(ds + acc_row(i, half));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float p = kda::fast_exp2(__builtin_fmaf(s[i + e], c, -lse[e]));
        if (edge && i0 + acc_row(i + e, half) < kj) p = 0.f;
        s[i + e] = p;
        dp[i + e] = p * (dp[i + e] - del[e]);
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const bf16x8 pf = acc_frag(s, k), sf = acc_frag(dp, k);
#pragma unroll
      for (int d = 0; d < DN / 32; ++d) dv[d] = mma(tr_frag<OP>(os, 16 * k, 32 * d, lane), pf, dv[d]);
#pragma unroll
      for (int d = 0; d < DQ / 32; ++d) dk[d] = mma(tr_frag<QP>(qs, 16 * k, 32 * d, lane), sf, dk[d]);
    }
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
