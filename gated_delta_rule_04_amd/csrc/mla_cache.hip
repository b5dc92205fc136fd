// Append of new tokens to the paged latent cache: RMS norm of the latent,
// rotation of the rotary key, rotation of the queries' rotary parts.
//
// Memory bound: each row is read once and written once, 2 (R + Dr) bytes a
// token each way, and 2 Dr bytes a query head each way: 185 MB at 32,768
// tokens, R 512, Dr 64, 12 heads, in 31 us (a 1 GiB copy moves as much in 36).
// 4 tokens take 2.8 us.  One launch: the first
// blocks take latents (R / 8 lanes a row, 16 bytes a lane, the sum of squares
// in float32 over lane shuffles), the others rotations (8 pairs a thread: two
// 16-byte loads and stores, the table row as 32-byte loads).

#include "mla_launch.h"

namespace mla {
namespace {

using kda::bf16x8;
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

__device__ __forceinline__ bool kept(const AppendArgs& a, int t, int& slot) {
  slot = a.slots[t];
  return (unsigned)slot < (unsigned)a.num_slots;
}

template <int R, int DR>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a, int latent_blocks) {
  constexpr int kLanes = R / 8;              // lanes of a latent row
  constexpr int kRows = kThreads / kLanes;   // latent rows of a block
  if ((int)blockIdx.x < latent_blocks) {
    const long long t = (long long)blockIdx.x * kRows + threadIdx.x / kLanes;
    const int c = threadIdx.x % kLanes;
    int slot = 0;
    const bool on = t < a.T && kept(a, (int)t, slot);
    bf16x8 x = {};
    if (on) x = *(const bf16x8*)(a.c + t * (R + DR) + c * 8);
    if (a.weight) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += (float)x[i] * (float)x[i];
#pragma unroll
      for (int m = 1; m < kLanes; m <<= 1) ss += __shfl_xor(ss, m);
      const float r = 1.f / sqrtf(ss * (1.f / R) + a.eps);
      const f32x4 w0 = *(const f32x4*)(a.weight + c * 8), w1 = *(const f32x4*)(a.weight + c * 8 + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = (bf16)((float)x[i] * r * (i < 4 ? w0[i & 3] : w1[i & 3]));
    }
    if (on) *(bf16x8*)(a.cache + (long long)slot * (R + DR) + c * 8) = x;
    return;
  }
  if constexpr (DR > 0) {
    // unit (row, i): the pairs 8i .. 8i+7 of a row; rows are a token's key, then its heads
    constexpr int kUnits = DR / 16;
    const long long u = (long long)(blockIdx.x - latent_blocks) * kThreads + threadIdx.x;
    const long long row = u / kUnits;
    const int i = (int)(u % kUnits);
    const int per = a.H + 1;
    const long long t = row / per;
    const int h = (int)(row - t * per);
    if (t >= a.T) return;
    const bf16* src;
    bf16* dst;
    if (h == 0) {
      int slot;
      if (!kept(a, (int)t, slot)) return;
      src = a.c + t * (R + DR) + R;
      dst = a.cache + (long long)slot * (R + DR) + R;
    } else {
      src = a.q_pe + (t * a.H + h - 1) * DR;
      dst = a.q + (t * a.H + h - 1) * (R + DR) + R;
    }
    const int lo = a.interleaved ? 16 * i : 8 * i, hi = a.interleaved ? lo + 8 : lo + DR / 2;
    bf16x8 x = *(const bf16x8*)(src + lo), y = *(const bf16x8*)(src + hi);
    if (a.rope) {
      const int p = min(max(a.positions[t], 0), a.num_pos - 1);
      const float* tab = a.rope + (long long)p * DR + 8 * i;
      float cs[8], sn[8];
      *(f32x4*)cs = *(const f32x4*)tab;
      *(f32x4*)(cs + 4) = *(const f32x4*)(tab + 4);
      *(f32x4*)sn = *(const f32x4*)(tab + DR / 2);
      *(f32x4*)(sn + 4) = *(const f32x4*)(tab + DR / 2 + 4);
      if (a.interleaved) {
        float v[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float p0 = (float)(j < 4 ? x[2 * j & 7] : y[2 * j & 7]);
          const float p1 = (float)(j < 4 ? x[(2 * j + 1) & 7] : y[(2 * j + 1) & 7]);
          v[2 * j] = p0 * cs[j] - p1 * sn[j];
          v[2 * j + 1] = p1 * cs[j] + p0 * sn[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] = (bf16)v[j];
          y[j] = (bf16)v[8 + j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float p0 = (float)x[j], p1 = (float)y[j];
          x[j] = (bf16)(p0 * cs[j] - p1 * sn[j]);
          y[j] = (bf16)(p1 * cs[j] + p0 * sn[j]);
        }
      }
    }
    *(bf16x8*)(dst + lo) = x;
    *(bf16x8*)(dst + hi) = y;
  }
}

template <int R, int DR>
hipError_t launch(const AppendArgs& a, hipStream_t stream) {
  constexpr int kRows = kThreads / (R / 8);
  const int latent = (a.T + kRows - 1) / kRows;
  const long long units = DR ? (long long)a.T * (a.H + 1) * (DR / 16) : 0;
  const long long blocks = latent + (units + kThreads - 1) / kThreads;
  append_kernel<R, DR><<<dim3((unsigned)blocks), dim3(kThreads), 0, stream>>>(a, latent);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_append(int R, int Dr, const AppendArgs& a, hipStream_t stream) {
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
