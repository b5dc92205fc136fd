// Append of new tokens to the paged latent cache, in bf16 or in 4 bits: RMS norm
// of the latent, rotation of the rotary key, rotation of the queries' rotary
// parts; and the gather that reads 4-bit rows back.
//
// Memory bound: each row is read once and written once, 2 (R + Dr) bytes a
// token each way, and 2 Dr bytes a query head each way: 185 MB at 32,768
// tokens, R 512, Dr 64, 12 heads, in 31 us (a 1 GiB copy moves as much in 36).
// 4 tokens take 2.8 us.  In 4 bits a latent of 512 + 64 channels becomes 400
// bytes: 21,600 tokens with 12 heads, 106 MB, in 24 us.  One launch: the first
// blocks take latents (R / 8 lanes a row, 16 bytes a lane, the sum of squares
// in float32 over lane shuffles), the others rotations (8 pairs a thread: two
// 16-byte loads and stores, the table row as 32-byte loads).

#include "mla_fp4.h"

namespace mla {
namespace {

using kda::bf16x8;
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

typedef __attribute__((address_space(1))) const u32x4 global_u32x4;
typedef __attribute__((address_space(1))) const unsigned global_u32;
typedef __attribute__((address_space(1))) const unsigned char global_u8;
typedef __attribute__((address_space(1))) const char global_char;

__device__ __forceinline__ bool kept(const AppendArgs& a, int t, int& slot) {
  slot = a.slots[t];
  return (unsigned)slot < (unsigned)a.num_slots;
}

// A latent row in 4 bits.  R / 32 lanes a row, a block of 32 channels a lane, so
// that a lane has all that its scale needs.  Everything up to the code is float64,
// in which it costs no more than float32 here (both units take a lane a cycle, and
// the row's bytes bound the pass): a relative error of 2^-50 in place of 2^-22 in
// a value beside a border of its code decides a whole step of the code, which would
// otherwise happen to a value in about 10^6.  The float64 value divided by 2^E goes
// to the conversion instruction (float32 to 4 bits, ties to even) as 21 bits of
// its mantissa with what lies below or-ed into the last of them, which rounds as
// the whole would: the borders have 3 bits.
template <int R, int DR>
__device__ __forceinline__ void append_latent_fp4(const AppendArgs& a, int block) {
  constexpr int kLanes = R / 32, kRows = kThreads / kLanes;
  const long long t = (long long)block * kRows + threadIdx.x / kLanes;
  const int c = threadIdx.x % kLanes;
  int slot = 0;
  const bool on = t < a.T && kept(a, (int)t, slot);
  double y[32];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    bf16x8 x = {};
    if (on) x = *(const bf16x8*)(a.c + t * (R + DR) + c * 32 + 8 * i);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[8 * i + j] = (double)(float)x[j];
  }
  if (a.weight) {
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 32; ++i) ss += y[i] * y[i];
#pragma unroll
    for (int m = 1; m < kLanes; m <<= 1) ss += __shfl_xor(ss, m);
    const double r = 1.0 / sqrt(ss * (1.0 / R) + (double)a.eps);
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      const f32x4 w = *(const f32x4*)(a.weight + c * 32 + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[i + j] = y[i + j] * r * (double)w[j];
    }
  }
  if (!on) return;
  // the upper word of |y|, the last bit set for anything below it
  auto upper = [](double x) {
    const unsigned long long b = __builtin_bit_cast(unsigned long long, x);
    return (unsigned)(b >> 32) | ((unsigned)b != 0);
  };
  unsigned most = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) most = max(most, upper(y[i]) & 0x7fffffffu);
  // max |y| = (1 + f) 2^k <= 7 2^E
  int e = (int)(most >> 20) - 1023 - 2 + ((most & 0xfffffu) > 0xc0000u);
  const bool finite = most < 0x7ff00000u;
  e = min(max(e, -125), 125);
  const double inv = __builtin_bit_cast(double, (unsigned long long)(1023 - e) << 52);
  unsigned code[4] = {};
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    float v[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const unsigned long long b = (unsigned long long)upper(y[i + j]) << 32;
      v[j] = (float)(__builtin_bit_cast(double, b) * inv);
    }
    switch (i / 2 % 4) {
      case 0: code[i / 8] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code[i / 8], v[0], v[1], 1.f, 0); break;
      case 1: code[i / 8] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code[i / 8], v[0], v[1], 1.f, 1); break;
      case 2: code[i / 8] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code[i / 8], v[0], v[1], 1.f, 2); break;
      default: code[i / 8] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code[i / 8], v[0], v[1], 1.f, 3);
    }
  }
  if (!finite) code[0] = code[1] = code[2] = code[3] = 0;
  constexpr int kRow = fp4_row_bytes(R, DR), kScales = R / 2 + 2 * DR;
  unsigned char* row = (unsigned char*)a.cache + (long long)slot * kRow;
  *(u32x4*)(row + c * 16) = u32x4{code[0], code[1], code[2], code[3]};
  row[kScales + c] = (unsigned char)(finite ? e + 127 : 255);
  for (int i = kScales + kLanes + c; i < kRow; i += kLanes) row[i] = 0;
}

template <int R, int DR, bool FP4>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a, int latent_blocks) {
  constexpr int kLanes = R / 8;              // lanes of a latent row
  constexpr int kRows = kThreads / kLanes;   // latent rows of a block
  if ((int)blockIdx.x < latent_blocks) {
    if constexpr (FP4) {
      append_latent_fp4<R, DR>(a, blockIdx.x);
      return;
    }
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
    if (on) *(bf16x8*)((bf16*)a.cache + (long long)slot * (R + DR) + c * 8) = x;
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
      dst = FP4 ? (bf16*)((char*)a.cache + (long long)slot * fp4_row_bytes(R, DR) + R / 2)
                : (bf16*)a.cache + (long long)slot * (R + DR) + R;
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

// The last n in [0, N) whose clamped start is not above t, 64 candidates a step; the same for all lanes.
__device__ __forceinline__ int starts_before(const GatherArgs& a, long long t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = a.N;
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) / 64, i = lo + lane * step;
    const int count = __popcll(__ballot(i < hi && min(max(a.cu[i], 0), a.T) <= t));
    lo += max(count - 1, 0) * step;
    hi = min(lo + step, hi);
  }
  return lo;
}

// Rows of a 4-bit cache as bf16.  A wavefront takes kGather rows: first a lane
// finds each row's place (sequence, page), then R / 8 lanes a row read the
// latent, 8 channels a lane (4 bytes in, 16 out), and 8 lanes a row the rotary
// key, all rows at once.  A row that is not there reads the first one (of the
// output, if the cache has none) and is put as zeros: without a branch, all
// loads are on their way together.  Memory bound: 102,000 rows of 512 + 64
// channels, 158 MB, in 25 us (part of it from the last-level cache; a copy moves
// as much in 31); a row a wavefront 61 us, with branches around the loads 85.
constexpr int kGather = 8;

template <int R, int DR>
__global__ __launch_bounds__(kThreads) void gather_kernel(GatherArgs a) {
  constexpr int kLanes = R / 8, kOnce = 64 / kLanes, kTimes = kGather / kOnce, kRow = fp4_row_bytes(R, DR);
  static_assert(DR == 0 || DR / 8 * kGather == 64, "8 rows' rotary keys in one load");
  const int lane = threadIdx.x & 63, c = lane % kLanes;
  const long long t0 = ((long long)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6)) * kGather;
  const int count = (int)(min(t0 + kGather, (long long)min(max(a.cu[a.N], 0), a.T)) - t0);
  if (count <= 0) return;
  const int first = starts_before(a, t0), last = starts_before(a, t0 + count - 1);
  constexpr int kMissing = -1, kLeave = -2;  // no cache row; no row of a sequence: left as it was
  int place = kLeave;
  if (lane < count) {
    const long long t = t0 + lane;
    int lo = first, hi = last + 1;
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2;
      if (min(max(a.cu[mid], 0), a.T) <= t)
        lo = mid;
      else
        hi = mid;
    }
    const long long in = t - min(max(a.cu[lo], 0), a.T), j = in + (a.starts ? a.starts[lo] : 0);
    if (in >= 0) place = kMissing;
    if (in >= 0 && j >= 0 && j < (long long)a.max_pages * a.page_size) {
      const unsigned p = (unsigned)j / (unsigned)a.page_size;
      const int page = a.table[(long long)lo * a.max_pages + p];
      if ((unsigned)page < (unsigned)a.num_pages) place = page * a.page_size + (int)((unsigned)j - p * a.page_size);
    }
  }
  const auto cache = (global_char*)(a.num_pages > 0 ? a.cache : (const unsigned char*)a.rows);
  auto row = [&](int i) { return cache + (long long)max(i, 0) * kRow; };
  const int pe_row = lane / 8, pe_place = __shfl(place, pe_row);
  u32x4 pe = {};
  if constexpr (DR > 0) pe = *(global_u32x4*)(row(pe_place) + R / 2 + 16 * (lane % 8));
  unsigned codes[kTimes], scale[kTimes];
  int at[kTimes];
#pragma unroll
  for (int i = 0; i < kTimes; ++i) {
    at[i] = __shfl(place, i * kOnce + lane / kLanes);
    codes[i] = *(global_u32*)(row(at[i]) + 4 * c);
    scale[i] = *(global_u8*)(row(at[i]) + R / 2 + 2 * DR + c / 4);
  }
  bf16* const out = a.rows + t0 * (R + DR);
#pragma unroll
  for (int i = 0; i < kTimes; ++i) {
    const int r = i * kOnce + lane / kLanes;
    const unsigned s = scale[i] >= kFp4NaN ? 255u : scale[i];
    const u32x4 v = fp4_values(codes[i], __builtin_bit_cast(float, s << 23));
    if (at[i] != kLeave) *(u32x4*)(out + r * (R + DR) + 8 * c) = at[i] >= 0 ? v : u32x4{};
  }
  if constexpr (DR > 0)
    if (pe_place != kLeave)
      *(u32x4*)(out + pe_row * (R + DR) + R + 8 * (lane % 8)) = pe_place >= 0 ? pe : u32x4{};
}

template <int R, int DR>
hipError_t launch_gather(const GatherArgs& a, hipStream_t stream) {
  constexpr int kRows = kThreads / 64 * kGather;
  gather_kernel<R, DR><<<dim3((unsigned)(((long long)a.T + kRows - 1) / kRows)), dim3(kThreads), 0, stream>>>(a);
  return hipGetLastError();
}

template <int R, int DR, bool FP4>
hipError_t launch(const AppendArgs& a, hipStream_t stream) {
  constexpr int kRows = kThreads / (R / (FP4 ? 32 : 8));
  const int latent = (a.T + kRows - 1) / kRows;
  const long long units = DR ? (long long)a.T * (a.H + 1) * (DR / 16) : 0;
  const long long blocks = latent + (units + kThreads - 1) / kThreads;
  append_kernel<R, DR, FP4><<<dim3((unsigned)blocks), dim3(kThreads), 0, stream>>>(a, latent);
  return hipGetLastError();
}

}  // namespace

template <bool FP4>
static hipError_t launch_append(int R, int Dr, const AppendArgs& a, hipStream_t stream) {
  switch (R + Dr) {
    case 128: return launch<128, 0, FP4>(a, stream);
    case 192: return launch<128, 64, FP4>(a, stream);
    case 256: return launch<256, 0, FP4>(a, stream);
    case 320: return launch<256, 64, FP4>(a, stream);
    case 512: return launch<512, 0, FP4>(a, stream);
    case 576: return launch<512, 64, FP4>(a, stream);
  }
  return hipErrorInvalidValue;
}
hipError_t launch_append(int R, int Dr, const AppendArgs& a, hipStream_t stream) {
  return launch_append<false>(R, Dr, a, stream);
}
hipError_t launch_append_fp4(int R, int Dr, const AppendArgs& a, hipStream_t stream) {
  return launch_append<true>(R, Dr, a, stream);
}

hipError_t launch_gather(int R, int Dr, const GatherArgs& a, hipStream_t stream) {
  switch (R + Dr) {
    case 128: return launch_gather<128, 0>(a, stream);
    case 192: return launch_gather<128, 64>(a, stream);
    case 256: return launch_gather<256, 0>(a, stream);
    case 320: return launch_gather<256, 64>(a, stream);
    case 512: return launch_gather<512, 0>(a, stream);
    case 576: return launch_gather<512, 64>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace mla
