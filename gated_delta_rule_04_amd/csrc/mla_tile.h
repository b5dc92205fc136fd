// Matrix tiles of the latent attention kernels (gfx950, v_mfma_f32_32x32x16_bf16).
//
// Every product is taken so that its result can feed the next one from
// registers.  The accumulator of a 32x32 product holds, in lane l, column
// l % 32 and rows 8 (i / 4) + 4 (l / 32) + i % 4 for i = 0 .. 15; a 16-deep
// operand holds, in lane l, row (A) or column (B) l % 32 and 8 values of the
// inner index.  Which 8 is free as long as A and B agree, so registers 8s ..
// 8s+7 of an accumulator, rounded, are a B operand over its rows 16s .. 16s+15
// in the order {4h .. 4h+3, 8+4h .. 8+4h+3}, h = l / 32; the A operand facing
// it is read in that order with two transposing LDS reads (tr_frag).
#pragma once

#include <float.h>

#include "mla_launch.h"

namespace mla {

using kda::bf16x8;
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

constexpr int kPad = 16;  // elements after each LDS row: 32 bytes, so that 8 rows' 16-byte reads and 4 rows'
                          // 32-byte transposing reads fall on different banks for rows of 64, 128 and 192

__device__ __forceinline__ f32x16 mma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// 16 inner values of a row-major LDS row: the lane's row, values 8h .. 8h+7.
__device__ __forceinline__ bf16x8 row_frag(const bf16* row, int s, int half) {
  return *(const bf16x8*)(row + 16 * s + 8 * half);
}

// A operand of M^T from a row-major tile M of row length P: its columns c0 ..
// c0+31 as rows, over its rows r0 .. r0+15 in the accumulator's order.  In each
// 16 lanes a transposing read takes 4 rows of 16 columns; lane 4e + q
// addresses row e, columns 4q .. 4q+3.
template <int P>
__device__ __forceinline__ bf16x8 tr_frag(const bf16* tile, int r0, int c0, int lane) {
  const bf16* lo = tile + (r0 + 4 * (lane >> 5) + ((lane >> 2) & 3)) * P + c0 + (lane & 16) + 4 * (lane & 3);
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)lo);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lo + 8 * P));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Registers 8s .. 8s+7 of an accumulator as a B operand.
__device__ __forceinline__ bf16x8 acc_frag(const f32x16& x, int s) {
  return __builtin_bit_cast(bf16x8, u32x4{kda::pk_bf16(x[8 * s], x[8 * s + 1]), kda::pk_bf16(x[8 * s + 2], x[8 * s + 3]),
                                          kda::pk_bf16(x[8 * s + 4], x[8 * s + 5]),
                                          kda::pk_bf16(x[8 * s + 6], x[8 * s + 7])});
}

// Row of accumulator register i.
__device__ __forceinline__ constexpr int acc_row(int i, int half) { return 8 * (i >> 2) + 4 * half + (i & 3); }

// The value of the lane 32 further (both halves get both: [lower, upper]).
__device__ __forceinline__ void halves(float x, float& lower, float& upper) {
  const unsigned b = __builtin_bit_cast(unsigned, x);
  const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  lower = __builtin_bit_cast(float, (unsigned)r[0]);
  upper = __builtin_bit_cast(float, (unsigned)r[1]);
}
__device__ __forceinline__ float halves_max(float x) {
  float a, b;
  halves(x, a, b);
  return fmaxf(a, b);
}
__device__ __forceinline__ float halves_sum(float x) {
  float a, b;
  halves(x, a, b);
  return a + b;
}

// Documents are cut into tiles of BLOCK tokens; tile c of document n has the
// number cu[n] / BLOCK + n + c, so that the numbers of the documents do not
// overlap and are below tokens / BLOCK + N.  The document of tile `slot`: the
// last n whose first number is not above it, 64 candidates a step.
template <int BLOCK>
__device__ __forceinline__ int slot_document(const int* cu, int N, int T, int slot) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = N;
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) / 64, n = lo + lane * step;
    const bool below = n < hi && min(max(cu[n], 0), T) / BLOCK + n <= slot;
    const int count = __popcll(__ballot(below));
    lo += max(count - 1, 0) * step;
    hi = min(lo + step, hi);
  }
  return lo;
}

// Launch order of the expanded kernels: a unit is a head of a batch row (or of
// the packed row), with `tiles` tiles.  Workgroups go round the 8 XCDs, so with
// a multiple of 8 units each unit's tiles are given to one XCD, whose L2 then
// holds the unit's keys and values; otherwise units alternate, which keeps the
// XCDs even.  The longest tiles (the last, for queries) come first.
struct TileMap {
  int tiles, units;
  __host__ long long blocks() const { return (long long)tiles * units; }
  __device__ __forceinline__ void get(unsigned id, int& unit, int& tile) const {
    if (units % 8 == 0) {
      const unsigned k = id >> 3;
      unit = (int)(k / (unsigned)tiles) * 8 + (int)(id & 7);
      tile = (int)(k % (unsigned)tiles);
    } else {
      unit = (int)(id % (unsigned)units);
      tile = (int)(id / (unsigned)units);
    }
  }
};

// Document and place of a workgroup's tile; false when there is none.
template <int BLOCK>
__device__ __forceinline__ bool tile_place(const AttnArgs& a, const TileMap& map, bool last_first, int& head,
                                           long long& token0, int& len, int& row0) {
  int unit, tile;
  map.get(blockIdx.x, unit, tile);
  if (last_first) tile = map.tiles - 1 - tile;
  int n, begin, end;
  if (a.cu) {
    head = unit;
    n = slot_document<BLOCK>(a.cu, a.N, a.T, tile);
    document(a.cu, a.T, n, begin, end);
    tile -= begin / BLOCK + n;
    if (tile < 0) return false;
  } else {
    n = unit / a.H;
    head = unit - n * a.H;
    document(a.cu, a.T, n, begin, end);
  }
  token0 = begin;
  len = end - begin;
  row0 = tile * BLOCK;
  return row0 < len;
}

template <int BLOCK>
TileMap tile_map(const AttnArgs& a) {
  return a.cu ? TileMap{a.T / BLOCK + a.N, a.H} : TileMap{(a.T + BLOCK - 1) / BLOCK, a.N * a.H};
}

}  // namespace mla
