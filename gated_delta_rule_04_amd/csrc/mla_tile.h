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
using kda::f32x2;
using kda::f32x4;
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x16 mma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// 16 inner values of a row in global memory: values 8h .. 8h+7 of step s.
__device__ __forceinline__ bf16x8 row_frag(const bf16* row, int s, int half) {
  return *(const bf16x8*)(row + 16 * s + 8 * half);
}

// Tiles in LDS: rows of W = 64 channels or 128 and more, without padding (the
// loads from global memory straight into LDS write 1024 bytes in a row), the
// 16-byte pieces of each row permuted instead: piece p of row r lies at p ^
// swizzle(r).  The LDS serves 16 lanes of a 16-byte read together, and 32 of a
// transposing one, from 64 banks; so 16 consecutive rows' equal pieces must lie
// on 16 places of 256 bytes, and 4 consecutive rows' 64-byte runs on 4.
template <int W>
__device__ __forceinline__ constexpr int swizzle(int row) {
  return W == 64 ? ((row >> 1) & 1) << 2 | ((row >> 2) & 3) : (row & 3) << 2 | ((row >> 2) & 3);
}

typedef __attribute__((address_space(3))) bf16x8 lds_bf16x8;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

template <typename T>
__device__ __forceinline__ unsigned lds_address(T* p) {
  return (unsigned)(size_t)(__attribute__((address_space(3))) char*)p;
}

// Addresses of a lane's fragments, to be added to a tile's.
//   row  of its row l % 32: step k is at (row ^ 32 (k % 8)) + 256 (k / 8)
//   col  of the transposing read of rows 0 .. 15, columns 0 .. 31: columns 32d
//        at (col ^ 64 (d % 4)) + 256 (d / 4); rows 8 further at 8 rows and ^ 32
template <int W>
struct LaneAt {
  unsigned row, col;
  __device__ __forceinline__ explicit LaneAt(int lane) {
    const int r = lane & 31, half = lane >> 5, t = 4 * half + ((lane >> 2) & 3);
    row = r * (W * 2) + (half ^ swizzle<W>(r)) * 16;
    col = t * (W * 2) + ((2 * ((lane >> 4) & 1) + ((lane >> 1) & 1)) ^ swizzle<W>(t)) * 16 + (lane & 1) * 8;
  }
};
template <int W>
__device__ __forceinline__ bf16x8 row_frag(unsigned tile, const LaneAt<W>& at, int r0, int k) {
  return *(const lds_bf16x8*)(((tile + r0 * (W * 2) + at.row) ^ (32 * (k % 8))) + 256 * (k / 8));
}
// A operand of M^T from a tile M: its columns 32d .. 32d+31 as rows, over its
// rows r0 .. r0+15 in the accumulator's order.  In each 16 lanes a transposing
// read takes 4 rows of 16 columns; lane 4e + q addresses row e, columns 4q ..
// 4q+3.
template <int W>
__device__ __forceinline__ bf16x8 tr_frag(unsigned tile, const LaneAt<W>& at, int r0, int d) {
  const unsigned lo = ((tile + r0 * (W * 2) + at.col) ^ (64 * (d % 4))) + 256 * (d / 4);
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)lo);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)((lo ^ 32) + 8 * (W * 2)));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// A value that is the same in all lanes, as a scalar.
__device__ __forceinline__ unsigned uniform(unsigned x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ unsigned long long uniform(unsigned long long x) {
  return (unsigned long long)uniform((unsigned)(x >> 32)) << 32 | uniform((unsigned)x);
}

// 16 (or 4) bytes a lane from base + off straight to lds + 16 (4) lane.  M0
// holds the LDS address; it may not be read by the instruction after the one
// that writes it.  The base is copied by a scalar instruction in between: it
// may come from a vector one (a lane's value made scalar), after which a memory
// instruction would have to wait, and the compiler does not see this one.  Nor
// do its wait counts see these loads, or that they write LDS: tile_barrier
// waits for them and orders what reads it.
__device__ __forceinline__ void load_lds(const void* base, unsigned off, unsigned lds) {
  unsigned long long at;
  asm volatile("s_mov_b32 m0, %1\n\ts_mov_b64 %0, %3\n\tglobal_load_lds_dwordx4 %2, %0"
               : "=&s"(at)
               : "s"(uniform(lds)), "v"(off), "s"(uniform((unsigned long long)base))
               : "m0");
}
__device__ __forceinline__ void load_lds4(const void* base, unsigned off, unsigned lds) {
  unsigned long long at;
  asm volatile("s_mov_b32 m0, %1\n\ts_mov_b64 %0, %3\n\tglobal_load_lds_dword %2, %0"
               : "=&s"(at)
               : "s"(uniform(lds)), "v"(off), "s"(uniform((unsigned long long)base))
               : "m0");
}
// The same for the lanes of `on` (all lanes are active before and after), and
// with an address a lane.
__device__ __forceinline__ void load_lds_if(unsigned long long on, const void* base, unsigned off, unsigned lds) {
  unsigned long long at;
  asm volatile(
      "s_mov_b32 m0, %1\n\ts_mov_b64 %0, %3\n\ts_mov_b64 exec, %4\n\tglobal_load_lds_dwordx4 %2, %0\n\t"
      "s_mov_b64 exec, -1"
      : "=&s"(at)
      : "s"(uniform(lds)), "v"(off), "s"(uniform((unsigned long long)base)), "s"(uniform(on))
      : "m0");
}
__device__ __forceinline__ void load_lds_if(unsigned long long on, const bf16* from, unsigned lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_mov_b64 exec, %2\n\tglobal_load_lds_dwordx4 %1, off\n\ts_mov_b64 exec, -1" ::"s"(
          uniform(lds)),
      "v"(from), "s"(uniform(on))
      : "m0");
}
// Waits until at most N of this wavefront's vector memory operations are on
// their way (they end in order), and for the other wavefronts.
template <int N>
__device__ __forceinline__ void tile_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Waits for operands loaded into registers, here and not inside the loop that
// uses them, where the wait would be for the tiles on their way too.
template <int N>
__device__ __forceinline__ void arrived(bf16x8 (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(x[i]));
}

// Rows 0 .. ROWS-1 of W channels from a strided tensor into a tile, by 4
// wavefronts; rows after `last` read it again (their weights are zero).
template <int ROWS, int W>
__device__ __forceinline__ void fetch_rows(const bf16* base, int stride, int last, unsigned tile, int wave, int lane) {
  constexpr int kPer = 512 / W, kN = ROWS / kPer;  // rows of one 1024-byte load, loads
  static_assert(kN % 4 == 0, "each wavefront has the same number of loads");
#pragma unroll
  for (int i = 0; i < kN / 4; ++i) {
    const int r0 = (wave + 4 * i) * kPer, r = r0 + lane / (W / 8);
    load_lds(base, (unsigned)(min(r, last) * stride + ((lane % (W / 8)) ^ swizzle<W>(r)) * 8) * 2, tile + r0 * (W * 2));
  }
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
