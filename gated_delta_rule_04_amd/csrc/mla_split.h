// How the paged attention kernels cut their work, and how split blocks are joined.
//
// The rows of a sequence's queries (new token, head) are cut into blocks of ROWS,
// the cache into tiles of TILE rows; a unit of work is a block and a tile.  Each
// workgroup takes an equal, contiguous run of all units, in front of each block
// PagedArgs::start units that stand for what beginning it costs.  A block that
// ends up split leaves float32 partial results (sums, running maximum and row sum) in its
// workgroups' slots, which combine_kernel joins in order.
#pragma once

#include <limits.h>
#include <math.h>

#include "mla_tile.h"

namespace mla {

struct PagedWork {
  PagedArgs a;
  long long* prefix;  // [N + 1]: units before sequence n
  float* ml;          // [2 * groups][block rows][2]
  float* po;          // [2 * groups][block rows][R]
};
// A kernel's arguments, these and 8 bytes more, are in two lines of 64 bytes: with a third one to fetch, the join and
// the 4-bit cache's kernels take 0.2 to 0.4 us longer (the join of one sequence of 131,072 rows 5.8 and 6.2 us).
static_assert(sizeof(PagedWork) + 8 <= 128, "two lines");

// A sequence's share: its rows of q, its cache length and its units.
struct Sequence {
  int first, Lq, L, blocks, tiles, span;  // span: units of a block
  __device__ __forceinline__ long long units() const { return (long long)blocks * span; }
};
template <int ROWS, int TILE>
__device__ __forceinline__ Sequence sequence(const PagedArgs& a, int n) {
  Sequence s;
  int last = n + 1;
  s.first = n;
  if (a.cu) document(a.cu, a.Tq, n, s.first, last);
  s.Lq = last - s.first;
  s.L = min(max(a.lens[n], 0), a.max_pages * a.page_size);
  s.blocks = (s.Lq * a.H + ROWS - 1) / ROWS;
  s.tiles = max((s.L + TILE - 1) / TILE, 1);
  s.span = a.start + s.tiles;
  return s;
}

// A workgroup's run of units.
struct Run {
  int n;            // sequence of its first unit
  long long base;   // units before sequence n
  long long begin, end;
};

// Finds the run of workgroup `group` (256 threads); false when there is none.  Workgroup 0 writes the sequences' prefix
// for the join.  A run is the same in all lanes, and said so: what follows from it stays in scalar registers (the bf16
// cache, R 512 + 64 in blocks of 128 rows: 14 vector registers spilled, 18 if not said; N64 H96 to 8,192: 155 us and
// 164).
template <int ROWS, int TILE>
__device__ __forceinline__ bool find_run(const PagedWork& w, int group, Run& run) {
  constexpr int kWaves = 4, kThreads = 64 * kWaves;
  __shared__ long long scan[kWaves];
  __shared__ long long found[2];
  const PagedArgs& a = w.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Inclusive sum over the workgroup of one value a thread, and the total.
  auto block_scan = [&](long long x, long long& all) {
    for (int m = 1; m < 64; m <<= 1) {
      const long long y = __shfl_up(x, m);
      if (lane >= m) x += y;
    }
    if (a.N > kThreads) __syncthreads();  // the sums before are read
    if (lane == 63) scan[wave] = x;
    __syncthreads();
    all = 0;
    for (int i = 0; i < kWaves; ++i) {
      if (i < wave) x += scan[i];
      all += scan[i];
    }
    return x;
  };
  long long total = 0, mine = 0, incl = 0, all;
  for (int n0 = 0; n0 < a.N; n0 += kThreads) {
    const int n = n0 + tid;
    mine = n < a.N ? sequence<ROWS, TILE>(a, n).units() : 0;
    incl = block_scan(mine, all) + total;
    if (group == 0 && n < a.N) w.prefix[n] = incl - mine;
    total += all;
  }
  if (group == 0 && tid == 0) w.prefix[a.N] = total;
  const long long share = (total + gridDim.x - 1) / gridDim.x;
  run.begin = uniform((unsigned long long)(share * group));
  run.end = uniform((unsigned long long)min(run.begin + share, total));
  if (run.begin >= run.end) return false;
  long long before = 0;
  for (int n0 = 0; n0 < a.N; n0 += kThreads) {
    if (a.N > kThreads) {
      const int n = n0 + tid;
      mine = n < a.N ? sequence<ROWS, TILE>(a, n).units() : 0;
      incl = block_scan(mine, all) + before;
      before += all;
    }
    if (incl - mine <= run.begin && run.begin < incl) {
      found[0] = n0 + tid;
      found[1] = incl - mine;
    }
    if (run.begin < before) break;
  }
  __syncthreads();
  run.n = (int)uniform((unsigned)found[0]);
  run.base = (long long)uniform((unsigned long long)found[1]);
  return true;
}

// Joins the parts of split blocks: a wavefront a row for few parts, or for many
// a workgroup for 64 channels of a row, 16 parts at a time.
template <int R, int ROWS, int TILE, bool MANY>
static __global__ __launch_bounds__(256) void combine_kernel(PagedWork w, int groups) {
  constexpr int kSlice = MANY ? 64 : R, kAcross = kSlice / 4;      // threads over the channels
  constexpr int kLanes = MANY ? 256 : 64, kWays = MANY ? kLanes / kAcross : 1;  // threads of a row, parts at a time
  constexpr int kQuads = MANY ? 1 : R / 256 > 0 ? R / 256 : 1;      // 4-channel pieces a thread (few parts)
  const PagedArgs& a = w.a;
  const int tid = threadIdx.x;
  const long long row = MANY ? blockIdx.x / (R / 64) : (long long)blockIdx.x * 4 + (tid >> 6);
  if (row >= (long long)a.Tq * a.H) return;
  int n = (int)(row / a.H);
  if (a.cu) {
    int lo = 0, hi = a.N;
    const int token = n;
    while (hi - lo > 1) {  // the last sequence that starts at or before the token
      const int step = (hi - lo + 63) / 64, i = lo + (tid & 63) * step;
      const int count = __popcll(__ballot(i < hi && min(max(a.cu[i], 0), a.Tq) <= token));
      lo += max(count - 1, 0) * step;
      hi = min(lo + step, hi);
    }
    n = lo;
  }
  const Sequence s = sequence<ROWS, TILE>(a, n);
  const long long in = row - (long long)s.first * a.H;
  if (in < 0 || in >= (long long)s.Lq * a.H) return;
  const long long share = (w.prefix[a.N] + groups - 1) / groups;
  const long long u0 = w.prefix[n] + in / ROWS * s.span, u1 = u0 + s.span - 1;
  const int g0 = (int)((u0 + a.start) / share), g1 = (int)(u1 / share);
  if (g0 == g1) return;  // in one piece: written already
  // part g's slot: its run's first segment, unless the block starts inside the run
  auto place = [&](int g) { return (long long)(2 * g + (g == g0 && u0 > g0 * share ? 1 : 0)) * ROWS + in % ROWS; };
  float m = -FLT_MAX;
  for (int g = g0 + (tid & 63); g <= g1; g += 64) m = fmaxf(m, w.ml[2 * place(g)]);
#pragma unroll
  for (int i = 1; i < 64; i <<= 1) m = fmaxf(m, __shfl_xor(m, i));
  float l = 0.f;
  f32x4 o[kQuads] = {};
  const int way = MANY ? tid / kAcross : 0;
  const int ch = MANY ? (blockIdx.x % (R / 64)) * 64 + (tid % kAcross) * 4 : (tid & 63) * 4;
  const bool in_row = MANY || ch < R;
#pragma unroll 8
  for (int g = g0 + way; g <= g1; g += kWays) {
    const long long at = place(g);
    const float f = kda::fast_exp2(w.ml[2 * at] - m);
    l += w.ml[2 * at + 1] * f;
    if (in_row) {
#pragma unroll
      for (int q = 0; q < kQuads; ++q) o[q] += *(const f32x4*)(w.po + at * R + ch + 256 * q) * f;
    }
  }
  if constexpr (MANY) {
    __shared__ f32x4 part[kWays][kAcross];
    __shared__ float lpart[kWays];
    part[way][tid % kAcross] = o[0];
    if (tid % kAcross == 0) lpart[way] = l;
    __syncthreads();
    if (way != 0) return;
    for (int i = 1; i < kWays; ++i) {
      o[0] += part[i][tid];
      l += lpart[i];
    }
  }
  const float r = l == 0.f ? 0.f : 1.f / l;
  if (in_row) {
#pragma unroll
    for (int q = 0; q < kQuads; ++q)
      *(u32x2*)(a.o + row * R + ch + 256 * q) =
          u32x2{kda::pk_bf16(o[q][0] * r, o[q][1] * r), kda::pk_bf16(o[q][2] * r, o[q][3] * r)};
  }
  if (a.lse && ch == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * (1.f / kda::kLog2e);
}

// `few`: parts a block can have up to which a row takes a wavefront, and with more several workgroups (8 rows of 15
// parts: 4.2 us, with a wavefront a row 9.7 us; 6,144 rows of about 5 parts: 38 us, with a wavefront a row 13.5 us).
template <int R, int ROWS, int TILE>
void launch_combine(const PagedWork& w, int groups, int few, hipStream_t stream) {
  if (groups <= 1) return;
  const long long rows = (long long)w.a.Tq * w.a.H;
  if (groups > few * (rows / ROWS + 1))
    combine_kernel<R, ROWS, TILE, true><<<dim3((unsigned)(rows * (R / 64))), dim3(256), 0, stream>>>(w, groups);
  else
    combine_kernel<R, ROWS, TILE, false><<<dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, stream>>>(w, groups);
}

// Workspace: unit prefix of the sequences at 0, (maximum, sum) rows, partial sums.
struct SplitSpace {
  size_t ml, o, total;
};
inline SplitSpace split_space(int N, int groups, int block_rows, int R) {
  SplitSpace s;
  const size_t slots = 2 * (size_t)groups * block_rows;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  s.ml = up(((size_t)N + 1) * sizeof(long long));
  s.o = s.ml + up(slots * 2 * sizeof(float));
  s.total = s.o + slots * R * sizeof(float);
  return s;
}
inline PagedWork split_work(const PagedArgs& a, const SplitSpace& s) {
  char* ws = static_cast<char*>(a.ws);
  PagedWork w{a, reinterpret_cast<long long*>(ws), reinterpret_cast<float*>(ws + s.ml),
              reinterpret_cast<float*>(ws + s.o)};
  if (a.num_pages == 0) w.a.max_pages = 0;  // no cache rows at all: every length is 0
  return w;
}

}  // namespace mla
