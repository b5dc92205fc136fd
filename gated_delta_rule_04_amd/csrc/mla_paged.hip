// Absorbed latent attention over the paged cache.
//
// The rows of a sequence's queries (new token, head) are cut into blocks of 32
// WQ, the cache into tiles of 64 rows; a unit of work is a block and a tile.
// Each workgroup takes an equal, contiguous run of all units, so a long cache
// is split over as many workgroups as there are, whatever the lengths; a block
// that ends up split leaves float32 partial results (sums, running maximum and
// row sum) that combine_kernel joins.  The split depends on the sizes and
// lengths alone, and the parts are joined in order.
//
// A workgroup has 4 wavefronts.  S^T = C Q^T with the queries as B operands in
// registers, the softmax a row a lane, O^T += C^T P^T.  With 128 rows a
// wavefront owns 32 of them and all R channels of O^T (256 registers of sums
// at R = 512), and shares nothing but the tile; with 64 or 32 rows, two or
// four wavefronts own the same rows: each forms the scores of half the tile
// and the sums of its share of the channels, the weights going through LDS.
// Tiles come from the pages straight into LDS (no registers pass through),
// the next one on its way during a tile, 16-byte pieces permuted within a row
// so that both the row reads and the transposing reads spread over the banks.

// N256 H8 R256 rows to 2,048: 44 us (4.0 TB/s, a copy moving 5.1); N64 H96
// R512+64 to 8,192: 151 us; 4 chunks of up to 512 tokens at H96: 2.7 to 2.8 ms
// (matrix units 23% and 35% busy).  Bound by memory for few heads; at R = 512
// nearly every product waits for its own operand from LDS (62 of 68 in the code
// of 128-row blocks), and one wavefront a SIMD has nothing else to do then.
// Units count a sequence's whole cache, while a block of a causal chunk stops at
// the last row it sees: the longest run of a first chunk (no cache before it)
// has up to twice the mean's work (4 x 512 tokens, H96: 393 us).  Each workgroup
// goes through all the sequences' lengths to find its run: 65,536 sequences of
// 16 rows, H1 R128, take 0.9 ms, 4,096 of them 61 us.

#include "mla_split.h"

namespace mla {
namespace {

constexpr int kTile = 64;    // cache rows of a tile
constexpr int kPlaces = 16;  // tiles whose rows' places are looked up at a time

// How a call is cut; the host and the kernels agree on it.
struct PagedPlan {
  int wq;             // wavefronts of 32 rows in a block
  int groups;         // workgroups
  SplitSpace space;
};

// Block height by the rows a sequence has, the smallest that holds them or 128:
// a low block leaves fewer rows of its products empty, a high one reads each
// tile once for more rows.  In blocks of 32 / 64 / 128 rows, N64, all of 8,192
// cache rows, R 512+64: H12 158 / 171 / 203 us, H64 234 / 165 / 200, H96 367 /
// 271 / 216; chunks of 4 x 512 tokens, H96: 8.9 / 5.2 / 4.3 ms.  (R 256, 4,096
// rows: H12 42 / 46 / 65 us, H64 60 / 49 / 69, H96 86 / 73 / 73.  At R 128, where
// 64 rows are no slower for H96, 52 against 57 us, the chunks still gain: 1.33
// and 1.11 ms.)  Workgroups: as many as run at once (by
// their LDS one a CU at R = 512 and 256, two at 128), or the units there can be.
PagedPlan paged_plan(int N, int Tq, int H, int R, int Dr, long long max_len) {
  PagedPlan p;
  const long long rows = (long long)Tq * H, per = N ? (rows + N - 1) / N : 0;
  p.wq = per <= 32 ? 1 : per <= 64 ? 2 : 4;
  const long long blocks = rows / (32 * p.wq) + N, tiles = (max_len + kTile - 1) / kTile;
  const long long most = R == 128 ? 512 : 256, units = blocks * (tiles > 0 ? tiles : 1);
  p.groups = (int)(units < most ? (units > 0 ? units : 1) : most);
  p.space = split_space(N, p.groups, 32 * p.wq, R);
  return p;
}

template <int R, int DR, int WQ>
struct Paged {
  static constexpr int WD = 4 / WQ;  // wavefronts for each 32 rows
  static constexpr int D = R + DR, kWaves = 4, kThreads = 64 * kWaves, kRows = 32 * WQ;
  static constexpr int kLatLoads = kTile * R / 512 / kWaves, kRotLoads = DR ? 8 / kWaves : 0;  // a wavefront's share
  static constexpr int kSubs = WD > 1 ? 1 : 2;  // 32-row halves of a tile whose scores a wavefront forms
  static constexpr int kOut = R / 32 / WD;  // 32-channel tiles of O a wavefront holds
};

template <int R, int DR, int WQ>
__global__ __launch_bounds__((Paged<R, DR, WQ>::kThreads), 1) void paged_kernel(PagedWork w) {
  using C = Paged<R, DR, WQ>;
  constexpr int D = C::D;
  __shared__ __align__(1024) bf16 lat[2][kTile * R];
  __shared__ __align__(1024) bf16 rot[2][DR ? kTile * DR : 8];
  __shared__ int places[kPlaces * kTile];
  __shared__ __align__(16) u32x4 handed[C::WD > 1 ? WQ : 1][2][2][64];  // weights of the tile's halves, as B operands
  __shared__ float rise[2][C::kRows], sums[2][C::kRows];
  const PagedArgs& a = w.a;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, l32 = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wq = wave % WQ, wd = wave / WQ;

  Run run;
  if (!find_run<C::kRows, kTile>(w, blockIdx.x, run)) return;
  const long long begin = run.begin, end = run.end;
  long long base = run.base;  // units before sequence n
  int n = run.n;
  Sequence sq = sequence<C::kRows, kTile>(a, n);
  const bf16* const cache = static_cast<const bf16*>(a.cache);
  const float c = a.scale * kda::kLog2e;
  const unsigned lds_lat = lds_address(&lat[0][0]), lds_rot = lds_address(&rot[0][0]);
  const LaneAt<R> at_lat(lane);
  const LaneAt<64> at_rot(lane);
  LaneAt<R> at_out = at_lat;  // of the channels whose sums this wavefront holds
  at_out.col = (at_lat.col ^ (64 * (wd * C::kOut % 4))) + 256 * (wd * C::kOut / 4);

  for (long long u = begin; u < end;) {
    while (u >= base + sq.units()) {
      base += sq.units();
      sq = sequence<C::kRows, kTile>(a, ++n);
    }
    const int block = (int)((u - base) / sq.tiles), t0 = (int)((u - base) % sq.tiles);
    const int t1 = (int)min((long long)sq.tiles, t0 + (end - u));
    const bool whole = t0 == 0 && t1 == sq.tiles;
    const int slot = 2 * blockIdx.x + (u == begin ? 0 : 1);
    u += t1 - t0;
    const int rows = sq.Lq * a.H;
    // the last cache row that a row of the block, and this lane's row, sees
    const int seen = sq.L - sq.Lq + (min(rows, (block + 1) * C::kRows) - 1) / a.H;
    const int stop = min(t1, seen < 0 ? 0 : seen / kTile + 1);
    const int m0 = block * C::kRows + 32 * wq, mi = m0 + l32;
    const bool on = mi < rows;
    const int lim = on ? sq.L - sq.Lq + mi / a.H : INT_MAX;
    const long long row = (long long)sq.first * a.H + mi;
    const int* table = a.table + (long long)n * a.max_pages;

    // the places of the rows of tiles p0 .. p0 + kPlaces - 1 into LDS: cache row, -1 when it is not there
    auto look_up = [&](int p0) {
      for (int e = tid; e < kPlaces * kTile; e += C::kThreads) {
        const unsigned j = (unsigned)p0 * kTile + e, p = j / (unsigned)a.page_size;
        int r = -1;
        if (j < (unsigned)sq.L) {
          const int page = table[p];
          if ((unsigned)page < (unsigned)a.num_pages) r = (int)((unsigned)page * a.page_size + (j - p * a.page_size));
        }
        places[e] = r;
      }
    };
    // Load i of this wavefront's share of a tile's latents, or of its rotary keys, into buffer b; rows that are not
    // there read row 0 of the cache and are cleared later.  `from` is the place of row `lane` of the tile.
    auto fetch_lat = [&](int i, int from, int b, unsigned long long on) {
      constexpr int kPer = 512 / R;  // rows of one 1024-byte load
      const int r0 = (wave + C::kWaves * i) * kPer, r = r0 + lane / (R / 8);
      const unsigned to = lds_lat + (b * kTile + r0) * (R * 2);
      if constexpr (R == 512)  // a row a load: its address is scalar
        load_lds_if(on, cache + (long long)__builtin_amdgcn_readlane(from, r0) * D, (lane ^ swizzle<R>(r0)) * 16, to);
      else
        load_lds_if(on, cache + (long long)__shfl(from, r) * D + ((lane % (R / 8)) ^ swizzle<R>(r)) * 8, to);
    };
    auto fetch_rot = [&](int i, int from, int b, unsigned long long on) {
      const int r0 = (wave + C::kWaves * i) * 8, r = r0 + lane / 8;
      load_lds_if(on, cache + (long long)__shfl(from, r) * D + R + ((lane % 8) ^ swizzle<64>(r)) * 8,
                  lds_rot + (b * kTile + r0) * (DR * 2));
    };

    f32x16 acc[C::kOut] = {};
    float m = -FLT_MAX, l = 0.f;
    if (t0 < stop) {
      // A row that is not one reads the last again, and is not written.  (With 256 registers of sums, loads a branch
      // each keep the register allocator from spilling.)
      constexpr bool kMost = R < 512 || C::WD > 1;
      const bf16* q_row = a.q + ((long long)sq.first * a.H + min(mi, rows - 1)) * D;
      bf16x8 qf[D / 16];
#pragma unroll
      for (int s = 0; s < D / 16; ++s) qf[s] = kMost || on ? row_frag(q_row, s, half) : bf16x8{};
      int p0 = t0;
      __syncthreads();  // the run before is done with the buffers
      look_up(p0);
      __syncthreads();
      if constexpr (kMost) arrived(qf);
      int mine = places[lane];
#pragma unroll
      for (int i = 0; i < C::kLatLoads; ++i) fetch_lat(i, max(mine, 0), 0, ~0ull);
#pragma unroll
      for (int i = 0; i < C::kRotLoads; ++i) fetch_rot(i, max(mine, 0), 0, ~0ull);
      for (int t = t0; t < stop; ++t) {
        const int b = (t - t0) & 1;
        const unsigned long long there = __ballot(mine >= 0);
        if (t + 1 == p0 + kPlaces) {
          lds_barrier();
          look_up(p0 = t + 1);
        }
        tile_barrier<0>();  // tile t is there, and all are done with tile t - 1
        if (t + 1 < stop) mine = places[(t + 1 - p0) * kTile + lane];
        const unsigned long long more = t + 1 < stop ? ~0ull : 0ull;
        if (there != ~0ull) {  // uniform: every wavefront has the same 64 places
          for (int e = tid; e < kTile * (D / 8); e += C::kThreads) {
            const int r = e / (D / 8), piece = e % (D / 8);
            if (!((there >> r) & 1))
              *(u32x4*)(piece < R / 8 ? &lat[b][r * R + piece * 8] : &rot[b][r * DR + (piece - R / 8) * 8]) = u32x4{};
          }
          lds_barrier();
        }
        const int from = max(mine, 0);
        if (C::WD == 1 && m0 >= rows) {  // no rows: only this wavefront's share of the next tile
#pragma unroll
          for (int i = 0; i < C::kLatLoads; ++i) fetch_lat(i, from, b ^ 1, more);
#pragma unroll
          for (int i = 0; i < C::kRotLoads; ++i) fetch_rot(i, from, b ^ 1, more);
          continue;
        }
        const long long span = (long long)lim - (long long)t * kTile;  // the lane's row sees tile rows 0 .. span
        unsigned long long sees = there & (span < 0 ? 0ull : span >= 63 ? ~0ull : (2ull << span) - 1);
        const bool full = __all(sees == ~0ull);
        sees >>= 4 * half;
        // S^T of 32 rows of the tile, scaled to log2 units later; masked rows at -infinity; its maximum a query
        f32x16 s;
        // The next tile's loads are put between the products, a few at a time: the memory system takes a tile no
        // faster than it delivers one, and a wavefront that issues all of its share at once waits for that.
        constexpr int kLat = C::kLatLoads / C::kSubs, kRot = C::kRotLoads / C::kSubs, kShare = kLat + kRot;
        auto scores = [&](int sub, int part) {
          s = f32x16{};
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            s = mma(k < R / 16 ? row_frag(lds_lat + b * (kTile * R * 2), at_lat, 32 * sub, k)
                               : row_frag(lds_rot + b * (kTile * DR * 2), at_rot, 32 * sub, k - R / 16),
                    qf[k], s);
#pragma unroll
            for (int i = k * kShare / (D / 16); i < (k + 1) * kShare / (D / 16); ++i)
              if (i < kLat)
                fetch_lat(part * kLat + i, from, b ^ 1, more);
              else
                fetch_rot(part * kRot + i - kLat, from, b ^ 1, more);
          }
          if (!full) {
            const unsigned bits = (unsigned)(sees >> (32 * sub));
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (!((bits >> acc_row(i, 0)) & 1)) s[i] = -INFINITY;
          }
          float mx = s[0];
#pragma unroll
          for (int i = 1; i < 16; ++i) mx = fmaxf(mx, s[i]);
          return halves_max(mx) * c;
        };
        // The sums keep their reference while the maximum rises by less than 2^8, as in the expanded forward.
        auto refer = [&](float mx) {
          const float mn = fmaxf(m, mx), f = kda::fast_exp2(m - mn);
          m = mn;
          l *= f;
#pragma unroll
          for (int d = 0; d < C::kOut; ++d) acc[d] *= f;
        };
        auto weights = [&](const f32x16& s, bf16x8* pf) {
          f32x16 p;
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            p[i] = kda::fast_exp2(__builtin_fmaf(s[i], c, -m));
            sum += p[i];
          }
          pf[0] = acc_frag(p, 0);
          pf[1] = acc_frag(p, 1);
          return sum;
        };
        auto values = [&](int sub, int k, bf16x8 pf) {
#pragma unroll
          for (int d = 0; d < C::kOut; ++d) {
            acc[d] = mma(tr_frag(lds_lat + b * (kTile * R * 2), at_out, 32 * sub + 16 * k, d), pf, acc[d]);
          }
        };
        bf16x8 pf[2];
        if constexpr (C::WD > 1) {
          // Wavefronts 0 and 1 of the rows form the scores of the tile's halves (2 and 3, where there are, the same
          // again) and hand the weights over.  The weights come with the rows' present reference, and again only
          // where a maximum rose past it: one barrier.
          const int sub = wd & 1;
          auto hand = [&] {
            if (wd < 2) {
#pragma unroll
              for (int k = 0; k < 2; ++k) handed[wq][sub][k][lane] = __builtin_bit_cast(u32x4, pf[k]);
            }
          };
          const float mx = scores(sub, 0);
          float sum = weights(s, pf);
          if (wd < 2) rise[sub][32 * wq + l32] = mx > m + 8.f ? mx : -FLT_MAX;
          hand();
          lds_barrier();
          const int r = lane % C::kRows;
          if (__any(fmaxf(rise[0][r], rise[1][r]) > -FLT_MAX)) {  // the same for all wavefronts
            refer(fmaxf(rise[0][32 * wq + l32], rise[1][32 * wq + l32]));
            sum = weights(s, pf);
            hand();
            lds_barrier();
          }
          l += sum;
#pragma unroll
          for (int k = 0; k < 2; ++k) values(sub, k, pf[k]);
#pragma unroll
          for (int k = 0; k < 2; ++k) values(sub ^ 1, k, __builtin_bit_cast(bf16x8, handed[wq][sub ^ 1][k][lane]));
        } else {
#pragma unroll 1
          for (int sub = 0; sub < 2; ++sub) {
            const float mx = scores(sub, sub);
            if (__any(mx > m + 8.f)) refer(mx);
            l += weights(s, pf);
            values(sub, 0, pf[0]);
            values(sub, 1, pf[1]);
          }
        }
      }
    }
    l = halves_sum(l);
    if constexpr (C::WD > 1) {
      lds_barrier();  // the run before has read its sums
      if (wd < 2) sums[wd][32 * wq + l32] = l;
      lds_barrier();
      l = sums[0][32 * wq + l32] + sums[1][32 * wq + l32];
    }
    if (on) {
      const int ch = wd * (32 * C::kOut) + 4 * half;
      const bool first = half == 0 && wd == 0;
      if (whole) {
        const float r = l == 0.f ? 0.f : 1.f / l;  // 0: the row sees nothing
#pragma unroll
        for (int d = 0; d < C::kOut; ++d)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *(u32x2*)(a.o + row * R + ch + 32 * d + acc_row(i, 0)) = u32x2{
                kda::pk_bf16(acc[d][i] * r, acc[d][i + 1] * r), kda::pk_bf16(acc[d][i + 2] * r, acc[d][i + 3] * r)};
        if (a.lse && first) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * (1.f / kda::kLog2e);
      } else {
        const long long at = (long long)slot * C::kRows + 32 * wq + l32;
#pragma unroll
        for (int d = 0; d < C::kOut; ++d)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *(f32x4*)(w.po + at * R + ch + 32 * d + acc_row(i, 0)) =
                f32x4{acc[d][i], acc[d][i + 1], acc[d][i + 2], acc[d][i + 3]};
        if (first) {
          w.ml[2 * at] = m;
          w.ml[2 * at + 1] = l;
        }
      }
    }
  }
}

template <int R, int DR, int WQ>
hipError_t launch(const PagedWork& w, const PagedPlan& p, hipStream_t stream) {
  using C = Paged<R, DR, WQ>;
  paged_kernel<R, DR, WQ><<<dim3(p.groups), dim3(C::kThreads), 0, stream>>>(w);
  launch_combine<R, C::kRows, kTile>(w, p.groups, 8, stream);
  return hipGetLastError();
}

template <int R, int DR>
hipError_t launch(const PagedArgs& a, hipStream_t stream) {
  const PagedPlan p = paged_plan(a.N, a.Tq, a.H, R, DR, (long long)a.max_pages * a.page_size);
  const PagedWork w = split_work(a, p.space);
  switch (p.wq) {
    case 1: return launch<R, DR, 1>(w, p, stream);
    case 2: return launch<R, DR, 2>(w, p, stream);
    default: return launch<R, DR, 4>(w, p, stream);
  }
}

}  // namespace

size_t paged_workspace(int N, int Tq, int H, int R, int Dr, long long max_len) {
  return N == 0 || Tq == 0 ? 0 : paged_plan(N, Tq, H, R, Dr, max_len).space.total;
}

hipError_t launch_paged(int R, int Dr, const PagedArgs& a, hipStream_t stream) {
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
