// Absorbed latent attention over the paged 4-bit cache.
//
// The work is cut as in mla_split.h, in blocks of 32 RB rows and tiles of 32 cache
// rows.  A workgroup has 4 wavefronts, and they split the channels: each holds a
// quarter of the block's queries (R / 4 latent channels and a quarter of the rotary
// ones) and of O^T, for all rows of the block.  So each needs only its own quarter
// of a tile, for the scores and for the sums: it loads it from the pages straight
// into the layout of the products' A operand (a lane holds a row's 8 channels of a
// step in one register of codes), converts it there (v_cvt_scalef32_pk_bf16_fp4:
// exact), and puts it as bf16 into LDS of its own for the transposing reads of
// O^T += C^T P^T; no part of a tile passes between wavefronts.  What does is the
// scores: S^T = C Q^T over a quarter of the channels is a partial sum, of which
// each wavefront finishes the 8 rows of the tile that are its share, so that no
// exponential is taken twice, and hands the weights to all.
//
// In the pass over the tiles, an interval between two barriers forms the weights
// of tile i + 1, the sums of tile i and the partial scores of tile i + 2, which do
// not wait for each other.  A row's reference for the exponentials is kept until a
// score passes it by 2^8; then all wavefronts raise it (and rescale) before the
// tile's weights are used.

#include "mla_fp4.h"
#include "mla_split.h"

namespace mla {
namespace {

constexpr int kTile = 32;  // cache rows of a tile

struct Fp4Plan {
  int rb;      // 32-row blocks
  int groups;  // workgroups
  SplitSpace space;
};

Fp4Plan fp4_plan(int N, int Tq, int H, int R, int Dr, long long max_len) {
  Fp4Plan p;
  const long long rows = (long long)Tq * H, per = N ? (rows + N - 1) / N : 0;
  const int most_rb = R == 512 ? 3 : 4;
  p.rb = 1;
  long long best = -1;
  for (int rb = 1; rb <= most_rb; ++rb) {
    const long long cost = (per + 32 * rb - 1) / (32 * rb) * (rb + 1);
    if (best < 0 || cost < best) {
      best = cost;
      p.rb = rb;
    }
  }
  const long long blocks = rows / (32 * p.rb) + N, tiles = (max_len + kTile - 1) / kTile;
  const long long most = p.rb > 1 ? 256 : R == 512 ? 512 : R == 256 ? 768 : 1024;
  const long long units = blocks * (tiles > 0 ? tiles : 1);
  p.groups = (int)(units < most ? (units > 0 ? units : 1) : most);
  p.space = split_space(N, p.groups, 32 * p.rb, R);
  return p;
}

// Division by a number that is the same for all, for dividends below 2^31: with
// 2^(s-1) < d <= 2^s and m = 2^(31+s) / d + 1 (rounded down), n m / 2^(31+s) is off
// from n / d by less than 1 / d.
struct Divide {
  unsigned m, shift;
  __host__ explicit Divide(unsigned d) {
    unsigned s = 0;
    while ((1ull << s) < d) ++s;
    m = (unsigned)((1ull << (31 + s)) / d + 1);
    shift = 31 + s;
  }
  __device__ __forceinline__ unsigned of(unsigned n) const { return (unsigned)(((unsigned long long)n * m) >> shift); }
};

template <int R, int DR, int RB>
struct Fp4 {
  static constexpr int kThreads = 256, kRows = 32 * RB, kRow = fp4_row_bytes(R, DR);
  static constexpr int CW = R / 4, KS = CW / 16, DT = CW / 32;  // a wavefront's channels, steps of its scores, tiles of its sums
};

// A lane's part of a tile: its row's codes, scales and rotary key.
template <int KS>
struct Raw {
  unsigned code[KS];
  unsigned scale;
  u32x4 pe;
};

template <int R, int DR, int RB>
__global__ __launch_bounds__(256, RB == 1 ? 2 : 1) void paged_fp4_kernel(PagedWork w, Divide by_page) {
  using C = Fp4<R, DR, RB>;
  constexpr int D = R + DR, CW = C::CW, KS = C::KS, DT = C::DT, QS = KS + (DR ? 1 : 0);
  __shared__ __align__(1024) bf16 val[4][2][kTile * CW];     // a wavefront's own
  __shared__ __align__(16) f32x4 part[2][4][3][RB][64];         // partial scores: of, from
  __shared__ __align__(16) u32x4 weight[2][RB][2][64];          // B operands
  __shared__ __align__(16) int rose[2][4];                      // a score passed its row's reference
  __shared__ float top[4][C::kRows], sums[4][C::kRows];
  const PagedArgs& a = w.a;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, l32 = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  Run run;
  Sequence sq;
  if (!find_run<C::kRows, kTile>(w, run, sq)) return;
  // The same in all lanes, and said so: what follows from them stays in scalar registers.
  const long long begin = uniform((unsigned long long)run.begin), end = uniform((unsigned long long)run.end);
  long long base = uniform((unsigned long long)run.base);  // units before sequence n
  int n = uniform((unsigned)run.n);
  sq = sequence<C::kRows, kTile>(a, n);
  const float c = a.scale * kda::kLog2e;
  // Row of a tile that this lane loads: the rows go round by 8 a wavefront, so that a wavefront's own share of the
  // scores is always the first group of 4 registers.
  const int mine = (l32 + 8 * wave) & 31;
  const LaneAt<CW> at(lane);
  const int code_at = wave * (CW / 2) + half * (CW / 4);
  const int scale_at = R / 2 + 2 * DR + (R == 512 ? 4 * wave + 2 * half : R == 256 ? 2 * wave + half : wave);
  const int pe_at = R / 2 + wave * 32 + half * 16;

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
    const int rows = sq.Lq * a.H, m0 = block * C::kRows;
    // the last cache row that a row of the block sees
    const int seen = sq.L - sq.Lq + (min(rows, m0 + C::kRows) - 1) / a.H;
    const int stop = min(t1, seen < 0 ? 0 : seen / kTile + 1), count = stop - t0;
    const int* table = a.table + (long long)n * a.max_pages;
    int lim[RB];  // the last cache row that the lane's row sees
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int mi = m0 + 32 * r + l32;
      lim[r] = mi < rows ? sq.L - sq.Lq + mi / a.H : INT_MAX;
    }

    f32x16 acc[RB][DT] = {};
    float m[RB], l[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) m[r] = -FLT_MAX, l[r] = 0.f;
    if (count > 0) {
      bf16x8 qf[RB][QS];
#pragma unroll
      for (int r = 0; r < RB; ++r) {  // a row that is not one reads the last again, and is not written
        const bf16* q = a.q + ((long long)sq.first * a.H + min(m0 + 32 * r + l32, rows - 1)) * D;
#pragma unroll
        for (int s = 0; s < KS; ++s) qf[r][s] = *(const bf16x8*)(q + wave * CW + half * (CW / 2) + 8 * s);
        if constexpr (DR > 0) qf[r][KS] = *(const bf16x8*)(q + R + wave * 16 + half * 8);
      }

      Raw<KS> raw[2];       // tile t in raw[t % 2]
      unsigned bits[3];     // rows of tiles i + 1 .. i + 3 that are there, bit of lane l32
      int page = -1, off = 0;  // looked up for the tile after those
      auto look_up = [&](int t) {  // t from t0 on
        const int j = (t0 + t) * kTile + mine;
        page = -1;
        if (t < count && j < sq.L) {
          const unsigned p = by_page.of(j);
          off = j - (int)p * a.page_size;
          page = table[p];
        }
      };
      auto fetch = [&](Raw<KS>& x) {  // the tile looked up last; which of its rows are there
        const bool in = (unsigned)page < (unsigned)a.num_pages;
        const unsigned char* row = a.cache4 + (long long)(in ? page * a.page_size + off : 0) * C::kRow;
        if constexpr (KS == 8) {
          *(u32x4*)x.code = *(const u32x4*)(row + code_at);
          *(u32x4*)(x.code + 4) = *(const u32x4*)(row + code_at + 16);
          x.scale = *(const unsigned short*)(row + scale_at);
        } else if constexpr (KS == 4) {
          *(u32x4*)x.code = *(const u32x4*)(row + code_at);
          x.scale = row[scale_at];
        } else {
          *(u32x2*)x.code = *(const u32x2*)(row + code_at);
          x.scale = row[scale_at];
        }
        if constexpr (DR > 0) x.pe = *(const u32x4*)(row + pe_at);
        return (unsigned)__ballot(in);
      };
      f32x4 own[RB];  // this wavefront's own part of its share of the scores
      // 8 channels of step s, as an A operand
      auto channels = [&](const Raw<KS>& x, int s) {
        if (s >= KS) return x.pe;
        const unsigned byte = KS == 8 && s >= 4 ? x.scale >> 8 : x.scale & 255;
        return fp4_values(x.code[s], __builtin_bit_cast(float, byte << 23));
      };
      // Partial scores of a tile (register i: the lane's row, tile row acc_row(i) + 8 wave), handed over in part[b];
      // its values into val[b].  The next step's operand is converted beside this step's products.
      auto scores = [&](const Raw<KS>& x, int b) {
        f32x16 S[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) S[r] = f32x16{};
        bf16* to = val[wave][b] + mine * CW;
        u32x4 k = channels(x, 0);
#pragma unroll
        for (int s = 0; s < QS; ++s) {
          u32x4 next = k;
          if (s + 1 < QS) next = channels(x, s + 1);
          if (s < KS) *(u32x4*)(to + ((half * KS + s) ^ swizzle<CW>(mine)) * 8) = k;
#pragma unroll
          for (int r = 0; r < RB; ++r) S[r] = mma(__builtin_bit_cast(bf16x8, k), qf[r][s], S[r]);
          k = next;
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          own[r] = f32x4{S[r][0], S[r][1], S[r][2], S[r][3]};
#pragma unroll
          for (int g = 1; g < 4; ++g)
            part[b][(wave + g) & 3][3 - g][r][lane] = f32x4{S[r][4 * g], S[r][4 * g + 1], S[r][4 * g + 2], S[r][4 * g + 3]};
        }
      };
      auto highest = [&](const f32x4& x) { return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * c; };
      float pend[RB];  // row sums of the weights of the tile before its sums
      auto weights = [&](int r, const f32x4& s, int b) {
        float p[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = kda::fast_exp2(__builtin_fmaf(s[k], c, -m[r]));
        pend[r] = (p[0] + p[1]) + (p[2] + p[3]);
        *((u32x2*)&weight[b][r][wave >> 1][lane] + (wave & 1)) = u32x2{kda::pk_bf16(p[0], p[1]), kda::pk_bf16(p[2], p[3])};
      };
      // Weights of the rows r of the share, which stays in part[b] for raise(); j: the cache rows of its scores.
      auto softmax = [&](int r, const int* j, int b) {
        f32x4 x = own[r];
#pragma unroll
        for (int g = 0; g < 3; ++g) x += part[b][wave][g][r][lane];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = j[k] > lim[r] ? -INFINITY : x[k];
        part[b][wave][0][r][lane] = x;
        weights(r, x, b);
        return highest(x) > m[r] + 8.f;
      };
      auto rows_of = [&](int t, unsigned in, int* j) {  // of this lane's share of tile t; absent ones behind all
#pragma unroll
        for (int k = 0; k < 4; ++k) j[k] = (t0 + t) * kTile + 8 * wave + 4 * half + k;
        if (in != ~0u) {
#pragma unroll
          for (int k = 0; k < 4; ++k) j[k] = (in >> (4 * half + k)) & 1 ? j[k] : INT_MAX;
        }
      };
      auto clear = [&](Raw<KS>& x, unsigned in) {  // rows that are not there: any finite values
        if (in != ~0u && !((in >> l32) & 1)) {
          x.scale = 0;
          x.pe = u32x4{};
        }
      };
      auto raise = [&](int b) {  // tile b's scores passed a reference: a new one, and the weights again
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          const float mx = halves_max(highest(part[b][wave][0][r][lane]));
          top[wave][32 * r + l32] = mx > m[r] + 8.f ? mx : -FLT_MAX;
        }
        lds_barrier();
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          float mn = m[r];
#pragma unroll
          for (int g = 0; g < 4; ++g) mn = fmaxf(mn, top[g][32 * r + l32]);
          const float f = kda::fast_exp2(m[r] - mn);
          m[r] = mn;
          l[r] *= f;
#pragma unroll
          for (int d = 0; d < DT; ++d) acc[r][d] *= f;
          weights(r, part[b][wave][0][r][lane], b);
        }
        lds_barrier();
      };
      // Interval i, b = i % 2: weights of tile i + 1, sums of tile i, partial scores of tile i + 2 (whose values take the
      // place of tile i's).  Tiles from `count` on have no rows, and add nothing.
      auto interval = [&](int i, int b) {
        if (uniform((unsigned)(rose[b][0] | rose[b][1] | rose[b][2] | rose[b][3]))) raise(b);
        int j[4];
        rows_of(i + 1, bits[0], j);
        clear(raw[b], bits[1]);
        constexpr int kSteps = 2 * DT;
        const unsigned tile = lds_address(&val[wave][b][0]);
        bf16x8 p[RB], v = tr_frag(tile, at, 0, 0);
        bool up = false;
#pragma unroll
        for (int e = 0; e < kSteps; ++e) {
          const int s = e / DT, d = e % DT;
          bf16x8 next = v;
          if (e + 1 < kSteps) next = tr_frag(tile, at, 16 * ((e + 1) / DT), (e + 1) % DT);
          if (d == 0) {
#pragma unroll
            for (int r = 0; r < RB; ++r) p[r] = __builtin_bit_cast(bf16x8, weight[b][r][s][lane]);
          }
#pragma unroll
          for (int r = 0; r < RB; ++r)
            if (r * kSteps / RB == e) {
              l[r] += pend[r];
              up |= softmax(r, j, b ^ 1);
            }
#pragma unroll
          for (int r = 0; r < RB; ++r) acc[r][d] = mma(v, p[r], acc[r][d]);
          v = next;
          __builtin_amdgcn_sched_barrier(0);
        }
        rose[b ^ 1][wave] = __any(up);
        scores(raw[b], b);
        bits[0] = bits[1], bits[1] = bits[2], bits[2] = fetch(raw[b]);
        look_up(i + 5);
        lds_barrier();
      };

      lds_barrier();  // the run before is done with the LDS
      look_up(0);
      const unsigned bits0 = fetch(raw[0]);
      look_up(1);
      bits[0] = fetch(raw[1]);
      look_up(2);
      clear(raw[0], bits0);
      scores(raw[0], 0);
      bits[1] = fetch(raw[0]);
      look_up(3);
      lds_barrier();
      {
        int j[4];
        rows_of(0, bits0, j);
        bool up = false;
#pragma unroll
        for (int r = 0; r < RB; ++r) up |= softmax(r, j, 0);
        rose[0][wave] = __any(up);
      }
      clear(raw[1], bits[0]);
      scores(raw[1], 1);
      bits[2] = fetch(raw[1]);
      look_up(4);
      lds_barrier();
      for (int i = 0; i < count; i += 2) {
        interval(i, 0);
        if (i + 1 < count) interval(i + 1, 1);
      }
    }

#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const float x = halves_sum(l[r]);
      if (half == 0) sums[wave][32 * r + l32] = x;
    }
    lds_barrier();
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      float x = 0.f;
#pragma unroll
      for (int g = 0; g < 4; ++g) x += sums[g][32 * r + l32];
      l[r] = x;
    }
    lds_barrier();  // the next run may write its sums
    const int ch = wave * CW + 4 * half;
    const bool first = half == 0 && wave == 0;
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int mi = m0 + 32 * r + l32;
      if (mi >= rows) continue;
      const long long row = (long long)sq.first * a.H + mi;
      if (whole) {
        const float f = l[r] == 0.f ? 0.f : 1.f / l[r];  // 0: the row sees nothing
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *(u32x2*)(a.o + row * R + ch + 32 * d + acc_row(i, 0)) =
                u32x2{kda::pk_bf16(acc[r][d][i] * f, acc[r][d][i + 1] * f),
                      kda::pk_bf16(acc[r][d][i + 2] * f, acc[r][d][i + 3] * f)};
        if (a.lse && first) a.lse[row] = l[r] == 0.f ? -INFINITY : (m[r] + log2f(l[r])) * (1.f / kda::kLog2e);
      } else {
        const long long to = (long long)slot * C::kRows + 32 * r + l32;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *(f32x4*)(w.po + to * R + ch + 32 * d + acc_row(i, 0)) =
                f32x4{acc[r][d][i], acc[r][d][i + 1], acc[r][d][i + 2], acc[r][d][i + 3]};
        if (first) {
          w.ml[2 * to] = m[r];
          w.ml[2 * to + 1] = l[r];
        }
      }
    }
  }
}

template <int R, int DR, int RB>
hipError_t launch(const PagedWork& w, const Fp4Plan& p, hipStream_t stream) {
  using C = Fp4<R, DR, RB>;
  paged_fp4_kernel<R, DR, RB><<<dim3(p.groups), dim3(C::kThreads), 0, stream>>>(w, Divide(w.a.page_size));
  launch_combine<R, C::kRows, kTile>(w, p.groups, stream);
  return hipGetLastError();
}

template <int R, int DR>
hipError_t launch(const PagedArgs& a, hipStream_t stream) {
  const Fp4Plan p = fp4_plan(a.N, a.Tq, a.H, R, DR, (long long)a.max_pages * a.page_size);
  const PagedWork w = split_work(a, p.space);
  switch (p.rb) {
    case 1: return launch<R, DR, 1>(w, p, stream);
    case 2: return launch<R, DR, 2>(w, p, stream);
    case 3: return launch<R, DR, 3>(w, p, stream);
  }
  if constexpr (R < 512) return launch<R, DR, 4>(w, p, stream);
  return hipErrorInvalidValue;
}

}  // namespace

size_t paged_fp4_workspace(int N, int Tq, int H, int R, int Dr, long long max_len) {
  return N == 0 || Tq == 0 ? 0 : fp4_plan(N, Tq, H, R, Dr, max_len).space.total;
}

hipError_t launch_paged_fp4(int R, int Dr, const PagedArgs& a, hipStream_t stream) {
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
