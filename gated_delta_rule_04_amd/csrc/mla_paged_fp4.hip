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
// not wait for each other.
//
// The exponentials of a row have one reference through a run of tiles, the largest
// score of the first: bf16 weights and float32 sums lose nothing by a reference
// that is below the row's largest score by 2^30.  Where a score passes it by more,
// or a sum is not finite, the run is done again with the largest score of all its
// tiles, found first; so a run takes three passes at most, and the loop has no
// rescaling of the sums, which would cost it their place in the accumulators.

#include "mla_fp4.h"
#include "mla_split.h"

namespace mla {
namespace {

constexpr int kTile = 32;    // cache rows of a tile
constexpr int kPlaces = 16;  // tiles whose rows' places are looked up at a time

typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
// Said to be global: an access that may be LDS too is counted with those of the LDS, and waited for with them.
typedef __attribute__((address_space(1))) u32x4 global_u32x4;
typedef __attribute__((address_space(1))) u32x2 global_u32x2;
typedef __attribute__((address_space(1))) unsigned short global_u16;
typedef __attribute__((address_space(1))) unsigned char global_u8;

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
  const int lds = 28 * 1024 * p.rb + 64 * R + 4096;  // of a workgroup, and what is static
  const long long most = 256 * (160 * 1024 / lds < 1 ? 1 : 160 * 1024 / lds > 4 ? 4 : 160 * 1024 / lds);
  const long long units = blocks * (tiles > 0 ? tiles : 1);
  p.groups = (int)(units < most ? (units > 0 ? units : 1) : most);
  p.space = split_space(N, p.groups, 32 * p.rb, R);
  return p;
}

// A value that the compiler does not know where it came from: what is computed from it stays where it is used (sums of
// it that are the same in every pass of a loop would each hold a register through the loop).
template <typename T>
__device__ __forceinline__ T opaque(T x) {
  asm("" : "+v"(x));
  return x;
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
  // In LDS, 1024 bytes (16 a lane) a piece: partial scores [2][of wavefront][from 3][RB], weights as B operands
  // [2][RB][2]; then each wavefront's values of two tiles.
  static constexpr int kPart = 0, kWeight = kPart + 24 * RB * 1024, kVal = kWeight + 4 * RB * 1024;
  static constexpr int kValTile = kTile * CW * 2, kLds = kVal + 8 * kValTile;
  static constexpr int kAhead = RB < 3 ? 4 : 2;  // tiles in registers, on their way or there
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
  __shared__ __align__(1024) char lds[C::kLds];
  __shared__ float top[4][C::kRows];
  __shared__ int places[2][kPlaces * kTile];  // cache rows, -1 where there is none: of two groups of tiles
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
  // The row of a tile that a lane loads is (lane + 8 wave) % 32, so that a wavefront's own share of the scores is always
  // the first group of 4 registers.
  const LaneAt<CW> at(lane);
  // LDS addresses: of the lane's 16 bytes of a piece
  const unsigned lds0 = lds_address(&lds[0]), mine16 = lds0 + 16 * lane;
  // of the values: a piece of 8 channels of the row that the lane loads, piece s at put_at ^ 16 s
  const unsigned val_at = lds0 + C::kVal + wave * (2 * C::kValTile);

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

    f32x16 acc[RB][DT];
    float m[RB], l[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      m[r] = -FLT_MAX, l[r] = 0.f;
#pragma unroll
      for (int d = 0; d < DT; ++d) acc[r][d] = f32x16{};
    }
    if (count > 0) {
      bf16x8 qf[RB][QS];
#pragma unroll
      for (int r = 0; r < RB; ++r) {  // a row that is not one reads the last again, and is not written
        const bf16* q = a.q + ((long long)sq.first * a.H + min(m0 + 32 * r + l32, rows - 1)) * D;
#pragma unroll
        for (int s = 0; s < KS; ++s) qf[r][s] = *(const bf16x8*)(q + wave * CW + half * (CW / 2) + 8 * s);
        if constexpr (DR > 0) {
          qf[r][KS] = *(const bf16x8*)(q + R + wave * 16 + half * 8);
          if constexpr (RB == 3 && KS == 8) asm("" : "+a"(qf[r][KS]));
        }
      }

      constexpr int kAhead = C::kAhead;
      Raw<KS> raw[kAhead];  // tile t in raw[t % kAhead]
      unsigned bits[kAhead + 1];  // rows of tiles i + 1 .. that are there, bit of lane l32
      // The places of the rows of group g of tiles: looked up, then put into LDS.  (Compared without a sign: a group may
      // begin behind all the rows that 31 bits count.)
      const int last = min((t0 + count) * kTile, sq.L);
      int page[2];
      auto look_up = [&](int g) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = (t0 + g * kPlaces) * kTile + tid + 256 * e;
          page[e] = -1;
          if ((unsigned)j < (unsigned)last) page[e] = table[by_page.of(j)];
        }
      };
      auto put_places = [&](int g) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = (t0 + g * kPlaces) * kTile + tid + 256 * e;
          const int off = j - (int)by_page.of(j) * a.page_size;
          places[g & 1][tid + 256 * e] = (unsigned)page[e] < (unsigned)a.num_pages ? page[e] * a.page_size + off : -1;
        }
      };
      auto place = [&](int t) {
        return (&places[0][0])[(t & (2 * kPlaces - 1)) * kTile + ((opaque(lane) + 8 * wave) & 31)];
      };
      // Tile t's part from its place on; which of its rows are there.
      auto fetch = [&](Raw<KS>& x, int from) {
        const auto row = (const global_u8*)opaque((unsigned long long)a.cache4 + (long long)max(from, 0) * C::kRow);
        const int h = opaque(lane) >> 5, code_at = wave * (CW / 2) + h * (CW / 4), pe_at = R / 2 + wave * 32 + h * 16;
        const int scale_at = R / 2 + 2 * DR + (R == 512 ? 4 * wave + 2 * h : R == 256 ? 2 * wave + h : wave);
        if constexpr (KS == 8) {
          *(u32x4*)x.code = *(const global_u32x4*)(row + code_at);
          *(u32x4*)(x.code + 4) = *(const global_u32x4*)(row + code_at + 16);
          x.scale = *(const global_u16*)(row + scale_at);
        } else if constexpr (KS == 4) {
          *(u32x4*)x.code = *(const global_u32x4*)(row + code_at);
          x.scale = row[scale_at];
        } else {
          *(u32x2*)x.code = *(const global_u32x2*)(row + code_at);
          x.scale = row[scale_at];
        }
        if constexpr (DR > 0) x.pe = *(const global_u32x4*)(row + pe_at);
        return (unsigned)__ballot(from >= 0);
      };
      f32x4 own[RB];  // this wavefront's part of its share of the scores
      f32x16 S[RB];   // partial scores of a tile; register i: the lane's row, tile row acc_row(i) + 8 wave
      // 8 channels of step s, as an A operand
      auto channels = [&](const Raw<KS>& x, int s) {
        if (s >= KS) return x.pe;
        const unsigned byte = KS == 8 && s >= 4 ? x.scale >> 8 : x.scale & 255;
        return fp4_values(x.code[s], __builtin_bit_cast(float, byte << 23));
      };
      // The partial scores of a tile, and its values into val_at[b].  The next step's operand is converted beside this
      // step's products; `last` is done beside the last ones.
      auto scores = [&](const Raw<KS>& x, int b, auto last) {
        const int me = opaque(lane), row = (me + 8 * wave) & 31;
        const unsigned to = opaque(val_at + b * C::kValTile + row * (CW * 2) + (((me >> 5) * KS) ^ swizzle<CW>(row)) * 16);
        u32x4 k = channels(x, 0);
#pragma unroll
        for (int s = 0; s < QS; ++s) {
          u32x4 next = k;
          if (s + 1 < QS) next = channels(x, s + 1);
          if (s < KS) *(lds_u32x4*)(to ^ (16 * s)) = k;
#pragma unroll
          for (int r = 0; r < RB; ++r)
            S[r] = mma(__builtin_bit_cast(bf16x8, k), qf[r][s], s == 0 ? f32x16{} : S[r]);
          k = next;
          if (s == QS - 1) last();
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      auto hand = [&](int r, int b) {
        own[r] = f32x4{S[r][0], S[r][1], S[r][2], S[r][3]};
#pragma unroll
        for (int g = 1; g < 4; ++g)
          *(lds_f32x4*)(opaque(mine16 + C::kPart + ((wave + g) & 3) * (3 * RB * 1024)) +
                        ((4 * b * 3 + 3 - g) * RB + r) * 1024) =
              f32x4{S[r][4 * g], S[r][4 * g + 1], S[r][4 * g + 2], S[r][4 * g + 3]};
      };
      auto part = [&](int b, int g, int r) {
        return *(const lds_f32x4*)(opaque(mine16 + C::kPart + wave * (3 * RB * 1024)) + ((4 * b * 3 + g) * RB + r) * 1024);
      };
      auto weight = [&](int b, int r, int s) {
        return __builtin_bit_cast(bf16x8, *(const lds_u32x4*)(opaque(mine16) + C::kWeight + ((b * RB + r) * 2 + s) * 1024));
      };
      auto highest = [&](const f32x4& x) { return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * c; };
      bool passed = false;  // a score is above its reference by more than 2^30
      auto rows_of = [&](int t, unsigned in, int* j) {  // of this lane's share of tile t; absent ones behind all
#pragma unroll
        for (int k = 0; k < 4; ++k) j[k] = (t0 + t) * kTile + 8 * wave + 4 * (opaque(lane) >> 5) + k;
        if (in != ~0u) {
#pragma unroll
          for (int k = 0; k < 4; ++k) j[k] = (in >> (4 * (opaque(lane) >> 5) + k)) & 1 ? j[k] : INT_MAX;
        }
      };
      auto mask = [&](int r, f32x4& x, const int* j) {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = j[k] > lim[r] ? -INFINITY : x[k];
      };
      auto softmax = [&](int r, const f32x4& x, int b) {  // weights of the rows r of the share x
        float p[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = kda::fast_exp2(__builtin_fmaf(x[k], c, -m[r]));
        l[r] += (p[0] + p[1]) + (p[2] + p[3]);
        *(lds_u32x2*)(opaque(mine16 + C::kWeight + (wave >> 1) * 1024 + (wave & 1) * 8) + (b * RB + r) * 2048) = u32x2{kda::pk_bf16(p[0], p[1]), kda::pk_bf16(p[2], p[3])};
        passed |= highest(x) > m[r] + 30.f;
      };
      auto clear = [&](Raw<KS>& x, unsigned in) {  // rows that are not there: any finite values
        if (in != ~0u && !((in >> (opaque(lane) & 31)) & 1)) {
          x.scale = 0;
          x.pe = u32x4{};
        }
      };
      // The rows' largest scores of those that the wavefronts found.
      auto refer = [&](const float* mx) {
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          const float x = halves_max(mx[r]);
          if (half == 0) top[wave][32 * r + l32] = x;
        }
        lds_barrier();
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          m[r] = -FLT_MAX;
#pragma unroll
          for (int g = 0; g < 4; ++g) m[r] = fmaxf(m[r], top[g][32 * r + l32]);
        }
        lds_barrier();
      };
      auto share = [&](int t, unsigned in, int b, f32x4* x) {  // the finished and masked share of a tile
        int j[4];
        rows_of(t, in, j);
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          x[r] = own[r] + ((part(b, 0, r) + part(b, 1, r)) + part(b, 2, r));
          mask(r, x[r], j);
        }
      };

      // Interval i, b = i % 2, k = i % kAhead: weights of tile i + 1, sums of tile i, partial scores of tile i + 2 (whose values take the
      // place of tile i's).  Tiles from `count` on have no rows, and add nothing.
      auto interval = [&](int i, int k) {
        const int b = k & 1;
        Raw<KS>& x2 = raw[(k + 2) % kAhead];
        const int from = place(i + 2 + kAhead);
        const unsigned tile = opaque(val_at + b * C::kValTile);
        constexpr int kFirst = DT < 2 ? DT : 2;  // reads of operands ahead of the products
        bf16x8 p[2][RB], v[2][DT];
        f32x4 y[RB][3];
        auto take = [&](int r) {
#pragma unroll
          for (int g = 0; g < 3; ++g) y[r][g] = part(b ^ 1, g, r);
        };
#pragma unroll
        for (int r = 0; r < RB; ++r) p[0][r] = weight(b, r, 0);
#pragma unroll
        for (int d = 0; d < kFirst; ++d) v[0][d] = tr_frag(tile, at, 0, d);
#pragma unroll
        for (int r = 0; r < RB; ++r)
          if (r * DT / RB == 0) take(r);
        int j[4];
        rows_of(i + 1, bits[0], j);
        clear(x2, bits[1]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          if (d + kFirst < DT) v[0][d + kFirst] = tr_frag(tile, at, 0, d + kFirst);
          if (DT < 4 || d >= DT - 2) {  // before the next tile's values are put in their place
            constexpr int kEach = DT < 4 ? 1 : DT / 2;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
              const int f = DT < 4 ? d : (d - (DT - 2)) * kEach + e;
              v[1][f] = tr_frag(tile, at, 16, f);
            }
          }
#pragma unroll
          for (int r = 0; r < RB; ++r)
            if (r * DT / RB == d + 1) take(r);
#pragma unroll
          for (int r = 0; r < RB; ++r) acc[r][d] = mma(v[0][d], p[0][r], acc[r][d]);
#pragma unroll
          for (int r = 0; r < RB; ++r)
            if (r * DT / RB == d) {
              f32x4 x = own[r] + ((y[r][0] + y[r][1]) + y[r][2]);
              mask(r, x, j);
              softmax(r, x, b ^ 1);
            }
          __builtin_amdgcn_sched_barrier(0);
        }
        scores(x2, b, [&] {
#pragma unroll
          for (int r = 0; r < RB; ++r) p[1][r] = weight(b, r, 1);
        });
#pragma unroll
        for (int d = 0; d < DT; ++d) {
#pragma unroll
          for (int r = 0; r < RB; ++r) acc[r][d] = mma(v[1][d], p[1][r], acc[r][d]);
          if (d == 0) {
#pragma unroll
            for (int e = 0; e < kAhead; ++e) bits[e] = bits[e + 1];
            bits[kAhead] = fetch(x2, from);
          }
#pragma unroll
          for (int r = 0; r < RB; ++r)
            if (r * DT / RB == d) hand(r, b);
          __builtin_amdgcn_sched_barrier(0);
        }
        // the next group but one of places, when its own place is free: looked up here, put there a few intervals later
        if (i % kPlaces == 2) look_up(i / kPlaces + 2);
        if (i % kPlaces == kPlaces - 2) put_places(i / kPlaces + 2);
        lds_barrier();
      };

      for (bool again = false;;) {
        lds_barrier();  // the run before is done with the LDS
        look_up(0);
        put_places(0);
        look_up(1);
        put_places(1);
        lds_barrier();
#pragma unroll
        for (int e = 0; e < kAhead; ++e) bits[e] = fetch(raw[e], place(e));
        clear(raw[0], bits[0]);
        scores(raw[0], 0, [] {});
#pragma unroll
        for (int r = 0; r < RB; ++r) hand(r, 0);
        bits[kAhead] = fetch(raw[0], place(kAhead));
        lds_barrier();
        f32x4 x[RB];
        share(0, bits[0], 0, x);
        if (!again) {
          float mx[RB];
#pragma unroll
          for (int r = 0; r < RB; ++r) mx[r] = highest(x[r]);
          refer(mx);
        }
#pragma unroll
        for (int r = 0; r < RB; ++r) softmax(r, x[r], 0);
        clear(raw[1], bits[1]);
        scores(raw[1], 1, [] {});
#pragma unroll
        for (int r = 0; r < RB; ++r) hand(r, 1);
#pragma unroll
        for (int e = 0; e < kAhead; ++e) bits[e] = bits[e + 1];
        bits[kAhead] = fetch(raw[1], place(kAhead + 1));
        lds_barrier();
        for (int i = 0; i < count; i += kAhead) {
#pragma unroll
          for (int k = 0; k < kAhead; ++k)
            if (k == 0 || i + k < count) interval(i + k, k);
        }
        if (again) break;
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          float sum = l[r];  // not finite if any term is not
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) sum = __builtin_fmaf(acc[r][d][i], 0.f, sum);
          passed |= !(fabsf(sum) <= FLT_MAX);
        }
        if (lane == 0) top[wave][0] = 0.f;
        if (passed) top[wave][0] = 1.f;
        lds_barrier();
        again = uniform(__builtin_bit_cast(unsigned, top[0][0] + top[1][0] + top[2][0] + top[3][0])) != 0;
        lds_barrier();
        if (!again) break;
        float mx[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) mx[r] = -INFINITY;
        for (int t = 0; t < count; ++t) {
          if (t % kPlaces == 0) {
            look_up(t / kPlaces);
            put_places(t / kPlaces);
            lds_barrier();
          }
          const unsigned in = fetch(raw[0], place(t));
          clear(raw[0], in);
          scores(raw[0], 0, [] {});
#pragma unroll
          for (int r = 0; r < RB; ++r) hand(r, 0);
          lds_barrier();
          share(t, in, 0, x);
#pragma unroll
          for (int r = 0; r < RB; ++r) mx[r] = fmaxf(mx[r], highest(x[r]));
          lds_barrier();
        }
        refer(mx);
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          l[r] = 0.f;
#pragma unroll
          for (int d = 0; d < DT; ++d) acc[r][d] = f32x16{};
        }
      }
    }

#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const float x = halves_sum(l[r]);
      if (half == 0) top[wave][32 * r + l32] = x;
    }
    lds_barrier();
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      float x = 0.f;
#pragma unroll
      for (int g = 0; g < 4; ++g) x += top[g][32 * r + l32];
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
