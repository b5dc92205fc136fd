// Absorbed latent attention over the paged 4-bit cache.
//
// The work is cut as in mla_split.h, in blocks of 32 WQ rows and tiles of 32 cache
// rows.  A workgroup has 4 wavefronts: WQ of them take 32 rows of the block each,
// and the WT = 4 / WQ groups of such take the tiles in turn.  A wavefront holds its
// rows' queries (vector registers) and their O^T for all channels (accumulators;
// at R = 512 all of them).
//
// A tile's codes go from the pages into registers, in the layout of the products'
// A operand: a lane holds half a row, 8 channels of a step in one register, and
// converts them as they are needed (v_cvt_scalef32_pk_bf16_fp4: exact).  S^T = C
// Q^T, the softmax a row a lane, and the weights are the B operand of O^T += C^T P^T
// as they are.  Its A operand is read by transposing reads from LDS, where the
// converted tile is put, by each of the WQ wavefronts in part; with WQ = 1 nothing
// passes between wavefronts and there is no barrier.  The products of tile i + 1's
// scores and of tile i's sums alternate, and each register of codes is loaded
// again, for the tile after, as soon as it has been converted.
//
// The exponentials of a row have one reference through a run of tiles, the largest
// score of the first: bf16 weights and float32 sums lose nothing by a reference
// that is below the row's largest score by 2^60, while values stay below 2^36 (the
// sums of 2^27 of them below 2^123).  Where a score passes it by more, or a scale
// is 2^33 or more, the run is done again with the largest score of all its tiles,
// found first; so a run takes three passes at most, and the loop has no rescaling
// of the sums, which would cost them their place in the accumulators.

#include <algorithm>
#include <type_traits>

#include "mla_fp4.h"
#include "mla_split.h"

namespace mla {
namespace {

constexpr int kTile = 32;  // cache rows of a tile
// What beginning and ending a block costs (queries, first loads, handing the sums on), counted as 12 / WQ tiles of a
// workgroup where the work is cut: it keeps workgroups from having the ends of several short sequences (N64 H96 to
// 8,192 rows of 512 + 64: 124 us without, 117 with, N256 H8 to 2,048 rows of 256: 34 and 31, N6 H64 to 274 rows of 512:
// 30 and 23, N31 H96 to 1,781 rows of 256 + 64: 37 and 30; where all ends fall on cuts, N256 H8 R256 of 2,048 each, it
// loses: 32 and 35).  At R = 512 it is 31,000 cycles of a wavefront in fact, and a tile 4,350.
constexpr int kStart = 12;

typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
// Said to be global: an access that may be LDS too is counted with those of the LDS, and waited for with them.
typedef __attribute__((address_space(1))) const u32x4 global_u32x4;
typedef __attribute__((address_space(1))) const u32x2 global_u32x2;
typedef __attribute__((address_space(1))) const unsigned global_u32;
typedef __attribute__((address_space(1))) const char global_char;

struct Fp4Plan {
  int wq;      // wavefronts of 32 rows in a block
  int groups;  // workgroups
  int start;   // PagedArgs::start
  SplitSpace space;
};

// Workgroups that a CU holds (a wavefront a SIMD each), by their registers.  256 channels: in blocks of 32 rows two
// with pieces of two steps fill each other's waits in short ragged runs (N256 H8 to 2,048: 31.5 us, one with pieces of
// four and all queries in registers 33.0), and lose in even and long ones (2,048 each 34.5 and 30.1 us, 8,192 each 114
// and 95), most with a rotary part, where the two have 32 registers spilled and each reload in the tile loop waits for
// the tile on its way (N256 H8 R256 + 64 of 2,048: 79 and 45 us).  In taller blocks one.
constexpr int per_cu(int R, int wq) { return R == 512 || (R == 256 && wq > 1) ? 1 : 2; }

Fp4Plan fp4_plan(int N, int Tq, int H, int R, int Dr, long long max_len) {
  Fp4Plan p;
  const long long rows = (long long)Tq * H, per = N ? (rows + N - 1) / N : 0;
  // Taller blocks convert and put a tile for fewer rows each and read the cache less often (4 chunks of 512 tokens, 96
  // heads of 512 + 64: 1.97 ms with 128 rows, 2.04 with 64, 2.22 with 32); lower ones cut evenly and pad less (N64 H96
  // to 8,192: 117 us with 32 rows, 121 with 64, 123 with 128; of 16,384 each, past the last-level cache, 368 with 32
  // and 309 with 128).  So the tallest that gives each CU a block and pads little.
  auto padded = [&](long long block) { return (per + block - 1) / block * block; };
  auto good = [&](long long block) { return rows / block >= 256 && 8 * padded(block) <= 9 * padded(32); };
  p.wq = good(128) ? 4 : good(64) ? 2 : 1;
  const long long blocks = rows / (32 * p.wq) + N, tiles = (max_len + kTile - 1) / kTile;
  // A tile for each wavefront, if there are too few for all workgroups, and so fewer parts to join (H96 R512 + 64,
  // 2,000 rows: 23.5 us with a workgroup a tile, 20.0 so; N8 H8 R256 of 1,000: no difference; H12 R512 + 64, 900 rows:
  // 16.8 and 17.3).
  const int at_once = 4 / p.wq;
  const long long most = 256 * per_cu(R, p.wq), units = blocks * std::max((tiles + at_once - 1) / at_once, 1ll);
  p.groups = (int)std::min(std::max(units, 1ll), most);
  p.start = blocks > 1 ? kStart / p.wq : 0;
  p.space = split_space(N, p.groups, 32 * p.wq, R);
  return p;
}

// A value that the compiler does not know where it came from: what is computed from it stays where it is used (sums of
// it that are the same in every pass of a loop would each hold a register through the loop).
template <typename T>
__device__ __forceinline__ T opaque(T x) {
  asm("" : "+v"(x));
  return x;
}

// The lane, found again where it is used.
__device__ __forceinline__ int lane_id() {
  return opaque((int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u)));
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

template <int R, int DR, int WQ>
struct Fp4 {
  static constexpr int kThreads = 256, kRows = 32 * WQ, kRow = fp4_row_bytes(R, DR), WT = 4 / WQ;
  static constexpr int KS = R / 16, PS = DR / 16;  // steps of 16 channels: of the latent, of the rotary key
  static constexpr int kOut = R / 32;              // 32-channel tiles of O^T
  // A lane's part of a row is loaded in pieces of E steps (E registers of codes), those of the two halves of the lanes
  // side by side: step s = E p + i is of channels 16 E p + 8 E half + 8 i.
  static constexpr int E = R == 512 || (R == 256 && WQ > 1) ? 4 : 2, kPieces = KS / E, kScales = R / 128;
  static constexpr int kTurn = kPieces / WQ;  // the wavefronts of a tile begin so many pieces apart, and put the first
                                              // kTurn of their pieces into LDS for all
  // At R = 512, and with two workgroups a CU at R = 256, there are no registers for all of the queries: the rotary part
  // and those of some steps are in LDS (each read of one takes the LDS as long as two of the values' reads).  At 256 +
  // 64 with two, that does not suffice (per_cu).
  static constexpr bool far(int s) {
    if (R == 512) return s >= KS || s % 4 == 3 || (WQ != 2 && s % 8 == 1);
    if (R == 256) return WQ == 1 && (s >= KS || s % 2 == 1);
    return false;
  }
  static constexpr int far_at(int s) {  // 1024 bytes a step
    int n = 0;
    for (int i = 0; i < s; ++i) n += far(i);
    return 1024 * n;
  }
  static constexpr int kVal = kTile * R * 2, kBuffers = WQ == 1 ? 1 : 2;  // bytes of a tile's values, tiles of a group
  static constexpr int kQuery = WT * kBuffers * kVal, kQueries = far_at(KS + PS);
  static constexpr int kLds = kQuery + WQ * kQueries;
  static constexpr int kPasses = 32 * R * 2 / (kQuery / 4);  // the queries go through a quarter of the values' LDS
};

template <int R, int DR, int WQ>
__global__ __launch_bounds__(256, per_cu(R, WQ)) void paged_fp4_kernel(PagedWork w, Divide by_page) {
  using C = Fp4<R, DR, WQ>;
  constexpr int D = R + DR, KS = C::KS, PS = C::PS, kOut = C::kOut, WT = C::WT, kRow = C::kRow;
  __shared__ __align__(1024) char lds[C::kLds];
  __shared__ float top[4][32], sums[4][32];
  __shared__ int flags[4];
  const PagedArgs& a = w.a;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wq = wave % WQ, wt = wave / WQ;
  Run run;
  // Workgroups go round the 8 XCDs: neighbours in the work, which share queries or cache rows, are put on one.
  const int xcd = blockIdx.x % 8, each = gridDim.x / 8, over = gridDim.x % 8;
  const int group = xcd * each + min(xcd, over) + blockIdx.x / 8;
  if (!find_run<C::kRows, kTile>(w, group, run)) return;
  const long long begin = run.begin, end = run.end;
  long long base = run.base;  // units before sequence n
  int n = run.n;
  Sequence sq = sequence<C::kRows, kTile>(a, n);
  const float c = a.scale * kda::kLog2e;
  const unsigned lds0 = lds_address(&lds[0]), val = lds0 + wt * (C::kBuffers * C::kVal);
  const unsigned query = lds0 + C::kQuery + wq * C::kQueries + lane * 16;  // the same for wavefronts of the same rows
  // The lane's row of a tile in LDS: its part of piece p (16 E bytes of 32 E) is at (put ^ 32 E p % 256) + 32 E p /
  // 256 * 256.
  constexpr int E = C::E, kPieces = C::kPieces, kTurn = C::kTurn;
  auto put = [](int id) { return (id & 31) * (R * 2) + ((E * (id >> 5)) ^ swizzle<R>(id & 31)) * 16; };

  for (long long u = begin; u < end;) {
    while (u >= base + sq.units()) {
      base += sq.units();
      sq = sequence<C::kRows, kTile>(a, ++n);
    }
    const int block = (int)((u - base) / sq.span), s0 = (int)((u - base) % sq.span);
    const int s1 = (int)min((long long)sq.span, s0 + (end - u));
    const int t0 = max(s0 - a.start, 0), t1 = s1 - a.start;
    const bool whole = t0 == 0 && t1 == sq.tiles;
    const int slot = 2 * group + (u == begin ? 0 : 1);
    u += s1 - s0;
    if (t1 <= t0) continue;  // only units in front of its tiles
    const int rows = sq.Lq * a.H, m0 = block * C::kRows;
    // the last cache row that a row of the block sees
    const int seen = sq.L - sq.Lq + (min(rows, m0 + C::kRows) - 1) / a.H;
    const int stop = min(t1, seen < 0 ? 0 : seen / kTile + 1), count = stop - t0;
    // this wavefront's tiles: t0 + wt + WT i for i < turns; with barriers in the loop, all wavefronts go round as often
    const int turns = count <= 0 ? 0 : WQ == 1 ? (count - wt + WT - 1) / WT : (count + WT - 1) / WT;
    const int* table = a.table + (long long)n * a.max_pages;
    const int last = min(stop * kTile, sq.L);  // behind the last row of the run
    const int mi = m0 + 32 * wq + (lane & 31);
    const bool on = mi < rows;
    const int lim = on ? sq.L - sq.Lq + mi / a.H : INT_MAX;  // the last cache row that the lane's row sees

    f32x16 acc[kOut];
#pragma unroll
    for (int d = 0; d < kOut; ++d) acc[d] = f32x16{};
    float m = -FLT_MAX, l = 0.f;
    if (WQ > 1) lds_barrier();  // the run before is done with the LDS
    if (turns > 0) {
      bf16x8 qf[KS + PS];
      // Through LDS (this wavefront's part of the values'), so that each load takes whole rows: 16 bytes a lane from 32
      // rows would take 64 lines for a part of each (18,000 cycles a block of 128 rows; 6,000).  A row that is not one
      // reads the last again, and is not written.
      auto load_query = [&] {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // what this wavefront put there last is there
        constexpr int kPasses = C::kPasses, kRun = kPieces / kPasses, kChunks = 2 * E * kRun, kAt = kChunks * 16;
        constexpr int kMany = 64 / kChunks;  // rows of a load, if there are several
        auto place = [](int r) { return kChunks >= 16 ? r & 15 : (r >> 1) & 7; };
        const int id = lane_id(), first = min(m0 + 32 * wq, rows - 1);
        const bf16* const q = a.q + ((long long)sq.first * a.H + first) * D;
        const int end_row = rows - 1 - first;
        const bf16* const mine = q + min(id & 31, end_row) * D;
#pragma unroll
        for (int s = 0; s < PS; ++s) qf[KS + s] = *(const bf16x8*)(mine + R + 16 * s + 8 * (id >> 5));
        const unsigned stage = lds0 + wave * (C::kQuery / 4);
        const unsigned from_lds = stage + (id & 31) * kAt;
#pragma unroll
        for (int pass = 0; pass < kPasses; ++pass) {
          if (pass > 0) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
          for (int i = 0; i < 32 / kMany; ++i) {
            const int r = i * kMany + id / kChunks, chunk = (id % kChunks) ^ place(r);
            const int p = (chunk / (2 * E) + pass * kRun + wq * kTurn) % kPieces;
            load_lds(q, (min(r, end_row) * D + 16 * E * p + 8 * (chunk % (2 * E))) * 2, stage + i * 1024);
          }
          asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
          for (int s = pass * kRun * E; s < (pass + 1) * kRun * E; ++s) {
            const int chunk = 2 * E * (s / E - pass * kRun) + s % E;
            qf[s] = *(const lds_bf16x8*)(from_lds + 16 * ((chunk + E * (id >> 5)) ^ place(id & 31)));
          }
        }
#pragma unroll
        for (int s = 0; s < KS + PS; ++s)
          if (C::far(s)) *(lds_u32x4*)(query + C::far_at(s)) = __builtin_bit_cast(u32x4, qf[s]);
        __builtin_amdgcn_sched_barrier(0);
        if (WQ > 1) lds_barrier();  // the values' LDS is all the wavefronts' again
      };
      auto far_query = [&](int s) { return __builtin_bit_cast(bf16x8, *(lds_u32x4*)(query + C::far_at(s))); };
      unsigned code[KS];
      u32x4 pe[PS > 0 ? PS : 1];
      unsigned scale[C::kScales], next_scale[C::kScales];
      // Where the lane's row of a tile lies (its half of each piece, and what follows the codes), whether it is there.
      int page = -1, off = 0;
      bool in = false, next_in = false;
      unsigned long long row = 0, row_end = 0;
      auto look_up = [&](int i) {  // of tile i; compared without a sign: it may begin past what 31 bits count
        const int j = (t0 + wt + WT * i) * kTile + (lane_id() & 31);
        page = -1;
        if ((unsigned)j < (unsigned)last) {
          const unsigned p = by_page.of(j);
          off = j - (int)p * a.page_size;
          // below 512 channels with a zero of its own: else it is one of a vector of zeros, which is spilled
          page = R == 512 ? table[p] : table[(unsigned long long)opaque(0u) << 32 | p];
        }
      };
      auto find = [&] {  // the tile looked up last is the next
        next_in = (unsigned)page < (unsigned)a.num_pages;
        const long long r = next_in ? page * a.page_size + off : 0;
        const int h = lane_id() >> 5;
        row = (unsigned long long)a.cache + r * kRow + 4 * E * h;
        row_end = (unsigned long long)a.cache + r * kRow + R / 2 + 16 * h;
      };
      auto load_codes = [&](int p) {
        const auto from = (global_char*)row + 8 * E * ((p + wq * kTurn) % kPieces);
        if constexpr (E == 4)
          *(u32x4*)(code + 4 * p) = *(global_u32x4*)from;
        else
          *(u32x2*)(code + 2 * p) = *(global_u32x2*)from;
      };
      auto load_key = [&](int s) { pe[s] = *(global_u32x4*)((global_char*)row_end + 32 * s); };
      // The scales in the order of the wavefront's pieces: R / 32 bytes, piece p has byte p (E = 2) or 2 p + half (E =
      // 4).
      constexpr int kBytes = E / 2, kRoll = kBytes * kTurn;
      auto load_scales = [&] {
        const auto from = (global_char*)row_end - 16 * (lane_id() >> 5) + 2 * DR;
#pragma unroll
        for (int i = 0; i < C::kScales; ++i)
          next_scale[i] = *(global_u32*)(from + 4 * ((i + wq * kRoll / 4) % C::kScales));
      };
      bool wide = false;               // a scale of 2^33 or more: bit 7 of a byte and one of the two below
      unsigned bad = 0, next_bad = 0;  // the tile's rows with a scale that stands for NaN
      // Rows that are not there have a scale of 2^-127, and so any finite values.  So have those with a NaN, whose scores
      // are made NaN (mask): in the sums a value counts for rows that do not see it too, with a weight of 0.
      auto turn_scales = [&] {
        const int h = E == 4 ? 8 * (lane_id() >> 5) : 0;
        unsigned large = 0;
#pragma unroll
        for (int i = 0; i < C::kScales; ++i) large |= next_scale[i] & (next_scale[i] << 1 | next_scale[i] << 2);
        next_bad = 0;
        bool kept = next_in;
        if (__any(kept && (large & 0x80808080u))) {
          bool nan = false;
#pragma unroll
          for (int i = 0; i < C::kScales; ++i)
            nan |= ((next_scale[i] & 0x7f7f7f7fu) + 0x01010101u * (256 - kFp4NaN) & next_scale[i] & 0x80808080u) != 0;
          next_bad = (unsigned)__ballot(kept && nan);
          kept = kept && !nan;
          wide |= kept && (large & 0x80808080u);
        }
#pragma unroll
        for (int i = 0; i < C::kScales; ++i) {
          const unsigned x = kRoll % 4 == 0 ? next_scale[i]
                                            : __builtin_amdgcn_alignbit(next_scale[(i + 1) % C::kScales], next_scale[i],
                                                                        wq * kRoll % 4 * 8);
          scale[i] = kept ? x >> h : 0u;
        }
      };

      f32x16 S;  // S^T of a tile; register i: the lane's row, tile row acc_row(i)
      bf16x8 P[2];
      auto scale_of = [&](int s) {  // step s's, as a float
        constexpr int kTop = 23;
        const int at_bit = 8 * (kBytes * (s / E) % 4);
        const unsigned x = scale[kBytes * (s / E) / 4];
        return __builtin_bit_cast(float, (at_bit <= kTop ? x << (kTop - at_bit) : x >> (at_bit - kTop)) & 255u << kTop);
      };
      auto score = [&](u32x4 k, bf16x8 q, bool first) {
        if constexpr (R == 512) {
          // In vector registers: the accumulators are full.  (The compiler takes all results of a kernel into one of
          // the two halves of the register file.)  The waits that it would place are written out: 2 between a vector
          // instruction's result and a matrix instruction that reads it.
          f32x16 x = S;
          if (first)
            asm("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, 0" : "=&v"(x) : "v"(k), "v"(q));
          else
            asm("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(x) : "v"(k), "v"(q));
          S = x;
        } else {
          S = mma(__builtin_bit_cast(bf16x8, k), q, first ? f32x16{} : S);
        }
      };
      // The scores of the tile in the registers (its values into `to`, the tile after it into the registers) and,
      // where SUMS, beside them the sums of the tile in `from` with the weights P.  A wavefront issues an instruction
      // every 4 cycles at best (a conversion takes 8) and a product takes 32, so what is between two products is kept
      // even: 3,700 cycles a tile at R = 512, where the 68 products alone take 2,176.
      auto products = [&](auto scores_too, auto sums_too, unsigned from, unsigned to) {
        constexpr bool kScores = decltype(scores_too)::value, kSums = decltype(sums_too)::value;
        // Steps that the reads of values are ahead.  With one buffer a tile is put where the one before is read: the
        // 16 E channels of piece p in steps E p .. E p + E - 1, so those of the E - 1 steps after have to be on their
        // way.
        constexpr int kFirst = C::kBuffers == 1 ? E : 2;
        static_assert(C::kBuffers > 1 || kFirst >= E);
        bf16x8 v[kFirst];
        const unsigned at_from = opaque(from + LaneAt<R>(lane_id()).col);
        auto read = [&](int e) {  // A operand of step e: channels 32 (e / 2) .., rows 16 (e % 2) ..
          const int d = e / 2, to_tile = 16 * (e % 2) * (R * 2) + 256 * (d / 4);
          const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)((at_from ^ (64 * (d % 4))) + to_tile));
          const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_s16x4*)((at_from ^ (64 * (d % 4) + 32)) + (to_tile + 8 * (R * 2))));
          return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        };
        if constexpr (kSums) {
#pragma unroll
          for (int e = 0; e < kFirst; ++e) v[e] = read(e);
        }
        u32x4 k = {};
        bf16x8 far = {}, far_key = {};  // queries from LDS, read ahead
        constexpr int kEvery = PS > 0 ? KS / PS : 1;  // a step of the rotary key after so many of the latent
        float by = 0.f;
        if constexpr (kScores) {
          load_scales();
          by = scale_of(0);
          k = fp4_values(code[0], by);
          if (C::far(1)) far = far_query(1);
        }
        constexpr int kShare = 32 * E * kTurn;  // bytes of a row that this wavefront puts
        const unsigned at_put = opaque(((to + put(lane_id())) ^ (wq * kShare % 256)) + 256 * (wq * kShare / 256));
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          u32x4 next = k;
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (kScores) {
            score(k, C::far(s) ? far : qf[s], s == 0);
            if (s + 1 < KS) {
              if ((s + 1) % E == 0) by = scale_of(s + 1);
              next[0] = fp4_pair<0>(code[s + 1], by);
              next[1] = fp4_pair<1>(code[s + 1], by);
            }
            if (s / E < kTurn)
              *(lds_u32x4*)((at_put ^ (32 * E * (s / E) % 256 + 16 * (s % E))) + 256 * (32 * E * (s / E) / 256)) = k;
            if (PS > 0 && s % kEvery == kEvery / 2 && C::far(KS)) far_key = far_query(KS + s / kEvery);
          }
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (kSums) acc[s / 2] = mma(v[s % kFirst], P[s % 2], acc[s / 2]);
          if constexpr (kScores) {
            if (s + 1 < KS) {
              next[2] = fp4_pair<2>(code[s + 1], by);
              next[3] = fp4_pair<3>(code[s + 1], by);
            }
            if (s + 2 < KS && C::far(s + 2)) far = far_query(s + 2);
            if (s % E == E - 1) load_codes(s / E);
          }
          if constexpr (kSums)
            if (s + kFirst < KS) v[s % kFirst] = read(s + kFirst);
          if constexpr (kScores && PS > 0)
            if (s % kEvery == kEvery - 1) {
              __builtin_amdgcn_sched_barrier(0);
              score(pe[s / kEvery], C::far(KS) ? far_key : qf[KS + s / kEvery], false);
              load_key(s / kEvery);
            }
          k = next;
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (kScores) {
          turn_scales();
          // the waits between a matrix instruction's result and its use, which the compiler does not place here
          if constexpr (R == 512) {
            f32x16 x = S;
            asm("s_nop 15\n\ts_nop 7" : "+v"(x));
            S = x;
          }
        }
      };
      bool passed = false;  // a score is above its reference by more than 2^60
      auto highest = [&] {
        float x = S[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) x = fmaxf(x, S[i]);
        return x * c;
      };
      auto mask = [&](int i) {
        const int j0 = (t0 + wt + WT * i) * kTile;
        const unsigned bits = (unsigned)__ballot(in);
        if (bits == ~0u && bad == 0 && j0 + kTile - 1 <= sq.L - sq.Lq + m0 / a.H) return;
        const int h = 4 * (lane_id() >> 5), sees = lim - j0 - h;  // rows up to this one, of those from h on
        if (bad != 0) {
          const unsigned nans = bad >> h;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if ((nans >> acc_row(e, 0)) & 1) S[e] = __builtin_nanf("");
        }
        const unsigned mine = bits >> h;
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (!((mine >> acc_row(e, 0)) & 1) || acc_row(e, 0) > sees) S[e] = -INFINITY;
      };
      auto softmax = [&] {
        f32x16 p;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          p[i] = kda::fast_exp2(__builtin_fmaf(S[i], c, -m));
          sum += p[i];
        }
        l += sum;
        P[0] = acc_frag(p, 0);
        P[1] = acc_frag(p, 1);
        passed |= highest() > m + 60.f;
      };
      constexpr std::true_type yes{};
      constexpr std::false_type no{};
      // The first tile into the registers, and the next one's place.
      auto start = [&] {
        look_up(0);
        find();
        look_up(1);
#pragma unroll
        for (int p = 0; p < kPieces; ++p) load_codes(p);
#pragma unroll
        for (int s = 0; s < PS; ++s) load_key(s);
        load_scales();
      };
      auto step = [&](int i) {  // the tile in the registers becomes the present one, i
        in = next_in, bad = next_bad;
        find();
        look_up(i + 2);
      };

      for (bool again = false;;) {
        unsigned from = val, to = C::kBuffers == 2 ? val + C::kVal : val;
        start();
        load_query();
        turn_scales();
        step(0);
        products(yes, no, from, from);
        mask(0);
        if (!again) m = fmaxf(halves_max(highest()), -FLT_MAX);
        softmax();
        for (int i = 1; i < turns; ++i) {
          if (WQ > 1) lds_barrier();
          step(i);
          products(yes, yes, from, to);
          mask(i);
          softmax();
          const unsigned was = from;
          from = to, to = was;
        }
        if (WQ > 1) lds_barrier();
        products(no, yes, from, to);
        if (again) break;
        again = __any((on && passed) || wide);  // a lane's row of the block may not be there, its row of a tile counts
        if (WQ > 1) {  // the wavefronts' loops have barriers: all do the run again, or none
          if (lane == 0) flags[wave] = again;
          lds_barrier();
          again = uniform((unsigned)(flags[0] | flags[1] | flags[2] | flags[3])) != 0;
          lds_barrier();
        }
        if (!again) break;
        start();
        load_query();
        turn_scales();
        m = -FLT_MAX;
        for (int i = 0; i < turns; ++i) {
          step(i);
          products(yes, no, val, val);
          mask(i);
          m = fmaxf(m, halves_max(highest()));
        }
        l = 0.f;
#pragma unroll
        for (int d = 0; d < kOut; ++d) acc[d] = f32x16{};
        if (WQ > 1) lds_barrier();
      }
    }

    l = halves_sum(l);
    const int id = lane_id(), row = id & 31, mo = m0 + 32 * wq + row;
    const bool written = mo < rows;
    // The sums of a row are handed on in units in which its l is near 1 (scaled by a power of two, exactly): with the
    // run's own reference, far below the row's largest score, what scales them later would leave the range of float32
    // where they, larger than 1, have not.
    const int size = __builtin_amdgcn_frexp_expf(l);
    m += (float)size;
    l = ldexpf(l, -size);
    float f[WT] = {1.f};
    if constexpr (WT > 1) {  // one reference and sum for the wavefronts of the same rows; f: their factors, from this one
      lds_barrier();  // all are done with the values
      if (id < 32) top[wave][row] = m, sums[wave][row] = l;
      lds_barrier();
      l = 0.f;
#pragma unroll
      for (int t = 0; t < WT; ++t) m = fmaxf(m, top[t * WQ + wq][row]);
#pragma unroll
      for (int t = 0; t < WT; ++t) l += sums[t * WQ + wq][row] * kda::fast_exp2(top[t * WQ + wq][row] - m);
#pragma unroll
      for (int t = 0; t < WT; ++t) f[t] = kda::fast_exp2(top[(wt + t) % WT * WQ + wq][row] - m);
    }
    const float fo = l == 0.f ? 0.f : 1.f / l;  // 0: the row sees nothing
    const long long out = (long long)sq.first * a.H + mo, to = (long long)slot * C::kRows + 32 * wq + row;
    if (written && id < 32 && wt == 0) {
      if (!whole) {
        w.ml[2 * to] = m;
        w.ml[2 * to + 1] = l;
      } else if (a.lse) {
        a.lse[out] = l == 0.f ? -INFINITY : (m + log2f(l)) * (1.f / kda::kLog2e);
      }
    }
    bf16* const to_o = a.o + out * R + 4 * (id >> 5);
    float* const to_part = w.po + to * R + 4 * (id >> 5);
    auto emit = [&](auto final) {
      auto shifted = [&](int d, int i) {
        return f32x4{ldexpf(acc[d][i], -size), ldexpf(acc[d][i + 1], -size), ldexpf(acc[d][i + 2], -size),
                     ldexpf(acc[d][i + 3], -size)};
      };
      auto write = [&](int d, int i, f32x4 x) {  // 4 channels of the lane's row
        const int ch = 32 * d + acc_row(i, 0);
        if constexpr (decltype(final)::value)
          *(u32x2*)(to_o + ch) = u32x2{kda::pk_bf16(x[0] * fo, x[1] * fo), kda::pk_bf16(x[2] * fo, x[3] * fo)};
        else
          *(f32x4*)(to_part + ch) = x;
      };
      if constexpr (WT == 1) {
        if (!written) return;
#pragma unroll
        for (int d = 0; d < kOut; ++d) {
#pragma unroll
          for (int i = 0; i < 16; i += 4) write(d, i, shifted(d, i));
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
        // Each of the WT wavefronts of the same rows sums a share of the channels, in two rounds (the LDS of one tile's
        // values a wavefront holds half of what the others hand over).  1024 bytes, 16 a lane, a piece of 4 channels.
        constexpr int kShare = kOut / WT, kRound = kShare * 2;  // 32-channel tiles, pieces a round
        static_assert(4 * (WT - 1) * kRound * 1024 <= C::kQuery, "the values' LDS holds a round");
        const unsigned there = lds0 + wq * (WT * (WT - 1) * kRound * 1024) + id * 16;
        auto mine = [&](int t, int round, int e) {
          const int x = round * kRound + e, d = t * kShare + x / 4, i = x % 4 * 4;
          return shifted(d, i);
        };
#pragma unroll
        for (int round = 0; round < 2; ++round) {
#pragma unroll
          for (int t = 0; t < WT; ++t)  // to wavefront t, from its ((wt - t) mod WT)-th neighbour
            if (t != wt) {
              const unsigned piece = there + (t * (WT - 1) + (wt - t + WT) % WT - 1) * (kRound * 1024);
#pragma unroll
              for (int e = 0; e < kRound; ++e) {
                *(lds_f32x4*)(piece + e * 1024) = mine(t, round, e);
                if (e % 4 == 3) __builtin_amdgcn_sched_barrier(0);
              }
            }
          lds_barrier();
#pragma unroll
          for (int t = 0; t < WT; ++t)
            if (t == wt && written) {
#pragma unroll
              for (int e = 0; e < kRound; ++e) {
                const int x = round * kRound + e;
                f32x4 sum = mine(t, round, e) * f[0];
#pragma unroll
                for (int g = 0; g < WT - 1; ++g)
                  sum += *(lds_f32x4*)(there + (t * (WT - 1) + g) * (kRound * 1024) + e * 1024) * f[g + 1];
                write(t * kShare + x / 4, x % 4 * 4, sum);
                if (e % 4 == 3) __builtin_amdgcn_sched_barrier(0);
              }
            }
          lds_barrier();
        }
      }
    };
    if (whole)
      emit(std::true_type{});
    else
      emit(std::false_type{});
  }
}

template <int R, int DR, int WQ>
hipError_t launch(const PagedWork& w, const Fp4Plan& p, hipStream_t stream) {
  using C = Fp4<R, DR, WQ>;
  paged_fp4_kernel<R, DR, WQ><<<dim3(p.groups), dim3(C::kThreads), 0, stream>>>(w, Divide(w.a.page_size));
  // a block's parts: with few rows it pays sooner to join them by several workgroups a row (8 rows of 8 parts: 6.0 us
  // with a wavefront a row, 3.9 with a workgroup for 64 channels)
  const int few = (long long)w.a.Tq * w.a.H * (R / 64) <= 4096 ? 3 : 8;
  launch_combine<R, C::kRows, kTile>(w, p.groups, few, stream);
  return hipGetLastError();
}

template <int R, int DR>
hipError_t launch(const PagedArgs& a, hipStream_t stream) {
  const Fp4Plan p = fp4_plan(a.N, a.Tq, a.H, R, DR, (long long)a.max_pages * a.page_size);
  PagedWork w = split_work(a, p.space);
  w.a.start = p.start;
  switch (p.wq) {
    case 1: return launch<R, DR, 1>(w, p, stream);
    case 2: return launch<R, DR, 2>(w, p, stream);
    default: return launch<R, DR, 4>(w, p, stream);
  }
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
