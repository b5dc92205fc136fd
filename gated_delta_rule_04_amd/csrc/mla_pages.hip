// Pages of the paged latent cache: the new tokens' pages, slots and positions
// from the requests' lengths (plan), and a finished request's pages back to the
// free list (release).
//
// A prefix sum over the sequences decides everything (who is served, which piece
// of the stack of free pages is whose), then every token or page is on its own.
// The sum is one workgroup's, a run of sequences a thread.  Nothing but the latency
// of the few dependent reads bounds it (lengths, then a token's sequence, page and
// table entry): 256 single tokens 5.8 us in one launch; 25,000 tokens of 256
// sequences 4.4 + 4.8 us in two.  Up to 1024 tokens or pages the workgroup of the
// sum goes on with them: a second launch costs more than its one pass.  No
// atomics: the same lengths give the same pages.

#include <limits.h>

#include "mla_launch.h"

namespace mla {
namespace {

constexpr int kScan = 1024;  // threads of the prefix sum
constexpr int kFill = 256;   // threads of a workgroup that goes through tokens or pages

// Sum of x over the threads before this one, and over all of them.
__device__ __forceinline__ long long before_me(long long x, long long& all) {
  __shared__ long long part[kScan / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  long long in = x;
  for (int m = 1; m < 64; m <<= 1) {
    const long long y = __shfl_up(in, m);
    if (lane >= m) in += y;
  }
  __syncthreads();
  if (lane == 63) part[wave] = in;
  __syncthreads();
  long long before = 0;
  all = 0;
  for (int i = 0; i < kScan / 64; ++i) {
    if (i < wave) before += part[i];
    all += part[i];
  }
  return before + in - x;
}

// The last n in [0, N) with first[n] <= t, for a t not below first[0].
__device__ __forceinline__ int holder(const int* first, int N, int t) {
  int lo = 0, hi = N;
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (first[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

struct Lengths {
  long long s, a;  // rows in the cache, new tokens
  __device__ __forceinline__ Lengths(const PlanArgs& p, int n)
      : s(min(max(p.seq_lens[n], 0), p.capacity)), a(max(p.new_lens[n], 0)) {}
  __device__ __forceinline__ bool fits(const PlanArgs& p, long long upto) const {
    return s + a <= p.capacity && upto <= p.T;
  }
  // pages that the new tokens need
  __device__ __forceinline__ int need(const PlanArgs& p) const {
    const unsigned P = p.page_size;
    return a > 0 ? (int)(((unsigned)(s + a) + P - 1) / P - ((unsigned)s + P - 1) / P) : 0;
  }
};

__device__ __forceinline__ void plan_sequences(const PlanArgs& p) {
  const int per = (p.N + kScan - 1) / kScan, n0 = min((int)threadIdx.x * per, p.N), n1 = min(n0 + per, p.N);
  const int free = min(max(p.free_count[0], 0), p.num_free);
  long long tokens = 0, pages = 0, all_tokens, all_pages;
  for (int n = n0; n < n1; ++n) tokens += Lengths(p, n).a;
  const long long before = before_me(tokens, all_tokens);
  long long upto = before;
  for (int n = n0; n < n1; ++n) {
    const Lengths l(p, n);
    upto += l.a;
    if (l.fits(p, upto)) pages += l.need(p);
  }
  long long took = before_me(pages, all_pages), most = 0;
  upto = before;
  for (int n = n0; n < n1; ++n) {
    const Lengths l(p, n);
    upto += l.a;
    const bool fits = l.fits(p, upto);
    const int need = fits ? l.need(p) : 0;
    took += need;
    const bool served = l.a == 0 || (fits && (need == 0 || took <= free));
    if (served && need) most = took;
    p.top[n] = served ? (int)(free - (took - need)) - 1 : -1;
    p.cu[n + 1] = (int)min(upto, (long long)p.T);
    p.kv_lens[n] = served ? (int)(l.s + l.a) : -1;
    p.lens_out[n] = (int)(served ? l.s + l.a : l.s);
  }
  // the sequences that got pages are a prefix of those that asked: the last one's sum is the largest
  for (int m = 1; m < 64; m <<= 1) most = max(most, __shfl_xor(most, m));
  __shared__ long long largest[kScan / 64];
  if ((threadIdx.x & 63) == 0) largest[threadIdx.x >> 6] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kScan / 64; ++i) most = max(most, largest[i]);
    p.cu[0] = 0;
    p.free_out[0] = free - (int)most;
  }
}

__device__ __forceinline__ void plan_token(const PlanArgs& p, int t) {
  int pos = 0, slot = -1;
  if (t < p.cu[p.N]) {
    const int n = holder(p.cu, p.N, t), begin = p.cu[n], kv = p.kv_lens[n];
    if (kv >= 0) {
      const int s = kv - (p.cu[n + 1] - begin);
      const unsigned P = p.page_size, first = ((unsigned)s + P - 1) / P;
      pos = s + t - begin;
      const unsigned i = (unsigned)pos / P, in = (unsigned)pos - i * P;
      int* entry = p.table + (long long)n * p.max_pages + i;
      int page;
      if (i >= first) {
        page = p.free_pages[p.top[n] - (int)(i - first)];
        if (in == 0) *entry = page;
      } else {
        page = *entry;
      }
      const long long row = (long long)page * P + in;
      if (page >= 0 && row <= INT_MAX) slot = (int)row;
    }
  }
  p.positions[t] = pos;
  p.slots[t] = slot;
}

template <bool ALL>
__global__ __launch_bounds__(kScan) void plan_kernel(PlanArgs p) {
  plan_sequences(p);
  if constexpr (ALL) {
    __syncthreads();  // what the sum wrote to global memory is read by the same workgroup
    for (int t = threadIdx.x; t < p.T; t += kScan) plan_token(p, t);
  }
}

__global__ __launch_bounds__(kFill) void plan_tokens_kernel(PlanArgs p) {
  const int t = blockIdx.x * kFill + threadIdx.x;
  if (t < p.T) plan_token(p, t);
}

// Where the pages of sequence n go in the list: first[n] .. first[n + 1] - 1.
__device__ __forceinline__ void release_sequences(const ReleaseArgs& p) {
  const int per = (p.N + kScan - 1) / kScan, n0 = min((int)threadIdx.x * per, p.N), n1 = min(n0 + per, p.N);
  const int free = min(max(p.free_count[0], 0), p.num_free);
  auto pages = [&](int n) {
    const unsigned s = min(max(p.seq_lens[n], 0), p.capacity), P = p.page_size;
    return p.finished[n] ? (int)((s + P - 1) / P) : 0;
  };
  long long mine = 0, all;
  for (int n = n0; n < n1; ++n) mine += pages(n);
  long long at = free + before_me(mine, all);
  for (int n = n0; n < n1; ++n) {
    p.first[n] = (int)min(at, (long long)p.num_free);
    at += pages(n);
    p.lens_out[n] = p.finished[n] ? 0 : min(max(p.seq_lens[n], 0), p.capacity);
  }
  if (threadIdx.x == 0) {
    const int end = (int)min(free + all, (long long)p.num_free);
    p.first[p.N] = end;
    p.first[p.N + 1] = free;
    p.free_out[0] = end;
  }
}

__device__ __forceinline__ void release_pages(const ReleaseArgs& p, int me, int step) {
  const int end = p.first[p.N];
  for (int e = p.first[p.N + 1] + me; e < end; e += step) {
    const int n = holder(p.first, p.N, e);
    p.free_pages[e] = p.table[(long long)n * p.max_pages + (e - p.first[n])];
    if (e > INT_MAX - step) break;
  }
}

template <bool ALL>
__global__ __launch_bounds__(kScan) void release_kernel(ReleaseArgs p) {
  release_sequences(p);
  if constexpr (ALL) {
    __syncthreads();
    release_pages(p, threadIdx.x, kScan);
  }
}

__global__ __launch_bounds__(kFill) void release_pages_kernel(ReleaseArgs p) {
  release_pages(p, blockIdx.x * kFill + threadIdx.x, gridDim.x * kFill);
}

}  // namespace

hipError_t launch_plan(const PlanArgs& p, hipStream_t stream) {
  if (p.T <= kScan) {
    plan_kernel<true><<<dim3(1), dim3(kScan), 0, stream>>>(p);
  } else {
    plan_kernel<false><<<dim3(1), dim3(kScan), 0, stream>>>(p);
    plan_tokens_kernel<<<dim3((p.T + kFill - 1) / kFill), dim3(kFill), 0, stream>>>(p);
  }
  return hipGetLastError();
}

hipError_t launch_release(const ReleaseArgs& p, hipStream_t stream) {
  const long long most = (long long)p.N * p.max_pages < p.num_free ? (long long)p.N * p.max_pages : p.num_free;
  if (most <= kScan) {
    release_kernel<true><<<dim3(1), dim3(kScan), 0, stream>>>(p);
  } else {
    release_kernel<false><<<dim3(1), dim3(kScan), 0, stream>>>(p);
    const long long blocks = (most + kFill - 1) / kFill;
    release_pages_kernel<<<dim3((unsigned)(blocks < 1024 ? blocks : 1024)), dim3(kFill), 0, stream>>>(p);
  }
  return hipGetLastError();
}

}  // namespace mla
