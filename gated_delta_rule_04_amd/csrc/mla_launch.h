// Internal interface between the latent attention's C-ABI layer (mla_api.hip)
// and its kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "kda_common.h"

namespace mla {

using kda::bf16;

struct AppendArgs {
  const bf16* c;        // [T][R + Dr]
  const float* weight;  // [R] or NULL
  float eps;
  const float* rope;    // [num_pos][Dr] (cos, then sin) or NULL
  int num_pos;
  int interleaved;
  const int* positions;
  const int* slots;
  void* cache;          // [num_slots] rows: bf16 [R + Dr], or fp4_row_bytes(R, Dr) bytes
  int num_slots;
  const bf16* q_pe;     // [T][H][Dr] or NULL
  bf16* q;              // [T][H][R + Dr]
  int T, H;
};
hipError_t launch_append(int R, int Dr, const AppendArgs& a, hipStream_t stream);
hipError_t launch_append_fp4(int R, int Dr, const AppendArgs& a, hipStream_t stream);

// A row of the 4-bit cache: codes, rotary key, scales, zeros to a multiple of 16.
__host__ __device__ constexpr int fp4_row_bytes(int R, int Dr) { return (R / 2 + 2 * Dr + R / 32 + 15) / 16 * 16; }

struct GatherArgs {
  const unsigned char* cache;  // [num_pages * page_size][fp4_row_bytes]
  const int* table;            // [N][max_pages]
  const int* cu;               // [N + 1]
  const int* starts;           // [N] or NULL
  bf16* rows;                  // [T][R + Dr]
  int N, T, num_pages, page_size, max_pages;
};
hipError_t launch_gather(int R, int Dr, const GatherArgs& a, hipStream_t stream);

struct PlanArgs {
  const int *new_lens, *seq_lens;  // [N]
  int* table;                      // [N][max_pages]
  const int *free_pages, *free_count;
  int *cu, *positions, *slots, *kv_lens, *lens_out, *free_out;
  int* top;                        // workspace [N]: where a sequence's first new page lies in the list
  int num_free, N, T, page_size, max_pages, capacity;
};
hipError_t launch_plan(const PlanArgs& p, hipStream_t stream);

struct ReleaseArgs {
  const unsigned char* finished;  // [N]
  const int *seq_lens, *table;
  int* free_pages;
  const int* free_count;
  int *lens_out, *free_out;
  int* first;                     // workspace [N + 2]: ends of the sequences' pages in the list, and the list's old end
  int num_free, N, page_size, max_pages, capacity;
};
hipError_t launch_release(const ReleaseArgs& p, hipStream_t stream);

struct PagedArgs {
  const bf16* q;      // [Tq][H][R + Dr]
  const void* cache;  // [num_pages * page_size] rows: bf16 [R + Dr], or fp4_row_bytes(R, Dr) bytes
  const int* table;   // [N][max_pages]
  const int* lens;    // [N]
  const int* cu;      // [N + 1] or NULL: one token a sequence
  bf16* o;            // [Tq][H][R]
  float* lse;         // [Tq][H] or NULL
  int N, Tq, H, num_pages, page_size, max_pages;
  float scale;
  int start = 0;  // what beginning a block of rows costs, in tiles, where the work is cut evenly
  void* ws;
};
size_t paged_workspace(int N, int Tq, int H, int R, int Dr, long long max_len);
hipError_t launch_paged(int R, int Dr, const PagedArgs& a, hipStream_t stream);
size_t paged_fp4_workspace(int N, int Tq, int H, int R, int Dr, long long max_len);
hipError_t launch_paged_fp4(int R, int Dr, const PagedArgs& a, hipStream_t stream);

// Expanded form.  Tokens are counted through the batch (b * T + t); documents
// come from cu, or are the rows of the batch when cu is NULL.
struct AttnArgs {
  const bf16* q;     // [tokens][H][Dn + Dr]
  const bf16* kv;    // [tokens][H][Dn + Dv]
  const bf16* k_pe;  // [tokens][Dr]
  const bf16* dout;  // backward
  bf16* o;           // forward
  float* lse;        // forward: written when set; backward: read
  bf16 *dq, *dkv, *dk_pe;
  const int* cu;
  int N, T, H;       // documents; tokens of a batch row, or all of them with cu
  float scale;
  float* delta;      // backward workspace: [tokens][H][2], lse in log2 units and delta
  float* pe_part;    // backward workspace: [H][tokens][Dr]
  int tokens;
};
hipError_t launch_attn_fwd(int Dn, int Dr, const AttnArgs& a, hipStream_t stream);
hipError_t launch_attn_bwd(int Dn, int Dr, const AttnArgs& a, hipStream_t stream);

// First and last-plus-one token of document n.
__device__ __forceinline__ void document(const int* cu, int T, int n, int& begin, int& end) {
  if (cu) {
    begin = min(max(cu[n], 0), T);
    end = min(max(cu[n + 1], begin), T);
  } else {
    begin = n * T;
    end = begin + T;
  }
}

}  // namespace mla
