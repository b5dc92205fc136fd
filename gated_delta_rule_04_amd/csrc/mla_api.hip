// C-ABI entry points of the latent attention (kda_mla_*): argument validation
// and kernel launches.  Every check runs on the host before the first HIP
// call; see include/kda.h.

#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "kda.h"
#include "mla_launch.h"

namespace {

constexpr int kMaxHeads = 1024;     // a 128-token span of one tensor stays below 2 GiB
constexpr int kMaxPagedSeqs = 65536;
// A launch counts its threads in 32 bits, and workgroups have 256: tiles of 128
// tokens of every document and head, 4 rows a workgroup of the paged form's
// join, 16 threads a token for dk_pe.
constexpr int kMaxBlocks = (1 << 24) - 1;
constexpr int kMaxPagedRows = (1 << 26) - 256;
constexpr int kMaxTokens = 1 << 27;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <typename... P>
bool aligned16(P... p) {
  return (aligned(p, 16) && ...);
}

// bf16 only: the other types of the enumeration are named, but not built.
kda_status check_type(kda_dtype dt) {
  if (dt == KDA_BF16) return KDA_OK;
  return dt == KDA_F32 || dt == KDA_F16 ? KDA_ERR_UNSUPPORTED : KDA_ERR_DTYPE;
}

bool latent_ok(int R, int Dr) { return (R == 128 || R == 256 || R == 512) && (Dr == 0 || Dr == 64); }
bool heads_ok(int Dn, int Dr, int Dv) { return (Dn == 64 || Dn == 128) && Dv == Dn && (Dr == 0 || Dr == 64); }
bool scale_ok(float s) { return s > 0.f && isfinite(s); }

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

kda_status check_attn(const int* cu, int num_seqs, int B, int T, int H, int Dn, int Dr, int Dv, float scale,
                      kda_dtype dt) {
  if (const kda_status s = check_type(dt)) return s;
  if (B < 0 || T < 0 || H <= 0 || H > kMaxHeads || num_seqs < 0 || !scale_ok(scale)) return KDA_ERR_SHAPE;
  if (!heads_ok(Dn, Dr, Dv)) return KDA_ERR_UNSUPPORTED;
  if (cu ? B != 1 : num_seqs != B) return KDA_ERR_SHAPE;
  const long long tokens = (long long)B * T;
  if (tokens > kMaxTokens || (tokens / 128 + num_seqs + 1) * H > kMaxBlocks) return KDA_ERR_SHAPE;
  return KDA_OK;
}

struct BwdLayout {
  size_t pe_part, total;
};
BwdLayout bwd_layout(int B, int T, int H, int Dr) {
  BwdLayout L;
  const size_t rows = (size_t)B * T * H;
  L.pe_part = align256(rows * 2 * sizeof(float));
  L.total = L.pe_part + align256(rows * Dr * sizeof(float));
  return L;
}

}  // namespace

extern "C" {

kda_status kda_mla_cache_append(const void* c_kv, const float* norm_weight, float eps, const float* rope,
                                int num_pos, int interleaved, const int* positions, const int* slots, void* cache,
                                int num_pages, int page_size, const void* q_pe, void* q, int T, int H, int R, int Dr,
                                kda_dtype dt, void* stream) {
  if (const kda_status s = check_type(dt)) return s;
  if (T < 0 || T > kMaxTokens || num_pages < 0 || page_size < 1 || !(eps >= 0.f)) return KDA_ERR_SHAPE;
  if ((long long)num_pages * page_size > INT_MAX) return KDA_ERR_SHAPE;
  if (q_pe && (H <= 0 || H > kMaxHeads)) return KDA_ERR_SHAPE;
  if (((long long)T * (64 + 4 * (1 + (q_pe ? H : 0)))) / 256 + 2 > kMaxBlocks) return KDA_ERR_SHAPE;
  if (rope && num_pos < 1) return KDA_ERR_SHAPE;
  if (!latent_ok(R, Dr) || (Dr == 0 && (q_pe || rope))) return KDA_ERR_UNSUPPORTED;
  if (T == 0) return KDA_OK;
  if (!c_kv || !slots || (num_pages > 0 && !cache) || (rope && !positions) || (q_pe && !q)) return KDA_ERR_NULL;
  if (!aligned16(c_kv, norm_weight, rope, cache, q_pe, q)) return KDA_ERR_UNSUPPORTED;
  mla::AppendArgs a;
  a.c = static_cast<const mla::bf16*>(c_kv);
  a.weight = norm_weight;
  a.eps = eps;
  a.rope = rope;
  a.num_pos = num_pos;
  a.interleaved = interleaved;
  a.positions = positions;
  a.slots = slots;
  a.cache = static_cast<mla::bf16*>(cache);
  a.num_slots = num_pages * page_size;
  a.q_pe = static_cast<const mla::bf16*>(q_pe);
  a.q = static_cast<mla::bf16*>(q);
  a.T = T;
  a.H = q_pe ? H : 0;
  return mla::launch_append(R, Dr, a, static_cast<hipStream_t>(stream)) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

static bool paged_sizes_ok(int N, int Tq, int H, int R, int Dr, int page_size, int max_pages) {
  return N >= 0 && N <= kMaxPagedSeqs && Tq >= 0 && H > 0 && H <= kMaxHeads && page_size >= 1 && max_pages >= 0 &&
         (long long)page_size * max_pages <= INT_MAX - 256 && (long long)Tq * H <= kMaxPagedRows;
}

size_t kda_mla_paged_workspace_bytes(int N, int Tq, int H, int R, int Dr, int page_size, int max_pages,
                                     kda_dtype dt) {
  if (check_type(dt) || !latent_ok(R, Dr) || !paged_sizes_ok(N, Tq, H, R, Dr, page_size, max_pages)) return 0;
  return mla::paged_workspace(N, Tq, H, R, Dr, (long long)page_size * max_pages);
}

kda_status kda_mla_paged_attn(const void* q, const void* cache, const int* block_table, const int* seq_lens,
                              const int* cu_seqlens, void* o, float* lse, int N, int Tq, int H, int R, int Dr,
                              int num_pages, int page_size, int max_pages, float scale, kda_dtype dt,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (const kda_status s = check_type(dt)) return s;
  if (!paged_sizes_ok(N, Tq, H, R, Dr, page_size, max_pages) || num_pages < 0 || !scale_ok(scale) ||
      (long long)num_pages * page_size > INT_MAX || (!cu_seqlens && Tq != N))
    return KDA_ERR_SHAPE;
  if (!latent_ok(R, Dr)) return KDA_ERR_UNSUPPORTED;
  if (N == 0 || Tq == 0) return KDA_OK;
  if (!q || !seq_lens || !o || (num_pages > 0 && !cache) || (max_pages > 0 && !block_table)) return KDA_ERR_NULL;
  if (!aligned16(q, cache, o, lse)) return KDA_ERR_UNSUPPORTED;
  const size_t need = kda_mla_paged_workspace_bytes(N, Tq, H, R, Dr, page_size, max_pages, dt);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return KDA_ERR_WORKSPACE;
  mla::PagedArgs a;
  a.q = static_cast<const mla::bf16*>(q);
  a.cache = static_cast<const mla::bf16*>(cache);
  a.table = block_table;
  a.lens = seq_lens;
  a.cu = cu_seqlens;
  a.o = static_cast<mla::bf16*>(o);
  a.lse = lse;
  a.N = N;
  a.Tq = Tq;
  a.H = H;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.scale = scale;
  a.ws = workspace;
  return mla::launch_paged(R, Dr, a, static_cast<hipStream_t>(stream)) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

kda_status kda_mla_attn_fwd(const void* q, const void* kv, const void* k_pe, void* o, float* lse,
                            const int* cu_seqlens, int num_seqs, int B, int T, int H, int Dn, int Dr, int Dv,
                            float scale, kda_dtype dt, void* stream) {
  if (const kda_status s = check_attn(cu_seqlens, num_seqs, B, T, H, Dn, Dr, Dv, scale, dt)) return s;
  if ((long long)B * T == 0 || num_seqs == 0) return KDA_OK;
  if (!q || !kv || !o || (Dr > 0 && !k_pe)) return KDA_ERR_NULL;
  if (!aligned16(q, kv, k_pe, o, lse)) return KDA_ERR_UNSUPPORTED;
  mla::AttnArgs a = {};
  a.q = static_cast<const mla::bf16*>(q);
  a.kv = static_cast<const mla::bf16*>(kv);
  a.k_pe = static_cast<const mla::bf16*>(k_pe);
  a.o = static_cast<mla::bf16*>(o);
  a.lse = lse;
  a.cu = cu_seqlens;
  a.N = num_seqs;
  a.T = T;
  a.H = H;
  a.scale = scale;
  a.tokens = B * T;
  return mla::launch_attn_fwd(Dn, Dr, a, static_cast<hipStream_t>(stream)) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t kda_mla_attn_bwd_workspace_bytes(int B, int T, int H, int Dn, int Dr, int Dv, int num_seqs, kda_dtype dt) {
  const int cu = 0;  // with or without documents the same
  if (check_attn(B == 1 ? &cu : nullptr, num_seqs, B, T, H, Dn, Dr, Dv, 1.f, dt)) return 0;
  return bwd_layout(B, T, H, Dr).total;
}

kda_status kda_mla_attn_bwd(const void* q, const void* kv, const void* k_pe, const void* o, const float* lse,
                            const void* dout, void* dq, void* dkv, void* dk_pe, const int* cu_seqlens,
                            int num_seqs, int B, int T, int H, int Dn, int Dr, int Dv, float scale, kda_dtype dt,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (const kda_status s = check_attn(cu_seqlens, num_seqs, B, T, H, Dn, Dr, Dv, scale, dt)) return s;
  if ((long long)B * T == 0 || num_seqs == 0) return KDA_OK;
  if (!q || !kv || !o || !lse || !dout || !dq || !dkv || (Dr > 0 && (!k_pe || !dk_pe))) return KDA_ERR_NULL;
  if (!aligned16(q, kv, k_pe, o, lse, dout, dq, dkv, dk_pe)) return KDA_ERR_UNSUPPORTED;
  const BwdLayout L = bwd_layout(B, T, H, Dr);
  if (!workspace || workspace_bytes < L.total || !aligned(workspace, 256)) return KDA_ERR_WORKSPACE;
  mla::AttnArgs a = {};
  a.q = static_cast<const mla::bf16*>(q);
  a.kv = static_cast<const mla::bf16*>(kv);
  a.k_pe = static_cast<const mla::bf16*>(k_pe);
  a.lse = const_cast<float*>(lse);
  a.dout = static_cast<const mla::bf16*>(dout);
  a.dq = static_cast<mla::bf16*>(dq);
  a.dkv = static_cast<mla::bf16*>(dkv);
  a.dk_pe = static_cast<mla::bf16*>(dk_pe);
  a.cu = cu_seqlens;
  a.N = num_seqs;
  a.T = T;
  a.H = H;
  a.scale = scale;
  a.tokens = B * T;
  char* ws = static_cast<char*>(workspace);
  a.delta = reinterpret_cast<float*>(ws);
  a.pe_part = reinterpret_cast<float*>(ws + L.pe_part);
  return mla::launch_attn_bwd(Dn, Dr, a, static_cast<hipStream_t>(stream)) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
