// spec_kv_abi.cu -- the extern "C" entry points of the KV cache: argument checks on the host and
// dispatch to the kernels.
#include <math.h>

#include <initializer_list>

#include "spec_kv.h"
#include "spec_verify.h"

using namespace specv;

namespace specv {
int launch_result(cudaError_t e);   // SPEC_ERR_LAUNCH, recording e for spec_last_cuda_error
}  // namespace specv

namespace {

constexpr long long kMaxNew = 1 << 20;      // new tokens per sequence
constexpr int kMaxHeads = 1024;

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The checks every call makes of the cache and the batch, shape before pointers, and the
// arguments they share. The tensors of an empty batch may be null: torch gives them no address.
int kv_common(KvArgs &a, const spec_kv_cache_t *c, const int32_t *page_table, int pps,
              const int32_t *seq_lens, const int32_t *new_lens, int B, int N,
              const uint32_t *mask_words, int32_t *status) {
  if (!c) return SPEC_ERR_NULL;
  if (B < 0 || N < 1 || N > kMaxNew || pps < 1) return SPEC_ERR_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128) return SPEC_ERR_SHAPE;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return SPEC_ERR_SHAPE;
  if (c->kv_heads < 1 || c->kv_heads > kMaxHeads || c->num_pages < 1) return SPEC_ERR_SHAPE;
  if (static_cast<long long>(c->num_pages) * c->kv_heads * c->page_size >= (1LL << 31))
    return SPEC_ERR_SHAPE;
  if (static_cast<long long>(pps) * c->page_size >= (1LL << 30)) return SPEC_ERR_SHAPE;
  if (mask_words && N > SPEC_MAX_NODES) return SPEC_ERR_SHAPE;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !status ||
      (B > 0 && (!page_table || !seq_lens)))
    return SPEC_ERR_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) ||
      !aligned(c->v_scale, 4) || !aligned(page_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(new_lens, 4) || !aligned(mask_words, 4) || !aligned(status, 4))
    return SPEC_ERR_ALIGN;
  a = KvArgs{};
  a.k = static_cast<uint8_t *>(c->k);
  a.v = static_cast<uint8_t *>(c->v);
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.new_lens = new_lens;
  a.mask = mask_words;
  a.status = status;
  a.num_pages = c->num_pages;
  a.page = c->page_size;
  a.page_shift = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  a.Hkv = c->kv_heads;
  a.D = c->head_dim;
  a.pps = pps;
  a.B = B;
  a.N = N;
  a.W = (N + 31) / 32;
  return SPEC_OK;
}

// a strided [B, N, heads, D] operand: tokens apart by at least their elements
bool stride_ok(int64_t stride, int heads, int D) {
  return stride >= static_cast<int64_t>(heads) * D && stride % 8 == 0 && stride < (1LL << 31);
}

}  // namespace

extern "C" {

int spec_kv_append(const spec_kv_cache_t *cache, const int32_t *page_table, int pages_per_seq,
                   const int32_t *seq_lens, const int32_t *new_lens, int B, int N, const void *k,
                   int64_t k_stride, const void *v, int64_t v_stride, const void *q,
                   int64_t q_stride, int q_heads, void *q_out, int dtype, const float *rope,
                   int rope_rows, int rope_dim, int interleaved, const int32_t *positions,
                   const uint32_t *mask_words, int32_t *status, void *stream) {
  if (dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_DTYPE;
  KvArgs a;
  const int rc = kv_common(a, cache, page_table, pages_per_seq, seq_lens, new_lens, B, N,
                           mask_words, status);
  if (rc != SPEC_OK) return rc;
  if (q_heads < 0 || q_heads > 16 * kMaxHeads) return SPEC_ERR_SHAPE;
  if (!stride_ok(k_stride, a.Hkv, a.D) || !stride_ok(v_stride, a.Hkv, a.D) ||
      (q_heads > 0 && !stride_ok(q_stride, q_heads, a.D)))
    return SPEC_ERR_SHAPE;
  if (rope_dim < 0 || rope_dim > a.D || rope_dim % 16 || (rope_dim > 0 && rope_rows < 1))
    return SPEC_ERR_SHAPE;
  if ((B > 0 && (!k || !v || (q_heads > 0 && (!q || !q_out)))) || (rope_dim > 0 && !rope))
    return SPEC_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(rope, 4) || !aligned(positions, 4) ||
      (q_heads > 0 && (!aligned(q, 16) || !aligned(q_out, 16))))
    return SPEC_ERR_ALIGN;
  // rotating in place needs the output's layout
  if (q_heads > 0 && q && q == q_out && q_stride != static_cast<int64_t>(q_heads) * a.D)
    return SPEC_ERR_SHAPE;
  if (B == 0) return SPEC_OK;
  a.Hq = q_heads;
  RopeArgs r{};
  r.q = q;
  r.k = k;
  r.v = v;
  r.q_stride = q_stride;
  r.k_stride = k_stride;
  r.v_stride = v_stride;
  r.q_out = q_out;
  r.rope = rope;
  r.positions = positions;
  r.rows = rope_rows;
  r.R = rope_dim;
  r.pairs = interleaved != 0;
  r.touched = (N + a.page - 2) / a.page + 1;
  r.vec4 = aligned(rope, 16);
  return launch_result(launch_kv_append(a, r, dtype, static_cast<cudaStream_t>(stream)));
}

size_t spec_kv_attention_workspace_bytes(int B, int N, int q_heads, int kv_heads, int head_dim) {
  if (B < 0 || N < 1 || N > kMaxNew || kv_heads < 1 || kv_heads > kMaxHeads || q_heads < 1 ||
      q_heads % kv_heads || q_heads > 16 * kMaxHeads || (head_dim != 64 && head_dim != 128))
    return 0;
  return kv_attention_workspace(B, N, q_heads, kv_heads, head_dim);
}

int spec_kv_attention(const spec_kv_cache_t *cache, const int32_t *page_table, int pages_per_seq,
                      const int32_t *seq_lens, const int32_t *new_lens, int B, int N, const void *q,
                      int64_t q_stride, int q_heads, int dtype, float scale,
                      const uint32_t *mask_words, void *out, float *lse, int32_t *status,
                      void *workspace, size_t workspace_bytes, void *stream) {
  if (dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_DTYPE;
  KvArgs a;
  const int rc = kv_common(a, cache, page_table, pages_per_seq, seq_lens, new_lens, B, N,
                           mask_words, status);
  if (rc != SPEC_OK) return rc;
  const size_t need = spec_kv_attention_workspace_bytes(B, N, q_heads, a.Hkv, a.D);
  if (need == 0) return SPEC_ERR_SHAPE;
  if (!stride_ok(q_stride, q_heads, a.D) || !isfinite(scale)) return SPEC_ERR_SHAPE;
  // rows, and the 128-token tiles of all sequences, key heads and row tiles, are counted in 31 bits
  const long long limit = 1LL << 31;
  const long long rows = static_cast<long long>(N) * (q_heads / a.Hkv);
  if (rows >= limit) return SPEC_ERR_SHAPE;
  const int height = kv_row_tile(rows);
  long long tiles = (static_cast<long long>(pages_per_seq) * a.page + 127) / 128;   // < 2^23
  for (const long long f : {(rows + height - 1) / height, static_cast<long long>(a.Hkv),
                            static_cast<long long>(B)}) {
    tiles *= f;   // both below 2^31
    if (tiles >= limit) return SPEC_ERR_SHAPE;
  }
  if ((B > 0 && (!q || !out)) || !workspace) return SPEC_ERR_NULL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 16))
    return SPEC_ERR_ALIGN;
  if (workspace_bytes < need) return SPEC_ERR_WORKSPACE;
  if (B == 0) return SPEC_OK;
  a.Hq = q_heads;
  return launch_result(launch_kv_attention(a, q, q_stride, dtype, scale, out, lse, workspace,
                                           static_cast<cudaStream_t>(stream)));
}

int spec_kv_commit(const spec_kv_cache_t *cache, int layers, const int32_t *page_table,
                   int pages_per_seq, const int32_t *seq_lens, int B, int N,
                   const int32_t *path_nodes, const int32_t *accept_len, int32_t *out_lens,
                   int32_t *status, void *stream) {
  KvArgs a;
  const int rc = kv_common(a, cache, page_table, pages_per_seq, seq_lens, nullptr, B, N, nullptr,
                           status);
  if (rc != SPEC_OK) return rc;
  if (layers < 1 || N > SPEC_MAX_NODES) return SPEC_ERR_SHAPE;
  if (B > 0 && (!path_nodes || !accept_len || !out_lens)) return SPEC_ERR_NULL;
  if (!aligned(path_nodes, 4) || !aligned(accept_len, 4) || !aligned(out_lens, 4))
    return SPEC_ERR_ALIGN;
  if (out_lens && out_lens == seq_lens) return SPEC_ERR_SHAPE;
  if (B == 0) return SPEC_OK;
  return launch_result(launch_kv_commit(a, layers, path_nodes, accept_len, out_lens,
                                        static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
