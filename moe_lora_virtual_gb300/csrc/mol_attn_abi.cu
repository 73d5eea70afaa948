// Exported C ABI of the attention half of a layer (include/mol_attn.h).
// Host code only: validation, dispatch to the launchers.

#include <cmath>

#include "mol_attend.h"
#include "mol_attn.h"
#include "mol_internal.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int32_t done(cudaError_t e) { return e == cudaSuccess ? MOL_OK : mol::cuda_fail(e); }

#define MOL_TRY(call)              \
  do {                             \
    const int32_t st_ = (call);    \
    if (st_ != MOL_OK) return st_; \
  } while (0)

// Heads of bf16 rows: 16-byte aligned, no stride below a head's width (one token or head needs none).
int32_t check_heads(const void* p, int64_t token_stride, int64_t head_stride, int64_t tokens,
                    int64_t heads, int64_t width) {
  if (!p || (tokens > 1 && token_stride < width) || (heads > 1 && head_stride < width))
    return MOL_ERR_INVALID_ARG;
  return token_stride % 8 != 0 || head_stride % 8 != 0 || !aligned16(p) ? MOL_ERR_UNSUPPORTED : MOL_OK;
}

int32_t check_rope(const mol_rope_table* r, int32_t head_dim) {
  if (!r->inv_freq || r->rotary_dim < 1 || r->rotary_dim > head_dim || !std::isfinite(r->magnitude) ||
      (r->interleaved != 0 && r->interleaved != 1))
    return MOL_ERR_INVALID_ARG;
  return r->rotary_dim % 16 != 0 ? MOL_ERR_UNSUPPORTED : MOL_OK;
}

int32_t check_tokens(int64_t num_tokens, int32_t num_heads, int32_t head_dim) {
  if (num_tokens < 0 || num_heads < 1 || head_dim < 1) return MOL_ERR_INVALID_ARG;
  return num_tokens >= (int64_t)1 << 31 || head_dim % 8 != 0 || head_dim > MOL_ROPE_MAX_HEAD_DIM ||
                 num_heads > 65536
             ? MOL_ERR_UNSUPPORTED
             : MOL_OK;
}

// A cache of no pages is one that nothing lies in.
int32_t check_cache(const mol_paged_cache* c) {
  if (!c || c->num_pages < 0 || c->page_size < 1 || c->num_heads < 1 || c->head_dim < 1)
    return MOL_ERR_INVALID_ARG;
  if (c->num_pages >= (int64_t)1 << 31 || c->num_pages * c->page_size >= (int64_t)1 << 31)
    return MOL_ERR_UNSUPPORTED;
  if (c->num_pages == 0) return MOL_OK;
  if (!c->k || !c->v || (c->num_pages > 1 && c->page_stride < c->head_dim) ||
      (c->page_size > 1 && c->token_stride < c->head_dim) ||
      (c->num_heads > 1 && c->head_stride < c->head_dim))
    return MOL_ERR_INVALID_ARG;
  return c->page_stride % 8 != 0 || c->token_stride % 8 != 0 || c->head_stride % 8 != 0 ||
                 !aligned16(c->k) || !aligned16(c->v)
             ? MOL_ERR_UNSUPPORTED
             : MOL_OK;
}

void set_rope(mol::RopeArgs& a, const mol_rope_table* r, const int32_t* positions) {
  if (!r) return;
  a.positions = positions;
  a.inv_freq = r->inv_freq;
  a.rotary_dim = r->rotary_dim;
  a.interleaved = r->interleaved != 0;
  a.magnitude = r->magnitude;
}

}  // namespace

extern "C" {

int32_t mol_rope(const void* x, int64_t x_token_stride, int64_t x_head_stride,
                 const int32_t* positions, const mol_rope_table* rope, int64_t num_tokens,
                 int32_t num_heads, int32_t head_dim, void* out, int64_t out_token_stride,
                 int64_t out_head_stride, void* stream) {
  MOL_TRY(check_tokens(num_tokens, num_heads, head_dim));
  if (!rope) return MOL_ERR_INVALID_ARG;
  MOL_TRY(check_rope(rope, head_dim));
  if (num_tokens == 0) return MOL_OK;
  if (!positions) return MOL_ERR_INVALID_ARG;
  MOL_TRY(check_heads(x, x_token_stride, x_head_stride, num_tokens, num_heads, head_dim));
  MOL_TRY(check_heads(out, out_token_stride, out_head_stride, num_tokens, num_heads, head_dim));
  MOL_TRY(mol::ensure_device());
  mol::RopeArgs a = {};
  a.in[0] = {x, x_token_stride, x_head_stride, num_heads};
  a.q_out = out;
  a.q_out_token_stride = out_token_stride;
  a.q_out_head_stride = out_head_stride;
  a.page_size = 1;
  a.head_dim = head_dim;
  a.num_tokens = num_tokens;
  set_rope(a, rope, positions);
  return done(mol::launch_rope(a, static_cast<cudaStream_t>(stream)));
}

int32_t mol_cache_append(const void* k, int64_t k_token_stride, int64_t k_head_stride,
                         const void* v, int64_t v_token_stride, int64_t v_head_stride,
                         const int32_t* slots, const int32_t* positions,
                         const mol_rope_table* rope, int64_t num_tokens,
                         const mol_paged_cache* cache, const void* q, int64_t q_token_stride,
                         int64_t q_head_stride, int32_t num_q_heads, void* q_out,
                         int64_t q_out_token_stride, int64_t q_out_head_stride, void* stream) {
  MOL_TRY(check_cache(cache));
  MOL_TRY(check_tokens(num_tokens, cache->num_heads, cache->head_dim));
  if (rope) MOL_TRY(check_rope(rope, cache->head_dim));
  if ((q == nullptr) != (q_out == nullptr) || (q && !rope)) return MOL_ERR_INVALID_ARG;
  if (num_tokens == 0) return MOL_OK;
  if (!slots || (rope && !positions)) return MOL_ERR_INVALID_ARG;
  MOL_TRY(check_heads(k, k_token_stride, k_head_stride, num_tokens, cache->num_heads, cache->head_dim));
  MOL_TRY(check_heads(v, v_token_stride, v_head_stride, num_tokens, cache->num_heads, cache->head_dim));
  mol::RopeArgs a = {};
  if (q) {
    MOL_TRY(check_tokens(num_tokens, num_q_heads, cache->head_dim));
    MOL_TRY(check_heads(q, q_token_stride, q_head_stride, num_tokens, num_q_heads, cache->head_dim));
    MOL_TRY(check_heads(q_out, q_out_token_stride, q_out_head_stride, num_tokens, num_q_heads,
                        cache->head_dim));
    a.in[0] = {q, q_token_stride, q_head_stride, num_q_heads};
    a.q_out = q_out;
    a.q_out_token_stride = q_out_token_stride;
    a.q_out_head_stride = q_out_head_stride;
  }
  MOL_TRY(mol::ensure_device());
  a.in[1] = {k, k_token_stride, k_head_stride, cache->num_heads};
  a.in[2] = {v, v_token_stride, v_head_stride, cache->num_heads};
  a.k_cache = cache->k;
  a.v_cache = cache->v;
  a.page_stride = cache->page_stride;
  a.token_stride = cache->token_stride;
  a.head_stride = cache->head_stride;
  a.num_slots = cache->num_pages * cache->page_size;
  a.page_size = cache->page_size;
  a.head_dim = cache->head_dim;
  a.slots = slots;
  a.num_tokens = num_tokens;
  set_rope(a, rope, positions);
  return done(mol::launch_rope(a, static_cast<cudaStream_t>(stream)));
}

size_t mol_paged_attention_workspace_bytes(int64_t num_seqs, int64_t num_tokens,
                                           int32_t num_q_heads, int32_t num_kv_heads,
                                           int32_t head_dim) {
  if (num_seqs <= 0 || num_tokens <= 0 || num_kv_heads < 1 || num_q_heads < num_kv_heads ||
      num_q_heads % num_kv_heads != 0 || num_q_heads / num_kv_heads > MOL_ATTN_MAX_GROUP ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return 0;
  return mol::attn_workspace_most(num_tokens, num_q_heads / num_kv_heads, head_dim);
}

int32_t mol_paged_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                            const mol_paged_cache* cache, const int32_t* page_table,
                            int64_t table_stride, int32_t max_pages, const int32_t* kv_lens,
                            const int32_t* q_starts, int64_t num_seqs, int64_t num_tokens,
                            int32_t num_q_heads, float scale, int32_t window, void* out,
                            int64_t out_token_stride, int64_t out_head_stride, void* workspace,
                            size_t workspace_bytes, void* stream) {
  MOL_TRY(check_cache(cache));
  const float scale_log2 = scale * 1.4426950408889634f;
  if (num_seqs < 0 || num_tokens < 0 || num_q_heads < 1 || max_pages < 0 || window < 0 ||
      !(scale > 0.f) || !std::isfinite(scale_log2) || (!q_starts && num_tokens != num_seqs) ||
      num_q_heads % cache->num_heads != 0 || (num_seqs > 1 && table_stride < max_pages))
    return MOL_ERR_INVALID_ARG;
  const int d = cache->head_dim;
  if ((d != 64 && d != 128 && d != 256) || num_q_heads / cache->num_heads > MOL_ATTN_MAX_GROUP ||
      num_q_heads > 65536 || num_seqs >= (int64_t)1 << 24 || num_tokens >= (int64_t)1 << 31 ||
      num_tokens * num_q_heads >= (int64_t)1 << 31)
    return MOL_ERR_UNSUPPORTED;
  // positions, a window before the first and a tile behind the last are 32-bit numbers
  const int64_t cached = (int64_t)max_pages * cache->page_size;
  if (num_tokens + cached > ((int64_t)1 << 31) - 1024) return MOL_ERR_UNSUPPORTED;
  // the rows of a key head, with a block's more, and the tiles of a head are counted in 32 bits
  const int64_t rows = num_tokens * (num_q_heads / cache->num_heads);
  if (rows > ((int64_t)1 << 31) - 1024) return MOL_ERR_UNSUPPORTED;
  if ((rows / 16 + num_seqs) * (cached / 64 + 4) >= (int64_t)1 << 31)
    return MOL_ERR_UNSUPPORTED;
  if (num_seqs == 0 || num_tokens == 0) return MOL_OK;
  if (!kv_lens || (max_pages > 0 && !page_table)) return MOL_ERR_INVALID_ARG;
  MOL_TRY(check_heads(q, q_token_stride, q_head_stride, num_tokens, num_q_heads, d));
  MOL_TRY(check_heads(out, out_token_stride, out_head_stride, num_tokens, num_q_heads, d));
  const int group = num_q_heads / cache->num_heads;
  if (!workspace || workspace_bytes < mol::attn_workspace_bytes(num_seqs, num_tokens, group, d))
    return MOL_ERR_CAPACITY;
  if (!aligned16(workspace)) return MOL_ERR_UNSUPPORTED;
  MOL_TRY(mol::ensure_attn_device());
  mol::AttnArgs a = {};
  a.q = static_cast<const uint16_t*>(q);
  a.q_token_stride = q_token_stride;
  a.q_head_stride = q_head_stride;
  a.k = static_cast<const uint16_t*>(cache->k);
  a.v = static_cast<const uint16_t*>(cache->v);
  a.page_stride = cache->page_stride;
  a.token_stride = cache->token_stride;
  a.head_stride = cache->head_stride;
  a.num_pages = (int)cache->num_pages;
  a.page_size = cache->page_size;
  a.kv_heads = cache->num_heads;
  a.group = group;
  a.head_dim = d;
  a.by_page = mol::divider((uint32_t)cache->page_size);
  a.by_group = mol::divider((uint32_t)group);
  a.page_table = page_table;
  a.table_stride = table_stride;
  a.max_pages = max_pages;
  a.kv_lens = kv_lens;
  a.q_starts = q_starts;
  a.num_seqs = (int)num_seqs;
  a.num_tokens = (int)num_tokens;
  a.scale_log2 = scale_log2;
  a.window = window < cached ? window : 0;  // (0: all)
  a.out = static_cast<uint16_t*>(out);
  a.out_token_stride = out_token_stride;
  a.out_head_stride = out_head_stride;
  a.workspace = workspace;
  return done(mol::launch_attention(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
