// Host-side launchers of the attention half of a layer (include/mol_attn.h; not exported).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mol {

// Division of a 32-bit number by one that a launch knows, with a multiplication (Granlund and Montgomery,
// "Division by invariant integers using multiplication", 1994): a few instructions where the
// compiler's take two dozen, in kernels whose code has to come from memory first.
struct Divider {
  uint32_t d, mul;
  int s1, s2;
};
inline Divider divider(uint32_t d) {
  int l = 0;
  while (l < 32 && ((uint64_t)1 << l) < d) ++l;
  const uint32_t mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << l) - d)) / d + 1);
  return {d, mul, l < 1 ? l : 1, l < 1 ? 0 : l - 1};
}

struct HeadRows {  // heads of bf16 values: x + token * token_stride + head * head_stride
  const void* x;
  int64_t token_stride, head_stride;
  int heads;
};
struct RopeArgs {
  HeadRows in[3];  // turned into out[0] (q), into the cache (k), copied into the cache (v)
  void* q_out;
  int64_t q_out_token_stride, q_out_head_stride;
  void* k_cache;
  void* v_cache;
  int64_t page_stride, token_stride, head_stride, num_slots;
  int page_size, head_dim;
  const int32_t* slots;
  const int32_t* positions;
  const float* inv_freq;
  int rotary_dim;
  bool interleaved;
  float magnitude;
  int64_t num_tokens;
  // set by launch_rope: a head's 16-byte chunks and its units; heads that a block has a thread a unit for
  int chunks, units, step;
  Divider by_chunks, by_units, by_page;
};
// in[0] into q_out; in[1] and in[2] into their slots. heads 0: not there.
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream);

struct AttnArgs {
  const uint16_t* q;
  int64_t q_token_stride, q_head_stride;
  const uint16_t* k;
  const uint16_t* v;
  int64_t page_stride, token_stride, head_stride;
  int num_pages, page_size, kv_heads, group, head_dim;
  Divider by_page, by_group, by_grid;  // by_grid: the launch's thread blocks
  const int32_t* page_table;
  int64_t table_stride;
  int max_pages;
  const int32_t* kv_lens;
  const int32_t* q_starts;
  int num_seqs, num_tokens;
  float scale_log2;  // scale * log2(e)
  int window;
  uint16_t* out;
  int64_t out_token_stride, out_head_stride;
  void* workspace;
  bool whole;  // blocks of rows are not dealt out in parts (set by the launches)
};
// Scratch of a call of these sizes, and the most that one of up to num_tokens takes.
size_t attn_workspace_bytes(int64_t num_seqs, int64_t num_tokens, int group, int head_dim);
size_t attn_workspace_most(int64_t num_tokens, int group, int head_dim);
cudaError_t prepare_attn_kernels();
cudaError_t take_rope_checks(unsigned long long* first, unsigned long long* count);
cudaError_t take_attn_checks(unsigned long long* first, unsigned long long* count);
cudaError_t take_many_checks(unsigned long long* first, unsigned long long* count);
cudaError_t take_wide_checks(unsigned long long* first, unsigned long long* count);
cudaError_t set_attn_wait_test(unsigned stall, unsigned long long limit_ns);
cudaError_t take_attn_faults(unsigned* out);
cudaError_t launch_attention(const AttnArgs& a, cudaStream_t stream);

}  // namespace mol
