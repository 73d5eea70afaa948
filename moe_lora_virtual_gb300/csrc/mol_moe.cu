// Host side of the experts and the 4-bit linear: the geometry of a launch (mol_moe.cuh has the
// kernel).

#include <algorithm>
#include <cmath>

#include "mol_block.h"
#include "mol_device.cuh"
#include "mol_internal.h"
#include "mol_moe.h"

namespace mol {
namespace {

int g_sm_count = 0;
int g_clusters[kClusterSizes] = {};  // clusters of 1 << i blocks that the device holds at once

constexpr int align_up(int v, int m) { return (v + m - 1) / m * m; }

cudaError_t launch_by_group(int group, const StreamArgs& a, int mode, int grid, size_t smem,
                            cudaStream_t stream) {
  switch (group) {
    case 0: return stream_launch<0>(a, mode, grid, smem, stream);
    case 32: return stream_launch<32>(a, mode, grid, smem, stream);
    case 64: return stream_launch<64>(a, mode, grid, smem, stream);
    default: return stream_launch<128>(a, mode, grid, smem, stream);
  }
}

// Tokens of an entry, a power of two: half as many again as the mean of an expert's pairs, so that few
// experts need a second entry (which reads their weights again), and no more room than the tokens
// need. From 8 on, where twice as many cost a second token tile, a tenth more than the mean suffices.
// Layers of 2048 x 768 at 8 and at 16 tokens an entry, us: 128 experts, top 8, 4 bits (32): 96 tokens
// 92 and 122, 127 tokens 113 and 126 (there 8 would be better); 4 bits (128): 110 tokens 93 and 104,
// 127 tokens 103 and 105; bf16: 64 tokens 192 and 201, 110 tokens 205 and 199, 127 tokens 252 and 200.
// Never more than 16: with the sums of 32 or 64 tokens in registers 8 experts, 128 tokens, top 2, took
// 39.5 and 61 us in bf16 where 16 take 39.4 (8: 55), in 4 bits 42 and 87 where 16 take 29 (8: 32). Their
// later entries find the weights in L2. They do not where the experts' weights are more than L2 holds,
// as an expert's entries are dealt to different blocks: 64 bf16 experts, 128 tokens, top 8: 143 us in
// entries of 64, 157 of 16, 146 of 8.
int entry_tokens(int num_tokens, int pairs, int experts) {
  int n = num_tokens == 1 ? 1 : num_tokens == 2 ? 2 : 4;
  while (n < 16 && n < num_tokens &&
         (n < 8 ? 2 * n * experts < 3 * pairs : 10 * n * experts < 11 * pairs))
    n *= 2;
  return n;
}

int token_tiles(int xrows) { return xrows <= 8 ? 1 : xrows <= 16 ? 2 : 4; }

constexpr int kLeastStage = 2304;  // down: stages are no smaller

// Rows of Kc inputs in a stage: as they lie in memory (one copy), or pieces of them (a copy each).
void row_layout(StreamArgs& a, int group, int rows, int Kc) {
  const int bytes = group ? align_up(Kc, 256) / 2 : Kc * 2;  // of a row
  const int scale_bytes = group ? align_up(Kc, 256) / group * 2 : 0;
  a.Kc = Kc;
  a.ksteps = (a.K + Kc - 1) / Kc;
  a.row_copies = a.ksteps > 1;
  a.row_pitch = a.row_copies ? align_up(bytes, 128) + 64 : bytes;
  a.span_shift = a.row_copies ? 0 : 64;  // (the pieces' pitch has the shift)
  a.scale_pitch = !group ? 0 : a.row_copies ? align_up(scale_bytes, 16) + 16 : scale_bytes;
  a.scale_off = align_up(rows * a.row_pitch + (rows + 7) / 8 * a.span_shift, 16);
  a.x_pitch = align_up(Kc * 2, 128) + 64;
}

// Bytes of gate_up's and the linear's rings, token slots and sums.
int stream_smem(const StreamArgs& a, int group) {
  const int nt = token_tiles(a.xrows);
  return consumer_warps(nt) * a.chunks * chunk_bytes(group) + a.xstages * a.xslot_bytes +
         a.teams * (a.parts - 1) * nt * 512;
}

// gate_up, linear: the token slots and the teams of a block that has `room` bytes, when the blocks
// share `entries` entries. False when nothing fits.
// Slots: whole rows where they fit, if need be beside rings of two chunks (16 tokens of 4096 inputs and
// 20000 rows 17.8 us; pieces beside rings of four, which read the tokens again for each group of tiles,
// 27.0).
// Teams: the warps of a team split the inputs of a tile, so more parts fill all warps where a block has
// few tiles, and leave less to wait for at the end; against that each tile costs its warps half a
// chunk's time, or two for each token tile where their sums are to be added, and two more with 4-bit
// weights, whose warps then wait for one another's products. Taken is the least of that model, with
// one more tile a warp for the end: measured, an output head of 49 tiles a block takes 30.1 us with
// one part and 37.7 with four, a linear of up to one tile a block (2048 inputs, 2432 rows) 5.8 us with
// one, 3.9 with four, and 4.5 with the 16 that the model takes there: among equals it takes the most,
// also more than a row has chunks.
bool plan(StreamArgs& a, int group, int mode, int room, int entries, int grid) {
  const int inputs = group ? 256 : 64, nt = token_tiles(a.xrows);
  a.tile_rows = mode == kGateUp ? 8 : 16;
  const int64_t tiles = (int64_t)entries * ((a.N + a.tile_rows - 1) / a.tile_rows);
  const double block_tiles = (double)tiles / grid;
  StreamArgs best = {};
  double least = 0;
  for (int parts = 1; parts <= consumer_warps(nt); ++parts) {
    a.parts = parts;
    a.teams = consumer_warps(nt) / parts;
    auto slots = [&](int Kc, int n, int chunks) {
      a.Kc = Kc;
      a.ksteps = (a.K + Kc - 1) / Kc;
      a.x_pitch = align_up(Kc * 2, 128) + 64;
      a.xslot_bytes = align_up(a.xrows * a.x_pitch, 128);
      a.xstages = n;
      a.chunks = chunks;
      return stream_smem(a, group) <= room;
    };
    // a second token slot lets the next expert's tokens come while the last one's weights are consumed
    bool fits = (entries > 1 && slots(a.K, 2, kChunks)) || slots(a.K, 1, kChunks);
    fits = fits || slots(a.K, 1, 2);
    for (int Kc = 2048; Kc >= 256 && !fits; Kc -= 256) fits = Kc < a.K && slots(Kc, 2, kChunks);
    fits = fits || slots(std::min(256, a.K), 1, kChunks);
    if (!fits) continue;
    const int per = (std::min(a.Kc, a.K) + inputs - 1) / inputs;
    const double one = a.ksteps * ((per + parts - 1) / parts) + (parts > 1 ? 2 * nt + (group ? 2 : 0) : 0.5);
    const double rounds = block_tiles / a.teams;
    const double cost = (std::max(1.0, (rounds + 2 * std::ceil(rounds)) / 3) + 1) * one;
    if (best.parts && cost > least) continue;
    least = cost;
    best = a;
  }
  if (!best.parts) return false;
  a = best;
  a.entry_rows = align_up(a.N, a.tile_rows * (a.ksteps > 1 ? a.teams : 1));
  return true;
}

// down: the stage and the teams of a block of `rows` output rows, with `fixed` bytes of lists and
// sums besides each team's `copy` of them. False when the stages that fit are fewer than `least`.
bool plan_down(StreamArgs& a, int group, int rows, int Kc, int fixed, int copy, int least) {
  a.parts = (rows + 15) / 16;
  row_layout(a, group, rows, Kc);
  a.x_off = align_up(a.scale_off + rows * a.scale_pitch + (group ? 16 * ((rows + 7) / 8) + 16 : 0), 128);
  a.stage_bytes = std::max(kLeastStage, a.x_off + align_up(a.xrows * a.x_pitch, 128));
  // as many teams as have a stage each, beside their sums
  for (a.teams = kBlockWarps / a.parts; a.teams >= 1; --a.teams) {
    a.stages = std::min(kMaxStages, (kSmem - fixed - a.teams * copy) / a.stage_bytes);
    if (a.stages >= a.teams) break;
  }
  a.stages = a.teams ? a.stages / a.teams * a.teams : 0;
  return a.stages >= least;
}

StreamArgs common_args(const MoeShape& s, const void* x, int64_t x_stride, const int32_t* ids,
                       const WeightRows& w, const void* delta, int64_t delta_stride, void* out,
                       int64_t out_stride) {
  StreamArgs a = {};
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.ids = ids;
  a.w = static_cast<const char*>(w.data);
  a.scales = static_cast<const __nv_bfloat16*>(w.scales);
  a.delta = static_cast<const __nv_bfloat16*>(delta);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.x_stride = x_stride;
  a.delta_stride = delta_stride;
  a.out_stride = out_stride;
  a.num_tokens = s.num_tokens;
  a.topk = s.topk;
  a.E = s.num_experts;
  a.K = w.K;
  a.cluster = 1;
  a.xrows = entry_tokens(s.num_tokens, s.num_tokens * s.topk, s.num_experts);
  return a;
}

// What grouping the pairs takes in shared memory besides the lists (build_lists: the ids, and each
// warp's counts of each expert).
int scratch_bytes(const MoeShape& s) {
  const int numel = s.num_tokens * s.topk;
  if (numel <= 32) return 0;
  const int rounds = (numel + kListThreads - 1) / kListThreads;
  const int warps = (numel + rounds * 32 - 1) / (rounds * 32);
  return 4 * numel + align_up(2 * warps * s.num_experts, 4);
}

int list_bytes(const MoeShape& s) { return s.num_tokens * s.topk * 16; }

constexpr int kCombineThreads = 128;

// The split form's second step, out[t] = sum over t's pairs of weight * partial, in the order of the
// slots, plus the same sum of the deltas. Four columns a thread; bound by the round trip of the fp32
// partials to L2, so the loads of eight slots are in flight at once (an absent pair's rows are read and
// not used), and the first slots' ids and weights, which the kernels before did not write, are loaded
// before those have ended.
__global__ void __launch_bounds__(kCombineThreads) moe_combine_kernel(const StreamArgs a) {
  const int t = blockIdx.y, n = (blockIdx.x * kCombineThreads + threadIdx.x) * 4;
  constexpr int U = 8;
  float w[U];
  bool has[U];
  auto slots = [&](int k0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t pair = t * a.topk + min(k0 + u, a.topk - 1);
      const int e = ld_cg_i32(a.ids + pair);  // (from L2: no stale L1 line)
      has[u] = k0 + u < a.topk && e >= 0 && e < a.E;
      w[u] = __ldcg(a.weights + pair);
    }
  };
  slots(0);
  pdl_wait();
  pdl_launch_dependents();
  if (n >= a.N) return;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f), deltas = sum;
  auto add = [](float4& s, float w, float v0, float v1, float v2, float v3) {
    s.x = fmaf(w, v0, s.x);
    s.y = fmaf(w, v1, s.y);
    s.z = fmaf(w, v2, s.z);
    s.w = fmaf(w, v3, s.w);
  };
  for (int k0 = 0; k0 < a.topk; k0 += U) {
    if (k0 > 0) slots(k0);
    float4 v[U];
    uint2 d[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t pair = t * a.topk + min(k0 + u, a.topk - 1);
      v[u] = *reinterpret_cast<const float4*>(a.partial + pair * a.N + n);
      d[u] = a.delta ? *reinterpret_cast<const uint2*>(a.delta + pair * a.delta_stride + n)
                     : make_uint2(0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!has[u]) continue;
      add(sum, w[u], v[u].x, v[u].y, v[u].z, v[u].w);
      if (a.delta)
        add(deltas, w[u], bf16_lo(d[u].x), bf16_hi(d[u].x), bf16_lo(d[u].y), bf16_hi(d[u].y));
    }
  }
  const uint2 o = make_uint2(pack_bf16x2(sum.x + deltas.x, sum.y + deltas.y),
                             pack_bf16x2(sum.z + deltas.z, sum.w + deltas.w));
  *reinterpret_cast<uint2*>(a.out + t * a.out_stride + n) = o;
}

}  // namespace

// The split form reads each activation row once and shares all weights evenly, for a second kernel
// and the partials' way through L2. It pays for 4-bit weights from a few pairs on, as theirs is the
// work of the warps (128 experts of 2048 x 768, top 8, layer, group 128: 32 pairs 28.4 us against 27.0,
// 64 pairs 41.0 against 46.1, 768 pairs 86 against 111), for bf16 where experts have many tokens (496
// pairs 191 us against 190, 768 pairs 197 against 201, 1016 pairs 200 against 242) or the down rows are
// short and their stages small (102 pairs of 103 experts of 2520 x 72: 26.6 us against 33.1; of 232 x
// 232, which are taken in one kernel, 13.6 against 15.5).
size_t moe_split_bytes(const MoeShape& s, int group) {
  const int pairs = s.num_tokens * s.topk;
  if (pairs <= 32) return 0;
  const bool short_rows = s.inter <= 192 && s.hidden >= 256;
  if (group == 0 && !short_rows && pairs < 6 * s.num_experts) return 0;
  return (size_t)pairs * s.hidden * sizeof(float);
}

cudaError_t launch_moe_down_split(const MoeShape& s, const void* act, const int32_t* topk_ids,
                                  const float* topk_weights, const WeightRows& w, const void* delta,
                                  int64_t delta_stride, void* workspace, void* out,
                                  int64_t out_stride, bool chained, cudaStream_t stream) {
  StreamArgs a = common_args(s, act, s.inter, topk_ids, w, delta, delta_stride, out, out_stride);
  a.weights = topk_weights;
  a.partial = static_cast<float*>(workspace);
  a.N = s.hidden;
  a.chained = chained;
  const int entries = std::min(s.num_tokens * s.topk, s.num_experts);
  if (!plan(a, w.group, kPairs, kSmem - list_bytes(s), entries, g_sm_count))
    return cudaErrorInvalidConfiguration;
  const size_t smem = stream_smem(a, w.group) + list_bytes(s);
  const cudaError_t e = launch_by_group(w.group, a, kPairs, g_sm_count, smem, stream);
  if (e != cudaSuccess) return e;
  const int columns = kCombineThreads * 4;
  return launch_pdl(moe_combine_kernel, dim3((s.hidden + columns - 1) / columns, s.num_tokens),
                    dim3(kCombineThreads), 0, stream, a);
}

cudaError_t launch_moe_gate_up(const MoeShape& s, const void* x, int64_t x_stride,
                               const int32_t* topk_ids, const WeightRows& w, const void* delta,
                               int64_t delta_stride, void* act, cudaStream_t stream) {
  StreamArgs a = common_args(s, x, x_stride, topk_ids, w, delta, delta_stride, act, s.inter);
  a.N = s.inter;
  const int entries = std::min(s.num_tokens * s.topk, s.num_experts);
  if (!plan(a, w.group, kGateUp, kSmem - list_bytes(s), entries, g_sm_count))
    return cudaErrorInvalidConfiguration;
  const size_t smem = stream_smem(a, w.group) + list_bytes(s);
  return launch_by_group(w.group, a, kGateUp, g_sm_count, smem, stream);
}

cudaError_t launch_moe_down(const MoeShape& s, const void* act, const int32_t* topk_ids,
                            const float* topk_weights, const WeightRows& w, const void* delta,
                            int64_t delta_stride, void* out, int64_t out_stride, bool chained,
                            cudaStream_t stream) {
  StreamArgs a = common_args(s, act, s.inter, topk_ids, w, delta, delta_stride, out, out_stride);
  a.weights = topk_weights;
  a.N = s.hidden;
  a.chained = chained;
  // Blocks alone or clusters that split the experts: the fewer rows a block has, the more often each
  // activation row is read. Taken is what brings the fewest bytes into one block, a cluster's
  // exchange counted as the 64 KB that arrive meanwhile, among those whose stages hold whole rows.
  // Many rows take several waves of blocks.
  const int pairs = s.num_tokens * s.topk, units = std::min(pairs, s.num_experts);
  const int64_t x_bytes = (int64_t)s.inter * 2 * ((pairs + units - 1) / units);
  const int64_t row_bytes = w.group ? w4_padded(s.inter) / 2 : s.inter * 2;
  StreamArgs best = {};
  int64_t least = INT64_MAX;
  int grid = 0;
  size_t smem = 0;
  auto consider = [&](int cluster, int blocks, int waves, int Kc, int stages) {
    const int rows = (s.hidden + blocks - 1) / blocks;
    a.cluster = cluster;
    a.acc_stride = align_up(rows, 4) + 4;
    const int copy = s.num_tokens * a.acc_stride * 4;
    const int fixed =
        list_bytes(s) + (cluster > 1 ? align_up(s.num_tokens, cluster) * a.acc_stride * 4 : 0);
    if (fixed + copy > kSmem / 2 || !plan_down(a, w.group, rows, Kc, fixed, copy, stages)) return;
    // the lists' scratch lies where the ring and, behind it, the teams' sums will be
    if (a.stages * a.stage_bytes + a.teams * copy < scratch_bytes(s)) return;
    const int64_t bytes =
        waves * ((units + cluster - 1) / cluster) * (rows * row_bytes + x_bytes) +
        (cluster > 1 ? 65536 : 0);
    if (bytes >= least) return;
    least = bytes;
    best = a;
    grid = blocks * cluster;
    smem = (size_t)a.stages * a.stage_bytes + a.teams * copy + fixed;
  };
  for (int i = 0; i < kClusterSizes; ++i) {
    const int at_once = g_clusters[i];
    if (at_once < 1) continue;
    const int waves = (s.hidden + at_once * kDownRows - 1) / (at_once * kDownRows);
    consider(1 << i, std::min(at_once * waves, (s.hidden + 7) / 8), waves, s.inter, 3);
  }
  // else pieces of rows, or fewer rows a block
  for (int blocks = g_clusters[0]; grid == 0; blocks *= 2) {
    const int n = std::min(blocks, s.hidden), rows = (s.hidden + n - 1) / n;
    if (rows <= kDownRows) {
      for (int Kc = 2048; Kc > 256 && grid == 0; Kc -= 256)
        if (Kc < s.inter) consider(1, n, 1, Kc, 3);
      if (grid == 0) consider(1, n, 1, std::min(256, s.inter), 2);
    }
    if (n == s.hidden) break;
  }
  if (grid == 0) return cudaErrorInvalidConfiguration;
  return launch_by_group(w.group, best, kDown, grid, smem, stream);
}

cudaError_t launch_w4_linear(const void* x, int64_t x_stride, int num_tokens, int N,
                             const WeightRows& w, void* out, int64_t out_stride,
                             cudaStream_t stream) {
  const MoeShape s{num_tokens, 1, 1, N, w.K};
  StreamArgs a = common_args(s, x, x_stride, nullptr, w, nullptr, 0, out, out_stride);
  a.N = N;
  // More tokens than 16 are entries of 16, which read the weights again, mostly from L2; up to 32 with
  // many rows one entry (32 tokens, 2048 inputs, 100001 rows: 50 us in one, 57 in two; 2000 rows: 10.1
  // and 7.2). Entries of 8 where 8 whole rows of tokens fit and 16 do not (24 tokens of 8192 inputs:
  // 20000 rows 53 us against 61 in pieces, 5000 rows 20 against 33; against it, 48 tokens, 20000 rows:
  // 107 against 85), none smaller (64 tokens of 16384 inputs, 20000 rows: 514 us in entries of 4, 267
  // in pieces of 16).
  const int tiles = (N + 15) / 16;
  int grid = 0;
  auto fits = [&](int rows) {
    a.xrows = rows;
    const int entries = (num_tokens + rows - 1) / rows;
    grid = (int)std::min<int64_t>((int64_t)tiles * entries, g_sm_count);
    return plan(a, w.group, kLinear, kSmem, entries, grid);
  };
  const int most = num_tokens <= 32 && tiles >= 4 * g_sm_count ? 32 : 16;
  bool ok = fits(std::min(num_tokens, most));
  if (ok && a.ksteps > 1) {
    for (int rows = most; rows >= 8 && a.ksteps > 1; rows /= 2)
      if (rows < num_tokens) ok = fits(rows);
    if (!ok || a.ksteps > 1) ok = fits(std::min(num_tokens, most));
  }
  if (!ok) return cudaErrorInvalidConfiguration;
  if ((int64_t)tiles * 16 * ((num_tokens + a.xrows - 1) / a.xrows) > 1 << 30) {
    // (the kernel counts the entries' rows in 32 bits: an entry a launch)
    const int rows = a.xrows;
    for (int t = 0; t < num_tokens; t += rows) {
      const cudaError_t e = launch_w4_linear(
          static_cast<const __nv_bfloat16*>(x) + t * x_stride, x_stride,
          std::min(rows, num_tokens - t), N, w, static_cast<__nv_bfloat16*>(out) + t * out_stride,
          out_stride, stream);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
  return launch_by_group(w.group, a, kLinear, grid, stream_smem(a, w.group), stream);
}

cudaError_t prepare_moe_kernels() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&g_sm_count, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = stream_prepare<0>(g_clusters);
  if (e == cudaSuccess) e = stream_prepare<32>(nullptr);
  if (e == cudaSuccess) e = stream_prepare<64>(nullptr);
  if (e == cudaSuccess) e = stream_prepare<128>(nullptr);
  if (e == cudaSuccess && g_clusters[0] < 1) e = cudaErrorInvalidConfiguration;
  return e;
}

cudaError_t take_moe_faults(unsigned* out) {
  *out = 0;
  for (auto take : {stream_take_faults<0>, stream_take_faults<32>, stream_take_faults<64>,
                    stream_take_faults<128>}) {
    unsigned f = 0;
    const cudaError_t e = take(&f);
    if (e != cudaSuccess) return e;
    *out |= f;
  }
  return cudaSuccess;
}

cudaError_t set_moe_wait_test(unsigned stall, unsigned long long limit_ns) {
  for (auto set : {stream_wait_test<0>, stream_wait_test<32>, stream_wait_test<64>,
                   stream_wait_test<128>}) {
    const cudaError_t e = set(stall, limit_ns);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t take_moe_checks(unsigned long long* first, unsigned long long* count) {
  *first = *count = 0;
  for (auto take : {stream_take_checks<0>, stream_take_checks<32>, stream_take_checks<64>,
                    stream_take_checks<128>}) {
    unsigned long long f = 0, n = 0;
    const cudaError_t e = take(&f, &n);
    if (e != cudaSuccess) return e;
    if (*first == 0) *first = f;
    *count += n;
  }
  return cudaSuccess;
}

}  // namespace mol
