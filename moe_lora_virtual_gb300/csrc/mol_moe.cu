// Host side of the experts and the 4-bit linear: the geometry of a launch (mol_moe.cuh has the
// kernel).

#include <algorithm>

#include "mol_block.h"
#include "mol_internal.h"
#include "mol_moe.h"

namespace mol {
namespace {

int g_sm_count = 0;
int g_clusters = 0;  // clusters of kCluster large blocks that fit the device

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

// Tokens of an entry, a power of two: twice the mean of an expert's pairs, so that few experts need
// a second entry (which reads their weights again), and no more room than the tokens need.
int entry_tokens(int num_tokens, int pairs, int experts) {
  int n = num_tokens == 1 ? 1 : num_tokens == 2 ? 2 : 4;
  while (n < 64 && n < num_tokens && n * experts < 2 * pairs) n *= 2;
  return n;
}

// A team's partial sums cost 512 bytes a stage for each further warp and tile of 8 tokens.
int parts_most(int xrows) { return xrows <= 16 ? 4 : 2; }
int token_tiles(int xrows) { return xrows <= 8 ? 1 : xrows <= 16 ? 2 : xrows <= 32 ? 4 : 8; }

// Chooses the stage and the rings for a block that has `room` bytes for them. xstages_most: token
// slots of use when they hold whole rows. False when nothing fits.
bool plan(StreamArgs& a, int group, int mode, int room, int xstages_most) {
  auto stage = [&](int rows, int Kc, int xstages) {
    const int bytes = group ? align_up(Kc, 256) / 2 : Kc * 2;  // of a row
    const int scale_bytes = group ? align_up(Kc, 256) / group * 2 : 0;
    a.Kc = Kc;
    a.ksteps = (a.K + Kc - 1) / Kc;
    a.stage_rows = rows;
    a.half_rows = rows / 2;
    a.tile_rows = mode == kGateUp ? rows / 2 : rows;
    // rows of 4 KB and more by a copy each (shorter copies are slower): padding keeps the lanes'
    // reads off the same banks
    a.row_copies = a.ksteps > 1 || bytes >= 4096;
    a.row_pitch = a.row_copies ? align_up(bytes, 128) + 64 : bytes;
    a.scale_pitch = !group ? 0 : a.row_copies ? align_up(scale_bytes, 16) + 16 : scale_bytes;
    a.scale_off = align_up(rows * a.row_pitch, 16);
    a.parts_off = align_up(a.scale_off + rows * a.scale_pitch + (group ? 32 : 0), 128);
    a.stage_bytes = a.parts_off + (parts_most(a.xrows) - 1) * 512 * token_tiles(a.xrows);
    a.x_pitch = align_up(Kc * 2, 128) + 64;
    a.xslot_bytes = align_up(a.xrows * a.x_pitch, 128);
    a.xstages = xstages;
    a.stages = std::min(kMaxStages, (room - xstages * a.xslot_bytes) / a.stage_bytes);
    return a.stages;
  };
  // Whole rows. 16 rows a tile use the tensor instruction's M side fully; tiles of 8 leave room for
  // more stages where rows are long. A second token slot lets the producer go on to the next
  // expert while the last one's stages are consumed.
  for (int x = xstages_most; x >= 1; --x) {
    if (stage(16, a.K, x) >= (x > 2 ? 12 : 6)) return true;
    if (stage(8, a.K, x) >= (x > 2 ? 12 : 4)) return true;
  }
  if (stage(8, a.K, 1) >= 3) return true;
  // pieces of rows, the longest that leave four stages
  for (int Kc = 2048; Kc > 256; Kc -= 256)
    if (Kc < a.K && stage(group || Kc <= 1024 ? 16 : 8, Kc, 2) >= 4) return true;
  return stage(8, std::min(256, a.K), 2) >= 2;
}

void fit_parts(StreamArgs& a) {
  a.parts = 1;
  while (2 * a.parts <= parts_most(a.xrows) && 2 * a.parts * a.teams <= a.consumers) a.parts *= 2;
}

// As many teams as there are stages, or fewer that share them evenly without leaving more unused.
void fit_teams(StreamArgs& a) {
  const int most = std::min(a.consumers, a.stages);
  a.teams = most;
  for (int w = most; w > most / 2; --w)
    if (a.stages / w * w > a.stages / a.teams * a.teams) a.teams = w;
  a.stages = a.stages / a.teams * a.teams;
  fit_parts(a);
  a.entry_rows = align_up(a.N, a.tile_rows * (a.ksteps > 1 ? a.teams : 1));
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

size_t list_bytes(const MoeShape& s) { return (size_t)s.num_tokens * s.topk * 16; }

// A step of a token or two: blocks of half an SM's shared memory and registers, so that the down
// kernel's blocks are resident, and their first weights on the way, while the gate_up kernel
// streams. Elsewhere the ring takes the whole SM.
bool small_step(const MoeShape& s) { return s.num_tokens * s.topk <= 16; }

}  // namespace

cudaError_t launch_moe_gate_up(const MoeShape& s, const void* x, int64_t x_stride,
                               const int32_t* topk_ids, const WeightRows& w, const void* delta,
                               int64_t delta_stride, void* act, cudaStream_t stream) {
  StreamArgs a = common_args(s, x, x_stride, topk_ids, w, delta, delta_stride, act, s.inter);
  a.N = s.inter;
  for (bool small = small_step(s);; small = false) {
    const int room = (small ? kSmemSmall : kSmemLarge) - (int)list_bytes(s);
    a.consumers = small ? kFewConsumers : kMostConsumers;
    if (plan(a, w.group, kGateUp, room, 2)) break;
    if (!small) return cudaErrorInvalidConfiguration;
  }
  fit_teams(a);
  const size_t smem = (size_t)a.stages * a.stage_bytes + a.xstages * a.xslot_bytes + list_bytes(s);
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
  // Rows over clusters (whose blocks read each activation row once instead of four times), or over
  // blocks when there are too few pairs to split. A block has at most `most` rows, so many rows
  // take several waves of blocks.
  const bool split = s.num_tokens * s.topk >= 2 * kCluster;
  a.cluster = split ? kCluster : 1;
  const int at_once = split ? g_clusters : g_sm_count;
  for (bool small = small_step(s);; small = false) {
    const int budget = (small ? kSmemSmall : kSmemLarge) - (int)list_bytes(s);
    a.consumers = small ? kFewConsumers : kMostConsumers;
    for (int most = 128; most >= 8; most /= 2) {
      const int waves = (s.hidden + at_once * most - 1) / (at_once * most);
      const int blocks = std::min(at_once * waves, (s.hidden + 7) / 8);
      const int rows = (s.hidden + blocks - 1) / blocks;
      a.acc_stride = align_up(rows, 4) + 4;
      // as many copies of the sums (each for `group` teams of its own) as there are teams
      const int copy = s.num_tokens * a.acc_stride * 4;
      for (a.sum_copies = a.consumers; a.sum_copies >= 1; --a.sum_copies) {
        if (a.sum_copies * copy > (a.sum_copies > 1 ? budget / 4 : budget / 3)) continue;
        if (!plan(a, w.group, kDown, budget - a.sum_copies * copy, 4)) continue;
        a.group = (rows + a.tile_rows - 1) / a.tile_rows;
        a.teams = a.group * a.sum_copies;
        // (a team keeps its row tile from one k step to the next only if it is the tile's only one)
        if (a.teams > std::min(a.consumers, a.stages) || (a.ksteps > 1 && a.sum_copies > 1))
          continue;
        a.stages = a.stages / a.teams * a.teams;
        fit_parts(a);
        const size_t smem = (size_t)a.stages * a.stage_bytes + a.xstages * a.xslot_bytes +
                            (size_t)a.sum_copies * copy + list_bytes(s);
        return launch_by_group(w.group, a, kDown, blocks * a.cluster, smem, stream);
      }
    }
    if (!small) return cudaErrorInvalidConfiguration;
  }
}

cudaError_t launch_w4_linear(const void* x, int64_t x_stride, int num_tokens, int N,
                             const WeightRows& w, void* out, int64_t out_stride,
                             cudaStream_t stream) {
  const MoeShape s{num_tokens, 1, 1, N, w.K};
  StreamArgs a = common_args(s, x, x_stride, nullptr, w, nullptr, 0, out, out_stride);
  a.N = N;
  a.xrows = num_tokens;
  a.consumers = kMostConsumers;
  if (!plan(a, w.group, kLinear, kSmemLarge, 1)) return cudaErrorInvalidConfiguration;
  fit_teams(a);
  const size_t smem = (size_t)a.stages * a.stage_bytes + a.xstages * a.xslot_bytes;
  return launch_by_group(w.group, a, kLinear, std::min((N + 7) / 8, g_sm_count), smem, stream);
}

cudaError_t prepare_moe_kernels() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&g_sm_count, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = stream_prepare<0>(kSmemLarge, &g_clusters);
  if (e == cudaSuccess) e = stream_prepare<32>(0, nullptr);
  if (e == cudaSuccess) e = stream_prepare<64>(0, nullptr);
  if (e == cudaSuccess) e = stream_prepare<128>(0, nullptr);
  if (e == cudaSuccess && g_clusters < 1) e = cudaErrorInvalidConfiguration;
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
