// What the host side (mol_moe.cu) and the kernels (mol_moe.cuh) of the experts share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mol {

enum StreamMode { kGateUp = 0, kDown = 1, kLinear = 2 };

// Consumer warps of a block: with the tokens' warp sixteen, so a thread may have 128 registers.
constexpr int kMostConsumers = 15;
constexpr int kFewConsumers = 7;
constexpr int kMaxStages = 32;  // of all teams of a block
constexpr int kMaxSlots = 8;    // token slots
// Blocks of a cluster that share output rows (down).
constexpr int kCluster = 4;
// Shared memory of a block: the small one leaves room for a block of the next kernel beside it.
constexpr int kSmemSmall = 112 * 1024;
constexpr int kSmemLarge = 222 * 1024;
struct StreamArgs {
  const __nv_bfloat16* x;  // activation rows: tokens (gate_up, linear) or pairs (down)
  const int32_t* ids;      // [num_tokens * topk], not for the linear
  const float* weights;    // [num_tokens * topk], down only
  const char* w;
  const __nv_bfloat16* scales;
  const __nv_bfloat16* delta;
  __nv_bfloat16* out;      // act, or the output rows
  int64_t x_stride, delta_stride, out_stride;
  int num_tokens, topk, E;
  int K;                   // contraction width
  int N;                   // outputs of one expert: I, H, or the linear's N
  int chained;             // the kernel before is this call's gate_up
  int cluster;             // blocks that share output rows (down), 1 otherwise
  // A stage: `stage_rows` (8 or 16) weight rows of Kc inputs, gate rows and from half_rows on up
  // rows (gate_up); tile_rows outputs.
  int stage_rows, half_rows, tile_rows, Kc, ksteps;
  int entry_rows;          // gate_up, linear: N rounded up to whole tiles (to a tile for each team
                           // where rows come in pieces)
  int row_copies;          // a copy for each row, row_pitch apart; else rows lie as in memory
  int row_pitch, scale_off, scale_pitch, stage_bytes, stages;
  // a token slot: `xrows` activation rows of Kc inputs
  int xrows, x_pitch, xslot_bytes, xstages;
  int group;               // down: row tiles of the block
  int consumers;           // consumer warps that the block has room for, besides the tokens' warp
  int teams, parts;        // teams of `parts` warps in use; the teams divide the stages
  int parts_off;           // of the partial sums inside a stage
  // output sums (down): one copy for each team of a row tile, [num_tokens][acc_stride] floats
  int sum_copies, acc_stride;
};

// One set for each weight format, each in a translation unit of its own (mol_moe_*.cu).
template <int G>
cudaError_t stream_launch(const StreamArgs& a, int mode, int grid, size_t smem, cudaStream_t stream);
template <int G>
cudaError_t stream_prepare(int smem, int* clusters);
template <int G>
cudaError_t stream_take_faults(unsigned* out);
template <int G>
cudaError_t stream_wait_test(unsigned stall, unsigned long long limit_ns);
template <int G>
cudaError_t stream_take_checks(unsigned long long* first, unsigned long long* count);

#define MOL_MOE_DECLARE(G)                                                                    \
  template <>                                                                                 \
  cudaError_t stream_launch<G>(const StreamArgs&, int, int, size_t, cudaStream_t);            \
  template <>                                                                                 \
  cudaError_t stream_prepare<G>(int, int*);                                                   \
  template <>                                                                                 \
  cudaError_t stream_take_faults<G>(unsigned*);                                               \
  template <>                                                                                 \
  cudaError_t stream_wait_test<G>(unsigned, unsigned long long);                              \
  template <>                                                                                 \
  cudaError_t stream_take_checks<G>(unsigned long long*, unsigned long long*);
MOL_MOE_DECLARE(0)
MOL_MOE_DECLARE(32)
MOL_MOE_DECLARE(64)
MOL_MOE_DECLARE(128)
#undef MOL_MOE_DECLARE

}  // namespace mol
