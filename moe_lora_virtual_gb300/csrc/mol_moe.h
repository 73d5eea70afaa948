// What the host side (mol_moe.cu) and the kernels (mol_moe.cuh) of the experts share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mol {

enum StreamMode { kGateUp = 0, kDown = 1, kLinear = 2, kPairs = 3 };  // kPairs: down's split form

// Warps of a block of down; at 16 a thread may have 128 registers.
constexpr int kBlockWarps = 16;
// gate_up, linear: consumer warps of a block, by its token tiles. One more brings the tokens' rows; a
// seventeenth warp lowers the registers of a thread to 96, too few for many tokens' sums.
__host__ __device__ constexpr int consumer_warps(int token_tiles) { return token_tiles <= 2 ? 16 : 15; }
// gate_up, linear: a warp's ring of chunks (of 2 where tokens need the room). A chunk is 128 bytes of
// each of a tile's 16 weight rows, and their scales.
constexpr int kChunks = 4;
__host__ __device__ constexpr int chunk_bytes(int group) { return 2048 + (group ? 16 * 512 / group : 0); }
constexpr int kListThreads = 512;  // of a block's first warps group the pairs by expert
constexpr int kMaxStages = 32;  // of all teams of a block
constexpr int kClusterSizes = 3;  // down: clusters of 1, 2 or 4 blocks
constexpr int kSmem = 222 * 1024;
constexpr int kDownRows = 64;     // output rows of a block of the down kernel at most

struct StreamArgs {
  const __nv_bfloat16* x;  // activation rows: tokens (gate_up, linear) or pairs (down)
  const int32_t* ids;      // [num_tokens * topk], not for the linear
  const float* weights;    // [num_tokens * topk], down only
  const char* w;
  const __nv_bfloat16* scales;
  const __nv_bfloat16* delta;
  __nv_bfloat16* out;      // act, or the output rows
  float* partial;          // kPairs: [num_tokens * topk, N]
  int64_t x_stride, delta_stride, out_stride;
  int num_tokens, topk, E;
  int K;                   // contraction width
  int N;                   // outputs of one expert: I, H, or the linear's N
  int chained;             // the kernel before is this call's gate_up
  int cluster;             // blocks that share output rows (down), 1 otherwise
  int Kc, ksteps;          // inputs of a step (all of them, or a piece), steps of a row
  int tile_rows;           // gate_up, linear: outputs of a tile
  int entry_rows;          // and N rounded up to whole tiles (to a tile for each team where rows come
                           // in pieces)
  int span_shift;          // down: bytes between spans of 8 rows
  int row_copies;          // pieces of rows: a copy for each row; else whole rows, a copy a span
  int row_pitch, scale_off, scale_pitch, stage_bytes, stages;
  // `xrows` activation rows of Kc inputs: a token slot, or at x_off of a stage (down)
  int xrows, x_pitch, xslot_bytes, xstages, x_off;
  int chunks;              // gate_up, linear: of a warp's ring
  int teams, parts;        // teams of `parts` warps in use; the teams divide the stages
  int acc_stride;          // down: floats between tokens of a team's sums
};

// One set for each weight format, each in a translation unit of its own (mol_moe_*.cu).
template <int G>
cudaError_t stream_launch(const StreamArgs& a, int mode, int grid, size_t smem, cudaStream_t stream);
template <int G>
cudaError_t stream_prepare(int* clusters);
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
  cudaError_t stream_prepare<G>(int*);                                                        \
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
