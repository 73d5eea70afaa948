// The host side of the experts and the 4-bit linear without a GPU: reads calls, prints the launches that
// they would make on a device of 152 SMs. A line "gate_up G T k E H I", "down ...", "split ..." or
// "linear G T K N" gives a line of launches, each "key=value" pairs in braces, or "none".
#include <cstdio>
#include <cstring>
#include <string>
#include <type_traits>

#include "mol_moe.cu"

namespace mol {
static std::string launches;

static cudaError_t record(const StreamArgs& a, int mode, int group, int grid, size_t smem) {
  char line[1024];
  std::snprintf(
      line, sizeof line,
      "{mode=%d group=%d grid=%d smem=%zu x=%lld out=%lld tokens=%d topk=%d E=%d K=%d N=%d cluster=%d Kc=%d "
      "ksteps=%d tile_rows=%d entry_rows=%d span_shift=%d row_copies=%d row_pitch=%d scale_off=%d "
      "scale_pitch=%d stage_bytes=%d stages=%d xrows=%d x_pitch=%d xslot_bytes=%d xstages=%d x_off=%d "
      "chunks=%d teams=%d parts=%d acc_stride=%d} ",
      mode, group, grid, smem, (long long)(uintptr_t)a.x, (long long)(uintptr_t)a.out, a.num_tokens,
      a.topk, a.E, a.K, a.N, a.cluster, a.Kc, a.ksteps, a.tile_rows, a.entry_rows, a.span_shift,
      a.row_copies, a.row_pitch, a.scale_off, a.scale_pitch, a.stage_bytes, a.stages, a.xrows, a.x_pitch,
      a.xslot_bytes, a.xstages, a.x_off, a.chunks, a.teams, a.parts, a.acc_stride);
  launches += line;
  return cudaSuccess;
}

#define STAND_IN(G)                                                                              \
  template <>                                                                                    \
  cudaError_t stream_launch<G>(const StreamArgs& a, int mode, int grid, size_t smem,             \
                               cudaStream_t) {                                                   \
    return record(a, mode, G, grid, smem);                                                       \
  }                                                                                              \
  template <>                                                                                    \
  cudaError_t stream_prepare<G>(int*) {                                                          \
    return cudaSuccess;                                                                          \
  }                                                                                              \
  template <>                                                                                    \
  cudaError_t stream_take_faults<G>(unsigned*) {                                                 \
    return cudaSuccess;                                                                          \
  }                                                                                              \
  template <>                                                                                    \
  cudaError_t stream_wait_test<G>(unsigned, unsigned long long) {                                \
    return cudaSuccess;                                                                          \
  }                                                                                              \
  template <>                                                                                    \
  cudaError_t stream_take_checks<G>(unsigned long long*, unsigned long long*) {                  \
    return cudaSuccess;                                                                          \
  }
STAND_IN(0)
STAND_IN(32)
STAND_IN(64)
STAND_IN(128)
void count_launch() {}
}  // namespace mol

int main() {
  using namespace mol;
  g_sm_count = 152;
  g_clusters[0] = 152;
  g_clusters[1] = 76;
  g_clusters[2] = 36;
  char what[16];
  int G;
  // (addresses are never followed; one away from 0 tells the tokens of each launch)
  char* const p = reinterpret_cast<char*>((uintptr_t)1 << 40);
  while (std::scanf("%15s %d", what, &G) == 2) {
    launches.clear();
    cudaError_t e = cudaSuccess;
    const void* scales = G ? p : nullptr;
    if (!std::strcmp(what, "linear")) {
      int T, K, N;
      if (std::scanf("%d %d %d", &T, &K, &N) != 3) return 1;
      e = launch_w4_linear(p, K, T, N, WeightRows{p, scales, K, G}, p, N, nullptr);
    } else {
      MoeShape s;
      if (std::scanf("%d %d %d %d %d", &s.num_tokens, &s.topk, &s.num_experts, &s.hidden, &s.inter) != 5)
        return 1;
      const int32_t* ids = reinterpret_cast<int32_t*>(p);
      const float* w = reinterpret_cast<float*>(p);
      if (!std::strcmp(what, "gate_up"))
        e = launch_moe_gate_up(s, p, s.hidden, ids, WeightRows{p, scales, s.hidden, G}, nullptr, 0, p,
                               nullptr);
      else if (!std::strcmp(what, "down"))
        e = launch_moe_down(s, p, ids, w, WeightRows{p, scales, s.inter, G}, nullptr, 0, p, s.hidden,
                            false, nullptr);
      else if (moe_split_bytes(s, G))  // (its sums, a launch of this file, fail without a GPU)
        launch_moe_down_split(s, p, ids, w, WeightRows{p, scales, s.inter, G}, nullptr, 0, p, p,
                              s.hidden, false, nullptr);
    }
    std::printf("%s\n", e == cudaSuccess && !launches.empty() ? launches.c_str() : "none");
  }
  return 0;
}
