// The C entry points' host code without CUDA: the calls of the runtime and the launchers that it makes
// are stand-ins here, so what each entry point prepares on a device can be counted.
#include <cstdio>

#include "mol_block.h"
#include "mol_internal.h"

namespace {
int lora_prepared = 0, moe_prepared = 0, launched = 0;
cudaError_t lora_result = cudaSuccess, moe_result = cudaSuccess;
}  // namespace

extern "C" cudaError_t cudaGetDevice(int* dev) {
  *dev = 0;
  return cudaSuccess;
}
extern "C" cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : 3;
  return cudaSuccess;
}

namespace mol {
cudaError_t prepare_kernels() {
  ++lora_prepared;
  return lora_result;
}
cudaError_t prepare_moe_kernels() {
  ++moe_prepared;
  return moe_result;
}
cudaError_t launch_virtual_topk(const int32_t*, const int32_t*, int64_t, int, int, int, int32_t*,
                                cudaStream_t) {
  ++launched;
  return cudaSuccess;
}
cudaError_t launch_block_norm(const NormArgs&, cudaStream_t) {
  ++launched;
  return cudaSuccess;
}
cudaError_t launch_moe_route(const void*, bool, int64_t, int64_t, int, int, bool, float, int32_t*,
                             float*, cudaStream_t) {
  ++launched;
  return cudaSuccess;
}
cudaError_t launch_moe_gate_up(const MoeShape&, const void*, int64_t, const int32_t*,
                               const WeightRows&, const void*, int64_t, void*, cudaStream_t) {
  ++launched;
  return cudaSuccess;
}
cudaError_t launch_moe_down(const MoeShape&, const void*, const int32_t*, const float*,
                            const WeightRows&, const void*, int64_t, void*, int64_t, bool,
                            cudaStream_t) {
  ++launched;
  return cudaSuccess;
}
size_t moe_split_bytes(const MoeShape&, int) { return 0; }
cudaError_t launch_w4_linear(const void*, int64_t, int, int, const WeightRows&, void*, int64_t,
                             cudaStream_t) {
  ++launched;
  return cudaSuccess;
}
}  // namespace mol

namespace {
alignas(16) char buf[64];
int32_t* ids = reinterpret_cast<int32_t*>(buf);
float* weights = reinterpret_cast<float*>(buf);

int32_t topk() { return mol_virtual_topk(ids, ids, 1, 1, 1, 1, ids, nullptr); }
int32_t norm() {
  return mol_block_norm(buf, 8, buf, 8, nullptr, nullptr, 0, 1.f, buf, 1e-6f, 1, 8, buf, 8, buf, 8, nullptr);
}
int32_t route() { return mol_moe_route(buf, MOL_F32, 8, 1, 8, 1, 1, 1.f, ids, weights, nullptr); }
int32_t gate_up() {
  return mol_moe_gate_up(buf, 8, ids, 1, 1, 1, 8, 8, buf, nullptr, 0, nullptr, 0, buf, nullptr);
}
int32_t down() {
  return mol_moe_down(buf, ids, weights, 1, 1, 1, 8, 8, buf, nullptr, 0, nullptr, 0, buf, 8, nullptr);
}
int32_t down_split() {
  return mol_moe_down_split(buf, ids, weights, 1, 1, 1, 8, 8, buf, nullptr, 0, nullptr, 0, nullptr, 0,
                            buf, 8, nullptr);
}
int32_t forward() {
  return mol_moe_forward(buf, 8, ids, weights, 1, 1, 1, 8, 8, buf, nullptr, buf, nullptr, 0, buf, buf, 8,
                         nullptr);
}
int32_t linear() { return mol_w4_linear(buf, 8, 1, 8, 1, buf, buf, 32, buf, 8, nullptr); }
}  // namespace

#define EXPECT(cond)                                       \
  do {                                                     \
    if (!(cond)) {                                         \
      std::printf("line %d: not %s\n", __LINE__, #cond);   \
      return 1;                                            \
    }                                                      \
  } while (0)

int main() {
  int32_t (*const experts[])() = {gate_up, down, down_split, forward, linear};
  // neither set of kernels can be had: everything is refused, nothing launched
  lora_result = moe_result = cudaErrorInvalidConfiguration;
  EXPECT(topk() == MOL_ERR_CUDA && route() == MOL_ERR_CUDA && linear() == MOL_ERR_CUDA);
  EXPECT(mol_last_cuda_error() == cudaErrorInvalidConfiguration && moe_prepared == 0);
  // the experts' kernels cannot be had: their calls alone are refused
  lora_result = cudaSuccess;
  EXPECT(topk() == MOL_OK && norm() == MOL_OK && route() == MOL_OK && moe_prepared == 0);
  const int before = launched;
  for (auto call : experts) EXPECT(call() == MOL_ERR_CUDA);
  EXPECT(launched == before && moe_prepared == 5);
  EXPECT(topk() == MOL_OK && norm() == MOL_OK && route() == MOL_OK);
  // they can: each set is prepared once
  moe_result = cudaSuccess;
  const int lora = lora_prepared;
  for (int i = 0; i < 2; ++i)
    for (auto call : experts) EXPECT(call() == MOL_OK);
  EXPECT(topk() == MOL_OK && lora_prepared == lora && moe_prepared == 6);
  std::printf("ok\n");
  return 0;
}
