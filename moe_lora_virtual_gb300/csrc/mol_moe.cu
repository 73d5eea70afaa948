// The experts of a MoE layer for a few tokens and the 4-bit linear (include/mol_block.h).
//
// Plain kernels: one warp per weight row and token, fp32 dot products.

#include <type_traits>

#include "mol_block.h"
#include "mol_device.cuh"
#include "mol_internal.h"

namespace mol {
namespace {

MOL_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The dot product of weight row `row` with x (K elements): every lane gets the sum.
// G = 0: bf16 rows; else 4-bit rows with a scale per G inputs.
template <int G>
MOL_DEV float row_dot(const WeightRows& w, int64_t row, const __nv_bfloat16* x) {
  const int lane = threadIdx.x & 31;
  float acc = 0.f;
  if constexpr (G == 0) {
    const uint4* wr = reinterpret_cast<const uint4*>(
        static_cast<const __nv_bfloat16*>(w.data) + row * w.K);
    const uint4* xr = reinterpret_cast<const uint4*>(x);
    for (int c = lane; c < w.K / 8; c += 32) {
      const uint4 a = wr[c], b = xr[c];
      const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc = fmaf(bf16_lo(av[i]), bf16_lo(bv[i]), acc);
        acc = fmaf(bf16_hi(av[i]), bf16_hi(bv[i]), acc);
      }
    }
  } else {
    const int Kp = w4_padded(w.K);
    const uint32_t* wr = static_cast<const uint32_t*>(w.data) + row * (Kp / 8);
    const __nv_bfloat16* sr = static_cast<const __nv_bfloat16*>(w.scales) + row * (Kp / G);
    for (int c = lane; c < w.K / 8; c += 32) {  // eight inputs 8c .. 8c + 7
      const int block = c >> 4, i = (c & 15) >> 2, t = c & 3;
      const uint32_t q = wr[block * 16 + 4 * t + i];
      const uint4 b = reinterpret_cast<const uint4*>(x)[c];
      const uint32_t bv[4] = {b.x, b.y, b.z, b.w};
      float s = 0.f;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        s = fmaf((float)((int)((q >> (4 * p)) & 15) - 8), bf16_lo(bv[p]), s);
        s = fmaf((float)((int)((q >> (16 + 4 * p)) & 15) - 8), bf16_hi(bv[p]), s);
      }
      acc = fmaf(__bfloat162float(sr[8 * c / G]), s, acc);
    }
  }
  return warp_sum(acc);
}

constexpr int kWarps = 8;

template <int G>
__global__ void __launch_bounds__(kWarps * 32)
    moe_gate_up_kernel(MoeShape s, const __nv_bfloat16* x, int64_t x_stride,
                       const int32_t* topk_ids, WeightRows w, const __nv_bfloat16* delta,
                       int64_t delta_stride, __nv_bfloat16* act) {
  pdl_wait();
  const int pair = blockIdx.y, j = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int e = topk_ids[pair];
  if (e < 0 || e >= s.num_experts || j >= s.inter) return;
  const __nv_bfloat16* xr = x + (pair / s.topk) * x_stride;
  const int64_t base = (int64_t)e * 2 * s.inter;
  float g = row_dot<G>(w, base + j, xr), u = row_dot<G>(w, base + s.inter + j, xr);
  if ((threadIdx.x & 31) != 0) return;
  if (delta) {
    g += __bfloat162float(delta[pair * delta_stride + j]);
    u += __bfloat162float(delta[pair * delta_stride + s.inter + j]);
  }
  act[(int64_t)pair * s.inter + j] = __float2bfloat16(g / (1.f + expf(-g)) * u);
}

template <int G>
__global__ void __launch_bounds__(kWarps * 32)
    moe_down_kernel(MoeShape s, const __nv_bfloat16* act, const int32_t* topk_ids,
                    const float* topk_weights, WeightRows w, const __nv_bfloat16* delta,
                    int64_t delta_stride, __nv_bfloat16* out, int64_t out_stride) {
  pdl_wait();
  const int t = blockIdx.y, n = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (n >= s.hidden) return;
  float acc = 0.f;
  for (int k = 0; k < s.topk; ++k) {
    const int pair = t * s.topk + k, e = topk_ids[pair];
    if (e < 0 || e >= s.num_experts) continue;
    float d = row_dot<G>(w, (int64_t)e * s.hidden + n, act + (int64_t)pair * s.inter);
    if (delta) d += __bfloat162float(delta[pair * delta_stride + n]);
    acc = fmaf(topk_weights[pair], d, acc);
  }
  if ((threadIdx.x & 31) == 0) out[t * out_stride + n] = __float2bfloat16(acc);
}

template <int G>
__global__ void __launch_bounds__(kWarps * 32)
    w4_linear_kernel(const __nv_bfloat16* x, int64_t x_stride, int N, WeightRows w,
                     __nv_bfloat16* out, int64_t out_stride) {
  pdl_wait();
  const int t = blockIdx.y, n = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (n >= N) return;
  const float d = row_dot<G>(w, n, x + t * x_stride);
  if ((threadIdx.x & 31) == 0) out[t * out_stride + n] = __float2bfloat16(d);
}

template <typename F>
cudaError_t by_group(int group, F f) {
  if (group == 0) return f(std::integral_constant<int, 0>{});
  if (group == 32) return f(std::integral_constant<int, 32>{});
  if (group == 64) return f(std::integral_constant<int, 64>{});
  return f(std::integral_constant<int, 128>{});
}

using bf16 = __nv_bfloat16;

}  // namespace

cudaError_t launch_moe_gate_up(const MoeShape& s, const void* x, int64_t x_stride,
                               const int32_t* topk_ids, const WeightRows& w, const void* delta,
                               int64_t delta_stride, void* act, cudaStream_t stream) {
  const dim3 grid((s.inter + kWarps - 1) / kWarps, s.num_tokens * s.topk);
  return by_group(w.group, [&](auto g) {
    return launch_pdl(moe_gate_up_kernel<decltype(g)::value>, grid, dim3(kWarps * 32), 0, stream, s,
                      static_cast<const bf16*>(x), x_stride, topk_ids, w,
                      static_cast<const bf16*>(delta), delta_stride, static_cast<bf16*>(act));
  });
}

cudaError_t launch_moe_down(const MoeShape& s, const void* act, const int32_t* topk_ids,
                            const float* topk_weights, const WeightRows& w, const void* delta,
                            int64_t delta_stride, void* out, int64_t out_stride, bool chained,
                            cudaStream_t stream) {
  (void)chained;
  const dim3 grid((s.hidden + kWarps - 1) / kWarps, s.num_tokens);
  return by_group(w.group, [&](auto g) {
    return launch_pdl(moe_down_kernel<decltype(g)::value>, grid, dim3(kWarps * 32), 0, stream, s,
                      static_cast<const bf16*>(act), topk_ids, topk_weights, w,
                      static_cast<const bf16*>(delta), delta_stride, static_cast<bf16*>(out),
                      out_stride);
  });
}

cudaError_t launch_w4_linear(const void* x, int64_t x_stride, int num_tokens, int N,
                             const WeightRows& w, void* out, int64_t out_stride,
                             cudaStream_t stream) {
  const dim3 grid((N + kWarps - 1) / kWarps, num_tokens);
  return by_group(w.group, [&](auto g) {
    return launch_pdl(w4_linear_kernel<decltype(g)::value>, grid, dim3(kWarps * 32), 0, stream,
                      static_cast<const bf16*>(x), x_stride, N, w, static_cast<bf16*>(out),
                      out_stride);
  });
}

cudaError_t prepare_moe_kernels() { return cudaSuccess; }

cudaError_t take_moe_checks(unsigned long long* first, unsigned long long* count) {
  CheckRecord r;
  const cudaError_t e = take_check_record_here(&r);
  *first = r.first;
  *count = r.count;
  return e;
}

}  // namespace mol
