// Norms between blocks and the router's choice (include/mol_block.h).

#include <algorithm>
#include <type_traits>

#include "mol_block.h"
#include "mol_device.cuh"
#include "mol_internal.h"

namespace mol {
namespace {

// Sum of one float per thread over the block, the same value in every thread; the
// warps' sums are added in their order (deterministic). `sh` holds one float per warp
// and is free again for another call on a different half.
template <int THREADS>
MOL_DEV float block_sum(float v, float* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (THREADS > 32) {
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) v += sh[w];
  }
  return v;
}

MOL_DEV void unpack8(const uint4& q, float (&f)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}
MOL_DEV uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

constexpr int kNormWarps = 4;

// One block per row, or a warp for short rows, CPT chunks of 8 elements per thread, the row held in fp32
// registers between the two sums: y, the residual and the gate are read once and both
// outputs written once, so the kernel moves what the operator cannot do without (8
// bytes an element, 10 with a gate per token) and is bound by HBM for many rows, by the
// launch and three dependent round trips (loads, two block sums) for a few.
// Shared-memory halves: a second sum may start before every thread has read the first.
template <int THREADS, int CPT>
__global__ void __launch_bounds__(THREADS == 32 ? 32 * kNormWarps : THREADS) block_norm_kernel(NormArgs a) {
  __shared__ float sh[2][THREADS / 32];
  const int chunks = a.H >> 3;
  const int64_t row = THREADS == 32 ? (int64_t)blockIdx.x * blockDim.y + threadIdx.y : blockIdx.x;
  if (THREADS == 32 && row >= a.rows) return;
  const uint4* yr = reinterpret_cast<const uint4*>(
      static_cast<const __nv_bfloat16*>(a.y) + row * a.y_stride);
  const uint4* rr = reinterpret_cast<const uint4*>(
      static_cast<const __nv_bfloat16*>(a.residual) + row * a.residual_stride);
  const uint4* gr = reinterpret_cast<const uint4*>(
      static_cast<const __nv_bfloat16*>(a.gate) + (a.gate ? row * a.gate_stride : 0));
  const uint4* post = static_cast<const uint4*>(a.post_weight);
  const uint4* pre = static_cast<const uint4*>(a.pre_weight);
  pdl_wait();
  pdl_launch_dependents();
  uint4 yq[CPT], rq[CPT], gq[CPT];
#pragma unroll
  for (int c = 0; c < CPT; ++c) {
    const int i = threadIdx.x + c * THREADS;
    const bool in = i < chunks;
    yq[c] = in ? yr[i] : make_uint4(0, 0, 0, 0);
    rq[c] = in ? rr[i] : make_uint4(0, 0, 0, 0);
    gq[c] = in && a.gate ? gr[i] : make_uint4(0, 0, 0, 0);
  }
  float v[CPT][8];
  float rn = 1.f;
  if (post) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      float f[8];
      unpack8(yq[c], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fmaf(f[j], f[j], s);
    }
    s = block_sum<THREADS>(s, sh[0]);
    rn = rsqrtf(s / (float)a.H + a.eps);
  }
  float s2 = 0.f;
#pragma unroll
  for (int c = 0; c < CPT; ++c) {
    const int i = threadIdx.x + c * THREADS;
    float f[8], r[8], m[8];
    unpack8(yq[c], f);
    unpack8(rq[c], r);
    if (post) {
      unpack8(i < chunks ? post[i] : make_uint4(0, 0, 0, 0), m);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = f[j] * rn * m[j];
    }
    if (a.gate) {
      unpack8(gq[c], m);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= m[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[c][j] = r[j] + a.residual_scale * f[j];
      s2 = fmaf(v[c][j], v[c][j], s2);
    }
    if (i < chunks)
      reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.residual_out) +
                               row * a.residual_out_stride)[i] = pack8(v[c]);
  }
  if (!pre) return;
  s2 = block_sum<THREADS>(s2, sh[1]);
  const float rn2 = rsqrtf(s2 / (float)a.H + a.eps);
#pragma unroll
  for (int c = 0; c < CPT; ++c) {
    const int i = threadIdx.x + c * THREADS;
    if (i >= chunks) break;
    float m[8];
    unpack8(pre[i], m);
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = v[c][j] * rn2 * m[j];
    reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.normed) + row * a.normed_stride)[i] =
        pack8(m);
  }
}

// Key whose unsigned order is the order of the logits: -infinity and NaN give 0 (never
// taken), zeros of both signs the same key.
MOL_DEV uint32_t order_key(float v) {
  if (!(v > -INFINITY)) return 0u;  // -infinity, NaN
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
MOL_DEV float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
MOL_DEV float load_logit(const float* p) { return *p; }
MOL_DEV float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// exp(l - max), 1 for l = max (also where both are +infinity).
MOL_DEV float soft(float l, float top) { return l == top ? 1.f : expf(l - top); }

constexpr int kRouteWarps = 4;

// A logit and its expert as one unsigned number, larger for what is taken first: the order key, then
// the lower index; 0 for what is never taken. bf16 keys fit 16 bits (the other 16 follow from the
// sign), so one 32-bit reduction finds a round's choice; fp32 takes 64 bits and two.
MOL_DEV void pack(float v, int e, uint32_t& out) {
  const uint32_t k = order_key(v) >> 16;
  out = k ? k << 16 | (0xFFFFu - e) : 0u;
}
MOL_DEV void pack(float v, int e, uint64_t& out) {
  const uint32_t k = order_key(v);
  out = k ? (uint64_t)k << 32 | (0xFFFFu - e) : 0ull;
}
MOL_DEV float packed_value(uint32_t c) {
  return key_value((c & 0xFFFF0000u) | ((c >> 31) ? 0u : 0xFFFFu));
}
MOL_DEV float packed_value(uint64_t c) { return key_value((uint32_t)(c >> 32)); }
template <typename P>
MOL_DEV int packed_expert(P c) {
  return 0xFFFF - (int)(c & 0xFFFFu);
}
MOL_DEV uint32_t warp_largest(uint32_t c) { return __reduce_max_sync(0xffffffffu, c); }
MOL_DEV uint64_t warp_largest(uint64_t c) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(c >> 32));
  const uint32_t lo = (uint32_t)(c >> 32) == hi ? (uint32_t)c : 0u;
  return (uint64_t)hi << 32 | __reduce_max_sync(0xffffffffu, lo);
}

// Sorts n (a power of two) numbers downwards: Batcher's odd-even merge.
template <int N, typename P>
MOL_DEV void sort_down(P (&c)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2) {
#pragma unroll
    for (int k = p; k >= 1; k /= 2) {
#pragma unroll
      for (int i = 0; i + k < N; ++i) {
        // (pairs i, i + k of one block of 2p, in every other run of k from k % p on)
        const bool pair = i >= k % p && (i - k % p) / k % 2 == 0 && i / (2 * p) == (i + k) / (2 * p);
        if (pair) {
          const P a = c[i], b = c[i + k];
          c[i] = a > b ? a : b;
          c[i + k] = a > b ? b : a;
        }
      }
    }
  }
}

// One warp per row: lane l sorts the logits of experts l, l + 32, ... in its registers; each of the
// topk rounds takes the largest of the lanes' first ones (one warp reduction, two for fp32), whose
// lane moves its list up. Comparisons only, so the choice is exact, and each number is distinct, so
// the lower index wins. The row is read once, its exponentials are summed in fp32. Bound by
// instructions for many rows: about 630 a row at 256 bf16 experts and topk 8, 76 % of the issue slots
// (8192 such rows: 6.6 us, 0.7 for their bytes, 11.0 with a search of all keys in each round); few
// rows by the launch and the rounds' latency (23 rows of 128: 1.6 us).
template <typename T, int VPL>
__global__ void __launch_bounds__(kRouteWarps * 32)
    moe_route_kernel(const T* __restrict__ logits, int64_t row_stride, int64_t rows, int E,
                     int topk, bool renorm, float scale, int32_t* __restrict__ ids,
                     float* __restrict__ weights) {
  using P = std::conditional_t<std::is_same_v<T, float>, uint64_t, uint32_t>;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  pdl_wait();
  pdl_launch_dependents();
  if (row >= rows) return;
  const T* p = logits + row * row_stride;
  float l[VPL];
  P c[VPL], best = 0;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = lane + 32 * j;
    l[j] = e < E ? load_logit(p + e) : -INFINITY;
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    pack(l[j], lane + 32 * j, c[j]);
    best = c[j] > best ? c[j] : best;
  }
  best = warp_largest(best);
  const float top = packed_value(best);
  float all = 0.f;
  if (!renorm) {
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (c[j]) all += soft(l[j], top);
  }
  sort_down(c);
  P mine = 0;
  for (int r = 0; r < topk && best != 0; ++r) {
    if (lane == r) mine = best;
    const bool taken = c[0] == best;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (taken) c[j] = j + 1 < VPL ? c[j + 1 < VPL ? j + 1 : j] : 0;
    best = warp_largest(c[0]);
  }
  const float my_w = mine ? soft(packed_value(mine), top) : 0.f;
  float sum = renorm ? my_w : all;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane < topk) {
    ids[row * topk + lane] = mine ? packed_expert(mine) : -1;
    weights[row * topk + lane] = mine ? my_w * scale / sum : 0.f;
  }
}

template <typename T>
cudaError_t route_by_width(const T* logits, int64_t row_stride, int64_t rows, int E, int topk,
                           bool renorm, float scale, int32_t* ids, float* weights,
                           cudaStream_t stream) {
  const dim3 grid((unsigned)((rows + kRouteWarps - 1) / kRouteWarps)), block(kRouteWarps * 32);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, block, 0, stream, logits, row_stride, rows, E, topk, renorm,
                      scale, ids, weights);
  };
  const int vpl = (E + 31) / 32;
  if (vpl <= 1) return go(moe_route_kernel<T, 1>);
  if (vpl <= 2) return go(moe_route_kernel<T, 2>);
  if (vpl <= 4) return go(moe_route_kernel<T, 4>);
  if (vpl <= 8) return go(moe_route_kernel<T, 8>);
  if (vpl <= 16) return go(moe_route_kernel<T, 16>);
  return go(moe_route_kernel<T, 32>);
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t stream) {
  // A warp a row, four rows a block where there are many: no sum waits for other warps, and small
  // blocks do not use up an SM's (8000 rows of 256: 3.6 us against 8.4 with a block each). Rows of up
  // to 512 only where there are many (8000: 5.9 us against 9.5; 23 rows: 2.2 against 1.8).
  const int chunks = a.H / 8;
  const bool many = a.rows > 2048;
  auto go = [&](auto kernel, int threads) {
    const int warps = threads == 32 && many ? kNormWarps : 1;
    return launch_pdl(kernel, dim3((unsigned)((a.rows + warps - 1) / warps)), dim3(threads, warps), 0,
                      stream, a);
  };
  if (chunks <= 32) return go(block_norm_kernel<32, 1>, 32);
  if (chunks <= 64 && many) return go(block_norm_kernel<32, 2>, 32);
  if (chunks <= 128) return go(block_norm_kernel<128, 1>, 128);
  if (chunks <= 256) return go(block_norm_kernel<256, 1>, 256);
  if (chunks <= 512) return go(block_norm_kernel<256, 2>, 256);
  if (chunks <= 1024) return go(block_norm_kernel<512, 2>, 512);
  return go(block_norm_kernel<512, 4>, 512);
}

cudaError_t launch_moe_route(const void* logits, bool bf16, int64_t row_stride, int64_t rows,
                             int num_experts, int topk, bool renormalize, float scale,
                             int32_t* ids, float* weights, cudaStream_t stream) {
  if (bf16)
    return route_by_width(static_cast<const __nv_bfloat16*>(logits), row_stride, rows, num_experts,
                          topk, renormalize, scale, ids, weights, stream);
  return route_by_width(static_cast<const float*>(logits), row_stride, rows, num_experts, topk,
                        renormalize, scale, ids, weights, stream);
}

cudaError_t take_block_checks(unsigned long long* first, unsigned long long* count) {
  CheckRecord r;
  const cudaError_t e = take_check_record_here(&r);
  *first = r.first;
  *count = r.count;
  return e;
}

}  // namespace mol
