// Rotary positions and the append to a paged cache (include/mol_attn.h).

#include "mol_attend.h"
#include "mol_device.cuh"
#include "mol_internal.h"

namespace mol {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kMaxPairs = 256;  // half of the widest head

// Eight bf16 values of a 16-byte chunk.
union Chunk {
  uint4 q;
  uint32_t w[4];
};

// cos and sin (times the magnitude) of position * f. The product and its turns are in 64 bits, since
// position 2^20 leaves an fp32 product less than a sixteenth of a radian; what is left after whole
// turns lies within [-pi, pi], where the fast sine and cosine are off by 2^-21 at most, far below
// half a bf16 step of the turned values (2^-9).
MOL_DEV float2 turn(int position, float f, float magnitude) {
  const double angle = (double)position * (double)f;
  const double turns = rint(angle * 0.15915494309189535);         // 1 / (2 pi)
  const float r = (float)fma(turns, -6.283185307179586, angle);   // 2 pi
  float s, c;
  __sincosf(r, &s, &c);
  return make_float2(c * magnitude, s * magnitude);
}

MOL_DEV void turn_pair(float& a, float& b, float2 cs) {
  const float x = a * cs.x - b * cs.y;
  b = b * cs.x + a * cs.y;
  a = x;
}

// A block per token. Its angles are the same for every head: computed once, one a thread, and kept in
// shared memory; then each thread turns 16-byte chunks (in the half layout a chunk and its partner,
// half the turned width on) of the token's heads, queries, keys and values in one list. Bound by HBM
// for many tokens (each value read and written once), by the launch and two dependent round trips
// (position or slot, then values) for a few.
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a) {
  __shared__ float2 cs[kMaxPairs];
  const int64_t t = blockIdx.x;
  const int chunks = a.head_dim >> 3;
  // units of a turned head: chunk pairs and single chunks behind them, or single chunks
  const int pairs = a.interleaved ? 0 : a.rotary_dim >> 4;
  const int turned = a.rotary_dim >> 3;
  const int units = chunks - pairs;
  pdl_wait();
  pdl_launch_dependents();
  if (a.inv_freq) {
    const int p = a.positions[t];
    for (int i = threadIdx.x; i < a.rotary_dim / 2; i += kRopeThreads)
      cs[i] = turn(p, a.inv_freq[i], a.magnitude);
  }
  int64_t slot = -1;
  if (a.slots) slot = a.slots[t];
  const bool keep = slot >= 0 && slot < a.num_slots;
  int64_t cache_at = 0;
  if (keep) {
    const int64_t page = slot / a.page_size;
    cache_at = page * a.page_stride + (slot - page * a.page_size) * a.token_stride;
  }
  __syncthreads();
  const int nq = a.in[0].heads * units, nk = keep ? a.in[1].heads * units : 0,
            nv = keep ? a.in[2].heads * chunks : 0;
  for (int i = threadIdx.x; i < nq + nk + nv; i += kRopeThreads) {
    const int which = i < nq ? 0 : i < nq + nk ? 1 : 2;
    const int j = which == 0 ? i : which == 1 ? i - nq : i - nq - nk;
    const int per = which == 2 ? chunks : units;
    const int head = j / per;
    const int u = j - head * per;
    const HeadRows& in = a.in[which];
    const uint16_t* src = static_cast<const uint16_t*>(in.x) + t * in.token_stride + head * in.head_stride;
    uint16_t* dst = which == 0 ? static_cast<uint16_t*>(a.q_out) + t * a.q_out_token_stride +
                                     head * a.q_out_head_stride
                               : static_cast<uint16_t*>(which == 1 ? a.k_cache : a.v_cache) + cache_at +
                                     head * a.head_stride;
    if (which == 2) {
      reinterpret_cast<uint4*>(dst)[u] = reinterpret_cast<const uint4*>(src)[u];
    } else if (a.interleaved) {
      Chunk c;
      c.q = reinterpret_cast<const uint4*>(src)[u];
      if (u < turned) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = bf16_lo(c.w[e]), y = bf16_hi(c.w[e]);
          turn_pair(x, y, cs[4 * u + e]);
          c.w[e] = pack_bf16x2(x, y);
        }
      }
      reinterpret_cast<uint4*>(dst)[u] = c.q;
    } else if (u < pairs) {
      Chunk c, d;
      c.q = reinterpret_cast<const uint4*>(src)[u];
      d.q = reinterpret_cast<const uint4*>(src)[u + pairs];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x0 = bf16_lo(c.w[e]), x1 = bf16_hi(c.w[e]), y0 = bf16_lo(d.w[e]), y1 = bf16_hi(d.w[e]);
        turn_pair(x0, y0, cs[8 * u + 2 * e]);
        turn_pair(x1, y1, cs[8 * u + 2 * e + 1]);
        c.w[e] = pack_bf16x2(x0, x1);
        d.w[e] = pack_bf16x2(y0, y1);
      }
      reinterpret_cast<uint4*>(dst)[u] = c.q;
      reinterpret_cast<uint4*>(dst)[u + pairs] = d.q;
    } else {
      reinterpret_cast<uint4*>(dst)[u + pairs] = reinterpret_cast<const uint4*>(src)[u + pairs];
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream) {
  return launch_pdl(rope_kernel, dim3((unsigned)a.num_tokens), dim3(kRopeThreads), 0, stream, a);
}

}  // namespace mol
