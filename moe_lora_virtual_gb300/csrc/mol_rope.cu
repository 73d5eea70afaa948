// Rotary positions and the append to a paged cache (include/mol_attn.h).

#include "mol_attend.cuh"
#include "mol_internal.h"

namespace mol {
namespace {

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

// A block per token. Its angles are the same for every head: computed once, one a thread, handed over in
// shared memory. A head is cut into units: a 16-byte chunk or, in the half layout's turned part, a chunk
// and its partner half the turned width on. A thread has one unit of every step-th head (queries, then
// keys), so that its addresses move by a constant; the first one, and the values, are asked for before
// the angles (position, frequency and 64-bit products are a chain of two round trips and some). Bound
// by HBM for many tokens (each value read and written once), by the launch and that chain for a few.
// What keeps HBM busy is bytes under way, so for many tokens a thread's later units are prefetched into L2,
// 14 tokens on a multiprocessor: 8192 tokens of 32 heads of 128, half of each turned, take 24.6 us (0.80 of a
// copy's rate) and 29.0 with keys and values into pages (0.83). Without the prefetch 26.4 and 31.8 with 16
// tokens (32 registers), 28.1 and 34.3 with 12, 33.5 and 41.7 with 64 registers; with it 24.9 and 29.1 with 16,
// 25.5 and 30.4 with 12, 26.3 and 30.9 with 28 blocks of 64 threads. Before it, cosines and four heads in
// registers (72) took 26.4 and 38.3, blocks that stay for several tokens (115) 30.6 and 43.5.
template <int THREADS, int BLOCKS, bool MANY>
__global__ void __launch_bounds__(THREADS, BLOCKS) rope_kernel(const __grid_constant__ RopeArgs a) {
  // Pairs 2 e and 2 e + 1 of unit u at [e * turned + u], so that neighbouring lanes read neighbouring
  // 16 bytes (in the pairs' own order four units share their banks).
  __shared__ float4 cs[kMaxPairs / 2];
  const int64_t t = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const int slot = a.slots ? a.slots[t] : -1;
  const int h0 = divide(threadIdx.x, a.by_units), unit = threadIdx.x - h0 * a.units;
  const int pairs = a.interleaved ? 0 : a.rotary_dim >> 4;  // units that are two chunks
  const bool two = unit < pairs;
  const int u = two ? unit : unit + pairs;                  // its (first) chunk
  const int shift = a.interleaved ? 2 : 3, turned = a.rotary_dim / 2 >> shift;  // pairs of a unit; units
  const int heads = a.in[0].heads + a.in[1].heads;
  const int first = h0 < a.step ? h0 : heads;               // (threads left over have none)
  auto from = [&](int h) {
    const bool key = h >= a.in[0].heads;
    const HeadRows& in = a.in[key];
    return reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(in.x) + t * in.token_stride +
                                          (int64_t)(key ? h - a.in[0].heads : h) * in.head_stride) + u;
  };
  Chunk c, d;
  if (first < heads) {
    c.q = from(first)[0];
    if (two) d.q = from(first)[pairs];
  }
  auto value = [&](int i, int h) {
    return reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.in[2].x) + t * a.in[2].token_stride +
                                          h * a.in[2].head_stride) + i - h * a.chunks;
  };
  if constexpr (MANY) {
    // What the thread asks for later is on its way to L2 at once, which takes no registers.
    auto soon = [](const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); };
#pragma unroll 1
    for (int h = first + a.step; h < heads; h += a.step) {
      soon(from(h));
      if (two) soon(from(h) + pairs);
    }
#pragma unroll 1
    for (int i = threadIdx.x; i < a.in[2].heads * a.chunks; i += THREADS) soon(value(i, divide(i, a.by_chunks)));
  }
  if (a.inv_freq) {
    const int p = a.positions[t];
    for (int i = threadIdx.x; i < a.rotary_dim / 2; i += THREADS) {
      const int in_unit = i & ((1 << shift) - 1);
      reinterpret_cast<float2*>(cs + (in_unit >> 1) * turned + (i >> shift))[in_unit & 1] =
          turn(p, a.inv_freq[i], a.magnitude);
    }
  }
  const bool in = slot >= 0 && slot < a.num_slots;
  const int page = in ? divide(slot, a.by_page) : 0;
  const bool keep = in && MOL_CHECK(slot - page * a.page_size >= 0 && slot - page * a.page_size < a.page_size,
                                    MOL_CHECK_ROW, slot);
  const int64_t cache_at = (int64_t)page * a.page_stride + (int64_t)(slot - page * a.page_size) * a.token_stride;
  if (keep) {
#pragma unroll 1
    for (int i = threadIdx.x; i < a.in[2].heads * a.chunks; i += THREADS) {
      const int h = divide(i, a.by_chunks);
      reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.v_cache) + cache_at + h * a.head_stride)[i - h * a.chunks] =
          *value(i, h);
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int h = first; h < heads; h += a.step) {
    if (h != first) {
      c.q = from(h)[0];
      if (two) d.q = from(h)[pairs];
    }
    if (two) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x0 = bf16_lo(c.w[e]), x1 = bf16_hi(c.w[e]);
        float y0 = bf16_lo(d.w[e]), y1 = bf16_hi(d.w[e]);
        const float4 f = cs[e * turned + u];
        turn_pair(x0, y0, make_float2(f.x, f.y));
        turn_pair(x1, y1, make_float2(f.z, f.w));
        c.w[e] = pack_bf16x2(x0, x1);
        d.w[e] = pack_bf16x2(y0, y1);
      }
    } else if (a.interleaved && u < turned) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 f = cs[e * turned + u];
        float x0 = bf16_lo(c.w[2 * e]), y0 = bf16_hi(c.w[2 * e]);
        float x1 = bf16_lo(c.w[2 * e + 1]), y1 = bf16_hi(c.w[2 * e + 1]);
        turn_pair(x0, y0, make_float2(f.x, f.y));
        turn_pair(x1, y1, make_float2(f.z, f.w));
        c.w[2 * e] = pack_bf16x2(x0, y0);
        c.w[2 * e + 1] = pack_bf16x2(x1, y1);
      }
    }
    uint16_t* dst;
    if (h < a.in[0].heads) {
      dst = static_cast<uint16_t*>(a.q_out) + t * a.q_out_token_stride + h * a.q_out_head_stride;
    } else {
      if (!keep) break;
      dst = static_cast<uint16_t*>(a.k_cache) + cache_at + (h - a.in[0].heads) * a.head_stride;
    }
    reinterpret_cast<uint4*>(dst)[u] = c.q;
    if (two) reinterpret_cast<uint4*>(dst)[u + pairs] = d.q;
  }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& args, cudaStream_t stream) {
  RopeArgs a = args;
  a.chunks = a.head_dim >> 3;
  a.units = a.chunks - (a.interleaved ? 0 : a.rotary_dim >> 4);
  a.by_chunks = divider(a.chunks);
  a.by_units = divider(a.units);
  a.by_page = divider(a.page_size);
  // Many tokens: as many as possible at a time. Few: 256 threads each, registers as they come (23 tokens of
  // 16 heads of 128 1.9 us, 2.1 with keys and values; 2.1 and 2.8 in the form for many).
  auto go = [&](auto kernel, int threads) {
    a.step = threads / a.units;
    return launch_pdl(kernel, dim3((unsigned)a.num_tokens), dim3(threads), 0, stream, a);
  };
  return a.num_tokens > 4 * 152 ? go(rope_kernel<128, 14, true>, 128) : go(rope_kernel<256, 4, false>, 256);
}

cudaError_t take_rope_checks(unsigned long long* first, unsigned long long* count) {
  CheckRecord r;
  const cudaError_t e = take_check_record_here(&r);
  *first = r.first;
  *count = r.count;
  return e;
}

}  // namespace mol
