// The experts of a MoE layer for a few tokens and the 4-bit linear (include/mol_block.h): the
// streaming kernels. One translation unit per weight format instantiates them (mol_moe_*.cu).
//
// Mathematics. Both halves of the experts and the linear are products w . x of weight rows with a
// few activation rows, every weight used by the tokens of its expert only (a few), so the time is
// that of reading the taken experts' weights once: 2 bytes (or about half a byte) for 2 n
// operations at n tokens an expert. 4-bit weights take about 170 instructions a KB to become bf16 and
// be multiplied, which costs the warps more than HBM takes to bring them. Two streaming loops:
//
// - stream_kernel: gate_up, the linear, and down's split form. A block owns tiles of 16 whole weight
//   rows (8 gate and 8 up rows) and a tile belongs to a team of warps, which split its inputs; each
//   warp streams its share of tile after tile through a ring of its own. A lane copies (cp.async) the
//   very 16 bytes that it will read, so nobody signals anybody: a chunk of 2 KB has landed when the
//   lane's own copies have, and three are in flight a warp, 96 KB a block. (Stages of whole tiles,
//   brought by bulk copies, kept shared memory full of tiles that were being multiplied: an output
//   head took 35 us instead of 29.5.) The tokens' rows come by bulk copies into slots that all warps
//   read, from a warp of its own, once for all the block's tiles of an expert. Measured: 23 tokens of
//   128 bf16 experts of 2048 x 768, top 8: both halves in 149 us, 6.3 TB/s, 0.92 of a copy's rate; a
//   4-bit head of 120001 rows of 2048 inputs, 5 tokens: 30.3 us, 4.2 TB/s, where the schedulers issue
//   in 64 % of the cycles and the tensor, ALU and load pipes share them.
// - down_kernel: few pairs, or bf16. A block or cluster owns rows of every expert, and a stage holds a
//   unit's weights and activation rows (bulk copies; rows of a tile are neighbours in memory). A team's
//   first warp asks for the next stage as soon as the team is through with one; its warps have 16 rows
//   each. One kernel, and no partial sums in memory.
// - The product is mma.sync m16n8k16: weight rows are the M side, tokens the N side (8 a tile), so
//   a single token wastes tensor work and no bandwidth. The contraction's order is free as long as
//   both sides agree: each lane takes 8 neighbouring inputs of its row in one 16-byte shared-memory
//   read, for two mma steps. Tokens of a tile are independent columns; lanes of columns past the
//   last token read that token's row again (a broadcast), their products are dropped.
// - 4-bit words become bf16 pairs with a mask and a subtraction that are exact ((128 + q) - 136);
//   a group's products are summed in fp32 first and multiplied by its scale after, so nothing is
//   rounded that fp32 arithmetic would not round. (The subtraction left to a product of the tokens
//   with -136 saves 32 instructions a KB and costs 8 products: 34.5 us for the head.)
// - Work is dealt by weight bytes: the rows of all taken experts form one list that the blocks of
//   stream_kernel share evenly, whatever the routing; the rows of down_kernel are dealt to blocks or
//   clusters, whose blocks split the experts. There a team adds its products into sums of its own in
//   the order of the experts; the teams' and the blocks' sums are added in a fixed order at the end,
//   through distributed shared memory. No atomics on results.
// - Each block groups the (token, slot) pairs by expert itself (at most 1024 of them: match masks,
//   counts in shared memory, one scan; 2 us, or 1 for up to 32 pairs), so the layer is two launches,
//   three in the split form. A block fills its SM (shared memory, registers), so one of the second
//   launch groups the pairs and asks for its first weights as soon as the first launch's block has left
//   its SM, while those of other SMs still run; HBM idles in between for a few microseconds.
// - The first half's values are rounded to bf16 between the halves, in mol_moe_forward too: act is what
//   the adapters' down stage reads, the products take bf16, and it is half the bytes. The second half
//   sums in fp32. This rounding is the whole difference from activations in fp32: relative error 0.0023
//   to 0.0025 instead of the 0.0017 of the output's own rounding.
#pragma once

#include <type_traits>

#include "mol_block.h"
#include "mol_device.cuh"
#include "mol_internal.h"
#include "mol_moe.h"

namespace mol {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kListWarps = kListThreads / 32;
constexpr int kExpertsPerThread = MOL_MOE_MAX_EXPERTS / kListThreads;
constexpr int kPairsPerThread = MOL_MOE_MAX_PAIRS / kListThreads;
constexpr uint32_t kWaitPolls = 1u << 22;

__device__ unsigned int g_moe_fault_flags;
// Test controls of the bounded waits, set only through mol_debug_wait_test.
__device__ unsigned int g_moe_test_stall;
__device__ unsigned long long g_moe_wait_limit_ns = kWaitLimitNs;

// Shared memory by 32-bit address: the loads are then shared loads whatever the compiler can see of
// the pointers, and addresses take one register. Volatile: they stay behind the waits before them.
MOL_DEV uint4 ld_s16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at));
  return v;
}
MOL_DEV uint2 ld_s8(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}
MOL_DEV uint32_t ld_s4(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
MOL_DEV uint32_t ld_s2(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return v;
}
MOL_DEV float ld_sf(uint32_t at) { return __uint_as_float(ld_s4(at)); }
MOL_DEV void st_s4(uint32_t at, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
MOL_DEV void st_sf(uint32_t at, float v) { st_s4(at, __float_as_uint(v)); }
MOL_DEV void st_s16(uint32_t at, float a, float b, float c, float d) {
  asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(at), "f"(a), "f"(b), "f"(c), "f"(d)
               : "memory");
}
MOL_DEV void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// A whole warp's bounded wait. The lanes vote: where the limit passes between two lanes' polls, some
// would see the phase complete and others not, and part ways before the warp's next barrier.
MOL_DEV bool warp_wait(uint64_t* bar, uint32_t parity, unsigned long long limit_ns) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, kWaitPolls, limit_ns));
}

// Tokens of one expert: a tile's columns.
struct Entry {
  int e, off, n;
};

// The pairs grouped by expert, in shared memory.
struct Lists {
  uint32_t order;   // [numel] pair | token << 16, by entry
  uint32_t weight;  // [numel] fp32, of the same pairs (down)
  uint32_t entry;   // pairs of words: expert, first pair | pairs << 16
  int count;        // entries
  bool repeated;    // some token lists an expert twice
  MOL_DEV Entry get(int i) const {
    const uint2 v = ld_s8(entry + 8 * i);
    return Entry{(int)v.x, (int)(v.y & 0xFFFF), (int)(v.y >> 16)};
  }
  MOL_DEV uint32_t pair(int i) const { return ld_s4(order + 4 * i); }
};

// Groups the pairs by expert, in the order of their index: every block finds the same entries, so
// blocks that hold different rows of one expert agree on which entry has which pair. An expert with
// more than xrows pairs (a power of two) takes several entries. `scratch`: 32 E + 4 numel bytes at most,
// free again afterwards. The block waits for nothing but its own ids, and the code is kept short: it
// runs once a launch, from cold instruction caches.
MOL_DEV void build_lists(const StreamArgs& a, Lists& l, char* scratch, bool weights) {
  __shared__ int scan[kListWarps];
  __shared__ int total_shared;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, numel = a.num_tokens * a.topk;
  const int xlog = 31 - __clz(a.xrows);
  if (numel <= 32) {
    // one warp: a lane for each pair, entries in the order of their first pair
    bool again = false;
    if (warp == 0) {
      int e = -1;
      float w = 0.f;
      if (lane < numel) {
        e = ld_cg_i32(a.ids + lane);
        if (weights) w = a.weights[lane];
      }
      if (e >= a.E) e = -1;
      const int tok = lane / a.topk;
      const unsigned same = __match_any_sync(0xffffffffu, e);
      const int n = __popc(same), before = __popc(same & lanemask_lt());
      const bool first = e >= 0 && before == 0;
      const int chunks = (n + a.xrows - 1) >> xlog;
      int at = first ? n | chunks << 16 : 0;
      const int own = at;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += v;
      }
      const int total = __shfl_sync(0xffffffffu, at, 31);
      at -= own;
      const int off = __shfl_sync(0xffffffffu, at, __ffs(same) - 1) & 0xFFFF;
      if (e >= 0) {
        st_s4(l.order + 4 * (off + before), (uint32_t)lane | (uint32_t)tok << 16);
        if (weights) st_sf(l.weight + 4 * (off + before), w);
      }
      if (first)
        for (int c = 0; c < chunks; ++c) {
          st_s4(l.entry + 8 * ((at >> 16) + c), e);
          st_s4(l.entry + 8 * ((at >> 16) + c) + 4,
                (off + (c << xlog)) | min(a.xrows, n - (c << xlog)) << 16);
        }
      // an expert twice at one token: some later lane of the same token and expert
      if (weights) {
        const unsigned mates = __match_any_sync(0xffffffffu, e < 0 ? -1 - lane : e << 8 | tok);
        again = __popc(mates) > 1;
      }
      if (lane == 0) total_shared = total >> 16;
    }
    l.repeated = __syncthreads_or(again);
    l.count = total_shared;
    return;
  }
  // Each warp ranks a contiguous run of pairs with match masks and per-warp counts; the counts are
  // then summed over the warps, one thread to an expert (to two beyond 512 experts).
  const int rounds = (numel + kListThreads - 1) / kListThreads;
  const int used = (numel + rounds * 32 - 1) / (rounds * 32);  // warps that hold pairs
  int* ids = reinterpret_cast<int*>(scratch);
  uint16_t* cnt = reinterpret_cast<uint16_t*>(ids + numel);  // [warp][expert]
  int mine[kPairsPerThread], pos[kPairsPerThread];
  float wt[kPairsPerThread];
  const int first = warp * rounds * 32 + lane;
#pragma unroll
  for (int j = 0; j < kPairsPerThread; ++j) {
    const int i = first + j * 32;
    const bool in = warp < used && j < rounds && i < numel;
    mine[j] = in ? ld_cg_i32(a.ids + i) : -1;
    wt[j] = in && weights ? a.weights[i] : 0.f;
  }
  for (int e = tid; e < (a.E * used + 1) / 2; e += blockDim.x) reinterpret_cast<uint32_t*>(cnt)[e] = 0;
  __syncthreads();
  if (warp < used) {
#pragma unroll
    for (int j = 0; j < kPairsPerThread; ++j) {
      if (j >= rounds) break;
      const int i = first + j * 32;
      if (mine[j] >= a.E) mine[j] = -1;
      if (i < numel) ids[i] = mine[j];
      const unsigned same = __match_any_sync(0xffffffffu, mine[j]);
      const int before = __popc(same & lanemask_lt());
      if (mine[j] >= 0) pos[j] = cnt[warp * a.E + mine[j]] + before;
      __syncwarp();
      if (mine[j] >= 0 && before == 0) cnt[warp * a.E + mine[j]] += (uint16_t)__popc(same);
      __syncwarp();
    }
  }
  __syncthreads();
  // Counts before each warp's pairs, then (count, entries) offsets of the experts in 16 bits each. A
  // thread's experts are neighbours, one where they suffice (all warps' counts are then loaded at
  // once: what this step takes is the latency of its chains).
  const int per = a.E > kListThreads ? kExpertsPerThread : 1;
  int c[kExpertsPerThread], before_warp[kExpertsPerThread][kListWarps], sum = 0;
#pragma unroll
  for (int j = 0; j < kExpertsPerThread; ++j) {
    const int e = tid * per + j;  // (threads past the lists' have none)
    const bool has = j < per && e < a.E && tid < kListThreads;
    c[j] = 0;
#pragma unroll
    for (int w = 0; w < kListWarps; ++w) before_warp[j][w] = has && w < used ? cnt[w * a.E + e] : 0;
#pragma unroll
    for (int w = 0; w < kListWarps; ++w) {
      const int n = before_warp[j][w];
      before_warp[j][w] = c[j];
      c[j] += n;
    }
    sum += c[j] | ((c[j] + a.xrows - 1) >> xlog) << 16;
  }
  int at = sum;  // exclusive sums over the first warps' threads
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at += n;
  }
  if (warp < kListWarps && lane == 31) scan[warp] = at;
  bool again = false;
  if (weights) {
#pragma unroll
    for (int j = 0; j < kPairsPerThread; ++j) {
      const int i = first + j * 32;
      if (mine[j] >= 0)
#pragma unroll 1
        for (int q = i - i % a.topk; q < i; ++q) again |= ids[q] == mine[j];
    }
  }
  l.repeated = __syncthreads_or(again);
  at -= sum;
  int total = 0;
#pragma unroll
  for (int w = 0; w < kListWarps; ++w) {
    if (w < warp) at += scan[w];
    total += scan[w];
  }
#pragma unroll
  for (int j = 0; j < kExpertsPerThread; ++j) {
    const int e = tid * per + j;
    if (c[j] == 0) continue;
    const int off = at & 0xFFFF;
    int idx = at >> 16;
#pragma unroll
    for (int w = 0; w < kListWarps; ++w)
      if (w < used) cnt[w * a.E + e] = (uint16_t)(off + before_warp[j][w]);
#pragma unroll 1
    for (int o = 0; o < c[j]; o += a.xrows, ++idx) {
      if (!MOL_CHECK(idx < numel, MOL_CHECK_SMEM, idx)) continue;
      st_s4(l.entry + 8 * idx, e);
      st_s4(l.entry + 8 * idx + 4, (off + o) | min(a.xrows, c[j] - o) << 16);
    }
    at = idx << 16 | (off + c[j]);
  }
  l.count = total >> 16;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPairsPerThread; ++j) {
    const int i = first + j * 32;
    if (mine[j] >= 0) {
      const int s = cnt[warp * a.E + mine[j]] + pos[j];
      if (!MOL_CHECK(s < numel, MOL_CHECK_SMEM, s)) continue;
      st_s4(l.order + 4 * s, (uint32_t)i | (uint32_t)(i / a.topk) << 16);
      if (weights) st_sf(l.weight + 4 * s, wt[j]);
    }
  }
  __syncthreads();
}

// A warp's place in its work, step after step: every teams-th tile of the block's share (up to hi) of
// the list of output rows (row pairs), in which every entry takes whole tiles; each tile with all its
// k steps.
struct Cursor {
  int pos, hi;         // first position of the tile in the list
  int entry, row, ks;  // row: first row of the tile
  bool valid;

  MOL_DEV void next(const StreamArgs& a) {
    if (++ks < a.ksteps) return;
    ks = 0;
    pos += a.teams * a.tile_rows;
    row += a.teams * a.tile_rows;
    while (row >= a.entry_rows) {
      row -= a.entry_rows;
      ++entry;
    }
    valid = pos < hi;
  }
};

// d += a . b as mma_16816, free to be scheduled among the loads around it; d = a . b.
MOL_DEV void mma_add(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                     uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
MOL_DEV void mma_set(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                     uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Two nibbles at bits 0 and 16 -> bf16 pair q - 8, exact: (v & mask) | 128 as one instruction (the
// compiler makes two of the expression, and the ALU's rate is what 4-bit weights are bound by). The
// constants follow from bf16's 7 bits of fraction: at 128 = 0x4300 their unit is 1, so an integer
// below 128 put there makes 128 + q.
MOL_DEV uint32_t w4_pair(uint32_t v) {
  uint32_t b;
  asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(b) : "r"(v), "r"(0x43004300u));
  const uint32_t c = 0x43084308u;  // 136
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&b),
                             *reinterpret_cast<const __nv_bfloat162*>(&c));
  return *reinterpret_cast<uint32_t*>(&r);
}

// Products of a warp's weight rows with NTC tiles of 8 tokens over the stage's `len` inputs. r0, r1: the
// lane's rows g and g + 8; x: its token's row in each tile (all at the lane's 16 bytes). mma.sync has
// 21 cycles of latency and issues every 8 a sub-partition, and a shared load takes 40: blocks are
// taken U at a time, loads first, and a block's two steps go to two accumulators.
template <int NTC, int NT>
MOL_DEV void multiply_bf16(float (&acc)[NT][4], uint32_t r0, uint32_t r1, const uint32_t (&x)[NT],
                           int len, int t) {
  constexpr int U = NTC == 1 ? 4 : 2;
  const int full = len >> 5;
  float two[NTC][4];
#pragma unroll
  for (int nt = 0; nt < NTC; ++nt) two[nt][0] = two[nt][1] = two[nt][2] = two[nt][3] = 0.f;
  int b = 0;
  for (; b + U <= full; b += U) {
    uint4 a0[U], a1[U], v[U][NTC];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t o = (b + u) * 64;
      a0[u] = ld_s16(r0 + o);
      a1[u] = ld_s16(r1 + o);
#pragma unroll
      for (int nt = 0; nt < NTC; ++nt) v[u][nt] = ld_s16(x[nt] + o);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int nt = 0; nt < NTC; ++nt) {
        mma_add(acc[nt], a0[u].x, a1[u].x, a0[u].y, a1[u].y, v[u][nt].x, v[u][nt].y);
        mma_add(two[nt], a0[u].z, a1[u].z, a0[u].w, a1[u].w, v[u][nt].z, v[u][nt].w);
      }
    }
  }
  // what is left, the last, partial block with it: inputs past len are zeros
#pragma unroll 1
  for (; b * 32 < len; ++b) {
    const bool in = b * 32 + t * 8 < len;
    const uint32_t o = b * 64;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint4 a0 = in ? ld_s16(r0 + o) : zero, a1 = in ? ld_s16(r1 + o) : zero;
#pragma unroll
    for (int nt = 0; nt < NTC; ++nt) {
      const uint4 v = in ? ld_s16(x[nt] + o) : zero;
      mma_add(acc[nt], a0.x, a1.x, a0.y, a1.y, v.x, v.y);
      mma_add(two[nt], a0.z, a1.z, a0.w, a1.w, v.z, v.w);
    }
  }
#pragma unroll
  for (int nt = 0; nt < NTC; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[nt][i] += two[nt][i];
}

// The scales of one row for a block of 128 inputs: bf16 pairs as they lie.
template <int G>
struct Scales {
  uint32_t v[G == 32 ? 2 : 1];
  MOL_DEV void load(uint32_t at) {
    if constexpr (G == 128) {
      v[0] = ld_s2(at);
    } else if constexpr (G == 64) {
      v[0] = ld_s4(at);
    } else {
      const uint2 w = ld_s8(at);
      v[0] = w.x;
      v[1] = w.y;
    }
  }
  MOL_DEV float get(int i) const { return i & 1 ? bf16_hi(v[i >> 1]) : bf16_lo(v[i >> 1]); }
};

// One block of 128 inputs of 4-bit rows, as loaded.
template <int G>
struct BlockW4 {
  uint4 a0, a1;  // rows g and g + 8
  Scales<G> f0, f1;
  MOL_DEV void load(uint32_t r0, uint32_t r1, uint32_t s0, uint32_t s1, int b) {
    a0 = ld_s16(r0 + b * 64);
    a1 = ld_s16(r1 + b * 64);
    f0.load(s0 + b * (256 / G));
    f1.load(s1 + b * (256 / G));
  }
};

// Its products; FULL: all of its inputs are below len.
template <int G, int NTC, int NT, bool FULL>
MOL_DEV void block_w4(float (&acc)[NT][4], const BlockW4<G>& w, const uint32_t (&x)[NT], int b,
                      int len, int t) {
  const uint32_t w0[4] = {w.a0.x, w.a0.y, w.a0.z, w.a0.w};
  const uint32_t w1[4] = {w.a1.x, w.a1.y, w.a1.z, w.a1.w};
  // the tokens' inputs of two words (64 inputs) at a time, all four with one tile: loads first
  constexpr int kAhead = NTC == 1 ? 4 : NTC == 2 ? 2 : 1;
  uint4 v[kAhead][NTC];
  float sum[NTC][4], odd[4];  // one tile and one group: two accumulators, for shorter chains
  constexpr bool kOdd = NTC == 1 && G == 128;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i % kAhead == 0) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const bool in = FULL || b * 128 + (i + u) * 32 + t * 8 < len;  // inputs past len are zeros
#pragma unroll
        for (int nt = 0; nt < NTC; ++nt)
          v[u][nt] = in ? ld_s16(x[nt] + b * 256 + (i + u) * 64) : make_uint4(0, 0, 0, 0);
      }
    }
    uint32_t p0[4], p1[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      p0[j] = w4_pair(w0[i] >> (4 * j));
      p1[j] = w4_pair(w1[i] >> (4 * j));
    }
#pragma unroll
    for (int nt = 0; nt < NTC; ++nt) {
      const uint4& y = v[i % kAhead][nt];
      if (kOdd && i == 1) {
        mma_set(odd, p0[0], p1[0], p0[1], p1[1], y.x, y.y);
        mma_add(odd, p0[2], p1[2], p0[3], p1[3], y.z, y.w);
      } else if (kOdd && i == 3) {
        mma_add(odd, p0[0], p1[0], p0[1], p1[1], y.x, y.y);
        mma_add(odd, p0[2], p1[2], p0[3], p1[3], y.z, y.w);
      } else {
        if (i * 32 % G == 0) mma_set(sum[nt], p0[0], p1[0], p0[1], p1[1], y.x, y.y);
        else mma_add(sum[nt], p0[0], p1[0], p0[1], p1[1], y.x, y.y);
        mma_add(sum[nt], p0[2], p1[2], p0[3], p1[3], y.z, y.w);
      }
    }
    if ((i + 1) * 32 % G == 0) {
      // a group wholly past len holds no weights: its scale may be anything
      const int grp = i * 32 / G;
      const bool has = FULL || b * 128 + grp * G < len;
      const float g0 = has ? w.f0.get(grp) : 0.f, g1 = has ? w.f1.get(grp) : 0.f;
#pragma unroll
      for (int nt = 0; nt < NTC; ++nt) {
        if (kOdd)
#pragma unroll
          for (int j = 0; j < 4; ++j) sum[nt][j] += odd[j];
        acc[nt][0] = fmaf(g0, sum[nt][0], acc[nt][0]);
        acc[nt][1] = fmaf(g0, sum[nt][1], acc[nt][1]);
        acc[nt][2] = fmaf(g1, sum[nt][2], acc[nt][2]);
        acc[nt][3] = fmaf(g1, sum[nt][3], acc[nt][3]);
      }
    }
  }
}

template <int G, int NTC, int NT>
MOL_DEV void multiply_w4(float (&acc)[NT][4], uint32_t r0, uint32_t r1, uint32_t s0, uint32_t s1,
                         const uint32_t (&x)[NT], int len, int t) {
  const int full = len >> 7;
#pragma unroll 1
  for (int b = 0; b < full; ++b) {
    BlockW4<G> w;
    w.load(r0, r1, s0, s1, b);
    block_w4<G, NTC, NT, true>(acc, w, x, b, len, t);
  }
  if (len & 127) {
    BlockW4<G> w;
    w.load(r0, r1, s0, s1, full);
    block_w4<G, NTC, NT, false>(acc, w, x, full, len, t);
  }
}

MOL_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
MOL_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
MOL_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
// A float into the same shared-memory address of another block of the cluster.
MOL_DEV void remote_store(uint32_t at, uint32_t rank, float v) {
  uint32_t p;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(at), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(p), "f"(v) : "memory");
}

// Adds column `col`'s values of rows `row` and row + 8 times its pair's weight into the sums.
MOL_DEV void add_sums(const StreamArgs& a, const Lists& l, uint32_t sums, const Entry& en, int col,
                      int row, int rows, float v0, float v1) {
  if (col >= en.n) return;
  const int tok = l.pair(en.off + col) >> 16;
  const float w = ld_sf(l.weight + 4 * (en.off + col));
  if (!MOL_CHECK(tok < a.num_tokens && rows <= a.acc_stride, MOL_CHECK_SMEM, tok)) return;
  const uint32_t s = sums + 4 * (tok * a.acc_stride + row);
  if (row < rows) st_sf(s, fmaf(w, v0, ld_sf(s)));
  if (row + 8 < rows) st_sf(s + 32, fmaf(w, v1, ld_sf(s + 32)));
}

// down: where row j of span q lies in a stage, and its scales. Spans of 8 rows are brought by a copy
// each, 64 bytes apart, and the lanes of odd g take the row of the odd span first: the eight lanes of a
// shared-memory phase then read two rows that lie an odd multiple of 64 bytes apart (rows of a multiple
// of 128 bytes) and no bank twice.
MOL_DEV uint32_t row_at(const StreamArgs& a, int q, int j) {
  return (q * 8 + j) * a.row_pitch + q * a.span_shift;
}
MOL_DEV uint32_t scale_at(const StreamArgs& a, int q, int j) {
  return a.scale_off + (q * 8 + j) * a.scale_pitch + q * 16;
}

// The part'th of `parts` nearly equal shares of [0, all).
MOL_DEV void share(int all, int parts, int part, int& from, int& to) {
  const int q = all / parts, r = all - q * parts;
  from = q * part + min(part, r);
  to = from + q + (part < r);
}

// v + the deltas of token tok's pairs at output column n, in the order of the slots; four loads in
// flight at once (an absent pair's delta is read and not used).
MOL_DEV float add_deltas(const StreamArgs& a, float v, int tok, int n) {
  constexpr int U = 4;
  for (int k0 = 0; k0 < a.topk; k0 += U) {
    float d[U], w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t pair = tok * a.topk + min(k0 + u, a.topk - 1);
      const int e = a.ids[pair];
      const bool has = k0 + u < a.topk && e >= 0 && e < a.E;
      const float x = __bfloat162float(a.delta[pair * a.delta_stride + n]), y = a.weights[pair];
      d[u] = has ? x : 0.f;
      w[u] = has ? y : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) v = fmaf(w[u], d[u], v);
  }
  return v;
}

// The bytes of some rows' scales, [at, at + len) of the tensor (4-byte aligned), for a bulk copy to a
// 16-byte aligned place: whole 16-byte units from `from` on. At the end of the tensor the last unit
// may not be there in full: its words are then copied one by one (`tail`).
struct ScaleRange {
  int64_t from;
  uint32_t bytes;
  bool tail;
  MOL_DEV ScaleRange(int64_t at, uint32_t len, int64_t total) {
    const uint32_t mis = (uint32_t)at & 15u;
    from = at - mis;
    bytes = (mis + len + 15u) & ~15u;
    tail = from + bytes > total;
    if (tail) bytes = (uint32_t)(max(from, total & ~(int64_t)15) - from);
  }
  MOL_DEV void copy_tail(const void* scales, uint32_t dst, int64_t at, uint32_t len) const {
    for (int64_t b = max(from + bytes, at); b < at + len; b += 4)
      st_s4(dst + (uint32_t)(b - from),
            *reinterpret_cast<const uint32_t*>(static_cast<const char*>(scales) + b));
  }
};

// Asynchronous copies of a lane, complete in the order of its groups. The first reads `bytes` of the 16
// (0 or 16) and fills the rest with zeros; WIDE: L2 brings the 256 bytes around (bf16 rows: 1 % of the
// time of a memory-bound layer less, 4-bit rows 1 % more).
template <bool WIDE>
MOL_DEV void copy16(uint32_t dst, const char* src, uint32_t bytes) {
  if constexpr (WIDE)
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(bytes)
                 : "memory");
  else
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
template <int BYTES>
MOL_DEV void copy_small(uint32_t dst, const char* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES)
                 : "memory");
}

// gate_up: act[pair, n] = silu(gate) * up, gate = w[e, n] . x[token] (+ delta), up = w[e, N + n] . x[token]
// (+ delta); kPairs: partial[pair, n] = w[e, n] . x[pair]; linear: out[t, n] = w[n] . x[t], its tokens in
// entries of one expert. Few tokens: bound by the launch, the lists and one round trip to HBM (about
// 4 us); many weights: bf16 by HBM, 4-bit by the warps' instructions.
template <int G, int MODE, int NT>
__global__ void __launch_bounds__(consumer_warps(NT) * 32 + 32, 1)
    stream_kernel(const __grid_constant__ StreamArgs a) {
  constexpr bool kW4 = G != 0;
  constexpr int GG = kW4 ? G : 32;  // (a group for code that bf16 does not reach)
  constexpr int kInputs = kW4 ? 256 : 64;  // of a chunk
  constexpr int kChunk = chunk_bytes(G);
  extern __shared__ __align__(128) char smem[];
  __shared__ uint64_t xfull[2], xempty[2];  // a token slot has landed, is free
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int numel = a.num_tokens * a.topk;
  const int consumers = a.teams * a.parts;
  const int rows_per_expert = MODE == kGateUp ? 2 * a.N : a.N;

  // shared memory: rings | token slots | sums of a team's warps | lists
  const uint32_t rings = smem_u32(smem);
  const uint32_t xslots = rings + consumer_warps(NT) * a.chunks * kChunk;
  const uint32_t sums = xslots + a.xstages * a.xslot_bytes;
  Lists lists;
  lists.entry = sums + a.teams * (a.parts - 1) * NT * 512;
  lists.order = lists.entry + (MODE == kLinear ? 0 : numel * 8);
  lists.weight = 0;
  lists.count = (a.num_tokens + a.xrows - 1) / a.xrows;  // (linear: entries of its tokens in order)
  lists.repeated = false;

  if (warp == consumer_warps(NT)) {
    for (int s = lane; s < a.xstages; s += 32) {
      mbar_init(&xfull[s], 1);
      mbar_init(&xempty[s], consumers);
    }
    fence_mbar_init();
  }
  // kPairs after this call's gate_up: only the tokens' rows are its work, the lists and the weights
  // need not wait for it
  const bool late = MODE == kPairs && a.chained;
  if (!late) pdl_wait();
  pdl_launch_dependents();
  if (MODE != kLinear) {
    build_lists(a, lists, smem, false);
    // the lists' scratch becomes rings and token slots: ordinary accesses before the copies
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  auto entry_of = [&](int i) {
    if (MODE == kLinear) return Entry{0, i * a.xrows, min(a.xrows, a.num_tokens - i * a.xrows)};
    return lists.get(i);
  };

  // this block's share: whole tiles, in pieces: groups of a tile for each team, which share the
  // tokens' pieces
  const bool whole = a.ksteps == 1;
  const int step = a.tile_rows * (whole ? 1 : a.teams);
  int lo, hi;
  share(lists.count * (a.entry_rows / step), gridDim.x, blockIdx.x, lo, hi);
  lo *= step;
  hi *= step;
  // Token slots in the order of their use: whole rows: one for each entry of the share; pieces: one
  // for each k step of each group of tiles.
  const int entry0 = lo / a.entry_rows;
  const int slots = lo >= hi ? 0
                    : whole  ? (hi - 1) / a.entry_rows - entry0 + 1
                             : (hi - lo) / step * a.ksteps;
  __syncthreads();
  const unsigned long long limit = g_moe_wait_limit_ns;
  bool fault = false;

  if (warp == consumer_warps(NT)) {
    // ---- the tokens' rows ----
    if (late) pdl_wait();
    if (!(g_moe_test_stall & 1)) {
      int entry = entry0, ks = 0;
      int left = a.entry_rows - (lo - entry0 * a.entry_rows);  // pieces: rows of the entry to come
      int i = 0, s = 0, use = 0;
      for (; i < slots; ++i) {
        if (use > 0 && !warp_wait(&xempty[s], (use - 1) & 1, limit)) {
          fault = true;
          break;
        }
        const Entry en = entry_of(entry);
        const int k0 = ks * a.Kc, len = min(a.Kc, a.K - k0);
        if (lane == 0) mbar_arrive_expect_tx(&xfull[s], (uint32_t)en.n * len * 2);
        __syncwarp();
        for (int j = lane; j < en.n; j += 32) {
          int row = en.off + j;
          if (MODE == kGateUp) row = lists.pair(en.off + j) >> 16;
          if (MODE == kPairs) row = lists.pair(en.off + j) & 0xFFFF;
          if (!MOL_CHECK(row < (MODE == kPairs ? numel : a.num_tokens), MOL_CHECK_ROW, row)) row = 0;
          bulk_copy(xslots + s * a.xslot_bytes + j * a.x_pitch, a.x + row * a.x_stride + k0, len * 2,
                    &xfull[s]);
        }
        // the next slot, its entry and k step
        if (++s == a.xstages) {
          s = 0;
          ++use;
        }
        if (++ks == a.ksteps) {
          ks = 0;
          if (!whole) left -= step;
          if (whole || left == 0) {
            left = a.entry_rows;
            ++entry;
          }
        }
      }
      // no copy may be in flight when the block leaves
      if (fault)
        for (int q = max(0, i - a.xstages); q < i; ++q)
          (void)warp_wait(&xfull[q % a.xstages], (q / a.xstages) & 1, limit);
    }
  } else if (slots > 0 && warp < consumers) {
    // ---- consumers ----
    const int g = lane >> 2, t = lane & 3;
    // (a team's warps are neighbours, so that they run on different sub-partitions)
    const int parts = a.parts, team = warp / parts, part = warp - team * parts;
    const int64_t spitch = kW4 ? w4_padded(a.K) / GG * 2 : 0;
    const int64_t pitch = kW4 ? w4_padded(a.K) / 2 : a.K * 2;
    Cursor cur;
    cur.hi = hi;
    cur.pos = lo + team * a.tile_rows;
    cur.entry = entry0;
    cur.row = cur.pos - entry0 * a.entry_rows;
    while (cur.row >= a.entry_rows) {
      cur.row -= a.entry_rows;
      ++cur.entry;
    }
    cur.ks = 0;
    cur.valid = cur.pos < hi;
    // chunks of a tile's step; none in a tile that only fills up a group
    auto chunks_of = [&](const Cursor& c) {
      return c.row >= a.N ? 0 : (min(a.Kc, a.K - c.ks * a.Kc) + kInputs - 1) / kInputs;
    };

    // The warp's weights, chunk after chunk of its tiles, asked for a.chunks - 1 ahead of their use.
    // Every lane copies what it reads itself (its rows' 16 bytes of each block), so a chunk has
    // landed when the lane's own copies have; scales: a lane for each row.
    const uint32_t ring = rings + warp * a.chunks * kChunk;
    const int last_slot = a.chunks - 1;  // (a power of two less one)
    Cursor ahead = cur;
    int next = part, count = 0;  // chunk of ahead's step, how many it has
    const char *w0 = nullptr, *w1 = nullptr, *ws = nullptr;
    int left = 0;  // bytes of the step's row from the lane's place on (bf16)
    const int64_t tile_bytes = a.teams * a.tile_rows * pitch;
    const int tile_scales = a.teams * a.tile_rows * (int)spitch;
    auto aim = [&]() {
      const int rows = min(a.tile_rows, a.N - ahead.row), k0 = ahead.ks * a.Kc;
      const int64_t first = (int64_t)entry_of(ahead.entry).e * rows_per_expert + ahead.row;
      // rows past the tile's last: that row again
      int64_t r0 = first + min(g, rows - 1);
      int64_t r1 = MODE == kGateUp ? r0 + a.N : first + min(g + 8, rows - 1);
      if (!MOL_CHECK(r1 < (int64_t)a.E * rows_per_expert, MOL_CHECK_WEIGHT_ROW, r1)) r0 = r1 = 0;
      const int64_t o = (kW4 ? k0 / 2 : k0 * 2) + t * 16;
      w0 = a.w + r0 * pitch + o;
      w1 = a.w + r1 * pitch + o;
      if (kW4) ws = reinterpret_cast<const char*>(a.scales) + (t & 1 ? r1 : r0) * spitch + k0 / GG * 2;
      else left = min(a.Kc, a.K - k0) * 2 - t * 16;
    };
    // the next step that has chunks for this warp
    auto advance = [&]() {
      const int entry = ahead.entry, ks = ahead.ks, pos = ahead.pos;
      do {
        ahead.next(a);
        next = part;
      } while (ahead.valid && next >= (count = chunks_of(ahead)));
      if (!ahead.valid) return;
      if (whole && ahead.entry == entry && ahead.row + a.tile_rows <= a.N) {
        w0 += tile_bytes;
        w1 += tile_bytes;
        if (kW4) ws += tile_scales;
      } else if (ahead.pos == pos) {
        const int k = (ahead.ks - ks) * a.Kc;
        w0 += kW4 ? k / 2 : k * 2;
        w1 += kW4 ? k / 2 : k * 2;
        if (kW4) ws += k / GG * 2;
        else left = min(a.Kc, a.K - ahead.ks * a.Kc) * 2 - t * 16;
      } else {
        aim();
      }
    };
    auto fetch = [&](int slot) {
      if (ahead.valid) {
        const uint32_t dst = ring + slot * kChunk + lane * 16;
        const int o = next * 128;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const bool in = kW4 || o + u * 64 < left;  // past the row: zeros
          copy16<!kW4>(dst + u * 512, in ? w0 + o + u * 64 : a.w, in ? 16 : 0);
          copy16<!kW4>(dst + 1024 + u * 512, in ? w1 + o + u * 64 : a.w, in ? 16 : 0);
        }
        if (kW4 && t < 2)
          copy_small<512 / GG>(ring + slot * kChunk + 2048 + (t * 8 + g) * (512 / GG),
                               ws + next * (512 / GG));
        next += parts;
        if (next >= count) advance();
      }
      cp_async_commit();
    };
    if (ahead.valid) {
      if (next < (count = chunks_of(ahead))) aim();
      else advance();
    }
    for (int i = 0; i < last_slot; ++i) fetch(i);

    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    int slot = 0, have = -1, finisher = 0;
    int xi = -1, xs = -1, xphase = 0;  // token slots so far, the newest one's place and phase
    auto next_tokens = [&]() {         // releases the token slot in use and waits for the next
      if (xi >= 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&xempty[xs]);
      }
      if (++xs == a.xstages) {
        xs = 0;
        xphase ^= 1;
      }
      if (++xi < slots) fault = !warp_wait(&xfull[xs], xphase, limit);
    };
    int want = 0;  // the token slot of this step
    Entry en{0, 0, 0};
    uint32_t x[NT];  // the lane's token row of each tile
    // After a fault nothing is read or written any more, but the team's warps still meet.
    for (; cur.valid; cur.next(a)) {
      if (whole) want = cur.entry - entry0;
      if (!fault && (xi < want || cur.entry != have)) {
        while (xi < want && !fault) next_tokens();  // (those passed over are released in their order)
        have = cur.entry;
        en = entry_of(have);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          x[nt] = xslots + xs * a.xslot_bytes + min(g + 8 * nt, en.n - 1) * a.x_pitch + t * 16;
      }
      ++want;
      const int chunks = fault ? 0 : chunks_of(cur), len = min(a.Kc, a.K - cur.ks * a.Kc);
      // the deltas of the tile's values, asked for before its chunks
      const int rows = fault ? 0 : min(a.tile_rows, a.N - cur.row);
      uint16_t delta[MODE == kGateUp ? NT : 1][2][2];
      if constexpr (MODE == kGateUp) {
        if (a.delta && cur.ks == a.ksteps - 1) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int col = nt * 8 + 2 * t + h;
              delta[nt][h][0] = delta[nt][h][1] = 0;
              if (col >= en.n || g >= rows) continue;
              const int64_t pair = lists.pair(en.off + col) & 0xFFFF;
              if (!MOL_CHECK(pair < numel, MOL_CHECK_ROW, pair)) continue;
              const uint16_t* dl =
                  reinterpret_cast<const uint16_t*>(a.delta) + pair * a.delta_stride + cur.row + g;
              delta[nt][h][0] = dl[0];
              delta[nt][h][1] = dl[a.N];
            }
          }
        }
      }
#pragma unroll 1
      for (int c = part; c < chunks; c += parts) {
        if (last_slot == kChunks - 1) cp_async_wait_group<kChunks - 2>();
        else cp_async_wait_group<0>();
        __syncwarp();  // the row's scales have landed too; the chunk before has been read by all
        fetch((slot + last_slot) & last_slot);
        const uint32_t st = ring + slot * kChunk;
        slot = (slot + 1) & last_slot;
        auto multiply = [&](auto tiles) {
          constexpr int NTC = decltype(tiles)::value;
          if constexpr (kW4) {
            auto block = [&](int u, auto full) {
              BlockW4<GG> w;
              w.a0 = ld_s16(st + u * 512 + lane * 16);
              w.a1 = ld_s16(st + 1024 + u * 512 + lane * 16);
              w.f0.load(st + 2048 + g * (512 / GG) + u * (256 / GG));
              w.f1.load(st + 2048 + (8 + g) * (512 / GG) + u * (256 / GG));
              block_w4<GG, NTC, NT, decltype(full)::value>(acc, w, x, c * 2 + u, len, t);
            };
            if ((c + 1) * 256 <= len) {
              block(0, std::true_type{});
              block(1, std::true_type{});
            } else {
#pragma unroll 1
              for (int u = 0; u < 2; ++u) block(u, std::false_type{});
            }
          } else {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int b = c * 2 + u;
              const uint4 a0 = ld_s16(st + u * 512 + lane * 16);
              const uint4 a1 = ld_s16(st + 1024 + u * 512 + lane * 16);
              const bool in = b * 32 + t * 8 < len;  // inputs past len are zeros
#pragma unroll
              for (int nt = 0; nt < NTC; ++nt) {
                const uint4 v = in ? ld_s16(x[nt] + b * 64) : make_uint4(0, 0, 0, 0);
                mma_add(acc[nt], a0.x, a1.x, a0.y, a1.y, v.x, v.y);
                mma_add(acc[nt], a0.z, a1.z, a0.w, a1.w, v.z, v.w);
              }
            }
          }
        };
        if (NT > 1 && en.n <= 8) multiply(std::integral_constant<int, 1>{});
        else multiply(std::integral_constant<int, NT>{});
      }
      if (cur.ks < a.ksteps - 1) continue;

      // The warps of a team take turns in adding the others' sums and finishing.
      if (parts > 1) {
        const bool mine = part == finisher;
        auto place = [&](int p) {
          return sums + (team * (parts - 1) + p - (p > finisher)) * NT * 512 + lane * 16;
        };
        named_sync(1 + team, parts * 32);  // (the tile before has been added)
        if (!mine) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            st_s16(place(part) + nt * 512, acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
        }
        named_sync(1 + team, parts * 32);
        if (mine) {
          for (int p = 0; p < parts; ++p) {
            if (p == part) continue;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint4 v = ld_s16(place(p) + nt * 512);
              acc[nt][0] += __uint_as_float(v.x);
              acc[nt][1] += __uint_as_float(v.y);
              acc[nt][2] += __uint_as_float(v.z);
              acc[nt][3] += __uint_as_float(v.w);
            }
          }
        }
        finisher = finisher + 1 == parts ? 0 : finisher + 1;
        if (!mine) {
#pragma unroll
          for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
          continue;
        }
      }
      // the tile's values: column 2t + h of each token tile; row g of the first eight in values h, of
      // the second (gate_up: the up row) in values 2 + h
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int col = nt * 8 + 2 * t + h, n = cur.row + g;
          float v0 = acc[nt][h], v1 = acc[nt][2 + h];
          if (col >= en.n || g >= rows) continue;
          if constexpr (MODE == kGateUp) {
            const int64_t pair = lists.pair(en.off + col) & 0xFFFF;
            if (!MOL_CHECK(pair < numel && n < a.N, MOL_CHECK_ROW, pair)) continue;
            if (a.delta) {
              v0 += __uint_as_float((uint32_t)delta[nt][h][0] << 16);
              v1 += __uint_as_float((uint32_t)delta[nt][h][1] << 16);
            }
            a.out[pair * a.N + n] = __float2bfloat16(v0 / (1.f + expf(-v0)) * v1);
          } else if (MODE == kPairs) {
            const int64_t pair = lists.pair(en.off + col) & 0xFFFF;
            if (!MOL_CHECK(pair < numel && cur.row + rows <= a.N, MOL_CHECK_ROW, pair)) continue;
            float* o = a.partial + pair * a.N + n;
            o[0] = v0;
            if (g + 8 < rows) o[8] = v1;
          } else {
            if (!MOL_CHECK(cur.row + rows <= a.N, MOL_CHECK_COLUMN, cur.row)) continue;
            bf16* o = a.out + (en.off + col) * a.out_stride + n;
            o[0] = __float2bfloat16(v0);
            if (g + 8 < rows) o[8] = __float2bfloat16(v1);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    }
    // the token slots that are left, for the warps that still need them to be refilled
    while (!fault && xi < slots) next_tokens();
    if (fault) cp_async_wait_all();  // no copy may be in flight when the block leaves
  }
  if (fault && lane == 0) atomicOr(&g_moe_fault_flags, kFaultBulkTimeout);
}

// out[t] = sum of weight * (w[e] . act[pair]) over t's pairs. A cluster (or one block) has up to 64
// output rows of every expert; its blocks split the (entry, k step) units. A unit is one stage of a
// team: the rows' weights, contiguous in memory, and the entry's activation rows. The warps of a team
// have 16 rows each. A team adds its products into sums of its own, unit after unit; the teams' and
// then the blocks' sums are added in their order.
template <int G, int NT>
__global__ void __launch_bounds__(kBlockWarps * 32, 1) down_kernel(const __grid_constant__ StreamArgs a) {
  constexpr bool kW4 = G != 0;
  constexpr int GG = kW4 ? G : 32;
  extern __shared__ __align__(128) char smem[];
  __shared__ uint64_t wfull[kMaxStages], pfull[kMaxStages];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int numel = a.num_tokens * a.topk;
  const int parts = a.parts, team = warp / parts, part = warp - team * parts;

  // shared memory: stages | sums of each team | sums from the cluster's blocks | lists
  const uint32_t ring = smem_u32(smem);
  const uint32_t all_sums = ring + a.stages * a.stage_bytes;
  const uint32_t copy_bytes = a.num_tokens * a.acc_stride * 4;
  const uint32_t received = all_sums + a.teams * copy_bytes;
  Lists lists;
  const int each = (a.num_tokens + a.cluster - 1) / a.cluster;  // tokens a block adds at most
  lists.entry = received + (a.cluster > 1 ? each * a.cluster * a.acc_stride * 4 : 0);
  lists.order = lists.entry + numel * 8;
  lists.weight = lists.order + numel * 4;

  if (warp == (int)(blockDim.x >> 5) - 1) {
    for (int s = lane; s < a.stages; s += 32) {
      mbar_init(&wfull[s], 1);
      mbar_init(&pfull[s], max(1, parts - 1));
    }
    fence_mbar_init();
  }
  if (!a.chained) {
    pdl_wait();
    pdl_launch_dependents();
  }
  const int ranks = a.cluster, rank = ranks > 1 ? (int)cluster_rank() : 0;
  if (ranks > 1) cluster_arrive();  // (waited for before the first access to another block)
  build_lists(a, lists, smem, true);
  // the scratch becomes the ring and the teams' sums (which are zeroed below, not before)
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  int first_row, end_row, lo, hi;
  share(a.N, gridDim.x / ranks, blockIdx.x / ranks, first_row, end_row);
  share(lists.count * a.ksteps, ranks, rank, lo, hi);
  const int rows = end_row - first_row;
  for (int i = tid; i < a.teams * (int)copy_bytes / 4; i += blockDim.x) st_s4(all_sums + 4 * i, 0u);
  __syncthreads();
  const unsigned long long limit = g_moe_wait_limit_ns;
  bool fault = false;

  if (team < a.teams && rows > 0) {
    const int g = lane >> 2, t = lane & 3;
    const int depth = a.stages / a.teams;
    const uint32_t my_ring = ring + team * depth * a.stage_bytes;
    uint64_t* my_full = wfull + team * depth;
    uint64_t* my_pfull = pfull + team * depth;
    const int spitch = kW4 ? w4_padded(a.K) / GG * 2 : 0;
    const int pitch = kW4 ? w4_padded(a.K) / 2 : a.K * 2;
    const int64_t stotal = kW4 ? (int64_t)a.E * a.N * spitch : 0;

    // Asks for a unit's weights and announces its activation rows as well: the team's first warp.
    auto put_weights = [&](int unit, int slot) {
      const int entry = unit / a.ksteps, ks = unit - entry * a.ksteps;
      const Entry en = lists.get(entry);
      const uint32_t dst = my_ring + slot * a.stage_bytes;
      uint64_t* bar = &my_full[slot];
      const int k0 = ks * a.Kc, len = min(a.Kc, a.K - k0);
      const int row0 = en.e * a.N + first_row;
      // a copy for each span of 8 rows, or for each row
      const int copies = a.row_copies ? rows : (rows + 7) / 8;
      auto each = [&](auto f) {
        for (int c = lane; c < copies; c += 32) {
          const int q = a.row_copies ? c >> 3 : c, j = a.row_copies ? c & 7 : 0;
          const int per = a.row_copies ? 1 : min(8, rows - 8 * q);
          const int row = row0 + 8 * q + j;
          if (!MOL_CHECK(row + per <= a.E * a.N, MOL_CHECK_WEIGHT_ROW, row)) continue;
          const uint32_t size = a.row_copies ? (kW4 ? (len + 127) / 128 * 64 : len * 2) : per * pitch;
          const uint32_t slen = !kW4 ? 0 : a.row_copies ? (len + GG - 1) / GG * 2 : per * spitch;
          f(q, j, row, size, slen, kW4 ? (int64_t)row * spitch + k0 / GG * 2 : 0);
        }
      };
      uint32_t bytes = 0;
      each([&](int q, int j, int row, uint32_t size, uint32_t slen, int64_t at) {
        bytes += size;
        if (kW4) {
          const ScaleRange sr(at, slen, stotal);
          bytes += sr.bytes;
          if (sr.tail) sr.copy_tail(a.scales, dst + scale_at(a, q, j), at, slen);
        }
      });
      bytes = __reduce_add_sync(0xffffffffu, bytes);
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(bar, bytes + en.n * len * 2);
      __syncwarp();
      each([&](int q, int j, int row, uint32_t size, uint32_t slen, int64_t at) {
        bulk_copy(dst + row_at(a, q, j), a.w + (int64_t)row * pitch + (kW4 ? k0 / 2 : k0 * 2), size,
                  bar);
        if (kW4) {
          const ScaleRange sr(at, slen, stotal);
          if (sr.bytes)
            bulk_copy(dst + scale_at(a, q, j), reinterpret_cast<const char*>(a.scales) + sr.from,
                      sr.bytes, bar);
        }
      });
    };
    auto put_x = [&](int unit, int slot) {
      const int entry = unit / a.ksteps, ks = unit - entry * a.ksteps;
      const Entry en = lists.get(entry);
      const int k0 = ks * a.Kc, len = min(a.Kc, a.K - k0);
      for (int j = lane; j < en.n; j += 32) {
        int pair = lists.pair(en.off + j) & 0xFFFF;
        if (!MOL_CHECK(pair < numel, MOL_CHECK_ROW, pair)) pair = 0;
        bulk_copy(my_ring + slot * a.stage_bytes + a.x_off + j * a.x_pitch,
                  a.x + pair * a.x_stride + k0, len * 2, &my_full[slot]);
      }
    };
    int filled = 0;  // first warp: stages asked for and not consumed
    if (part == 0 && !(g_moe_test_stall & 1)) {
      for (int u = lo + team; u < hi && filled < depth; u += a.teams) put_weights(u, filled++);
      if (a.chained) {  // the rows that the kernel before writes
        pdl_wait();
        pdl_launch_dependents();
      }
      for (int i = 0; i < filled; ++i) put_x(lo + team + i * a.teams, i);
    }
    const uint32_t sums = all_sums + team * copy_bytes;
    const int my_row = part * 16;
    int slot = 0, phase = 0;
    for (int unit = lo + team; unit < hi; unit += a.teams) {
      fault = !warp_wait(&my_full[slot], phase, limit);
      if (fault) break;
      const int entry = unit / a.ksteps, ks = unit - entry * a.ksteps;
      const Entry en = lists.get(entry);
      const uint32_t st = my_ring + slot * a.stage_bytes;
      const int k0 = ks * a.Kc, len = min(a.Kc, a.K - k0);
      float acc[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
      // the lane's rows of the warp's two spans, that of the odd span first where g is odd; rows past
      // the block's last read that row again, their products are dropped
      const int i0 = min(my_row + (g & 1) * 8 + g, rows - 1);
      const int i1 = min(my_row + (g & 1 ? 0 : 8) + g, rows - 1);
      uint32_t x[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        x[nt] = st + a.x_off + min(g + 8 * nt, en.n - 1) * a.x_pitch + t * 16;
      const uint32_t r0 = st + row_at(a, i0 >> 3, i0 & 7) + t * 16;
      const uint32_t r1 = st + row_at(a, i1 >> 3, i1 & 7) + t * 16;
      if constexpr (kW4) {
        // the copy that brought a row's scales began at the 16 bytes' boundary at or before them, or
        // before those of its span's first row
        auto scales_of = [&](int i) {
          const uint32_t from = en.e * a.N + first_row + (a.row_copies ? i : i & ~7);
          return st + scale_at(a, i >> 3, i & 7) + ((from * spitch + k0 / GG * 2) & 15u);
        };
        if (NT > 1 && en.n <= 8)
          multiply_w4<GG, 1, NT>(acc, r0, r1, scales_of(i0), scales_of(i1), x, len, t);
        else
          multiply_w4<GG, NT, NT>(acc, r0, r1, scales_of(i0), scales_of(i1), x, len, t);
      } else {
        if (NT > 1 && en.n <= 8) multiply_bf16<1, NT>(acc, r0, r1, x, len, t);
        else multiply_bf16<NT, NT>(acc, r0, r1, x, len, t);
      }
      __syncwarp();
      if (parts > 1) {
        if (part > 0) {
          if (lane == 0) mbar_arrive(&my_pfull[slot]);
        } else {
          fault = !warp_wait(&my_pfull[slot], phase, limit);
          if (fault) break;
        }
      }
      if (part == 0) {  // the team is through with the stage: the next one into its place
        const int next = unit + depth * a.teams;
        if (next < hi) {
          put_weights(next, slot);
          put_x(next, slot);
        } else {
          --filled;
        }
      }
      if (++slot == depth) {
        slot = 0;
        phase ^= 1;
      }
      // column 2t + h of each token tile: rows my_row + g and + 8 + g, in values h and 2 + h, the
      // other way round where g is odd. Columns of one step may hold the same token where a token
      // lists its expert twice: they take turns.
      for (int turn = 0; turn < (lists.repeated ? 4 : 1); ++turn) {
        if (!lists.repeated || t == turn) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              add_sums(a, lists, sums, en, nt * 8 + 2 * t + h, my_row + g, rows,
                       g & 1 ? acc[nt][2 + h] : acc[nt][h], g & 1 ? acc[nt][h] : acc[nt][2 + h]);
        }
        __syncwarp();
      }
    }
    // no copy may be in flight when the block leaves
    if (fault && part == 0)
      for (int q = 0; q < filled; ++q) {
        (void)warp_wait(&my_full[slot], phase, limit);
        if (++slot == depth) {
          slot = 0;
          phase ^= 1;
        }
      }
  }
  if (fault && lane == 0) atomicOr(&g_moe_fault_flags, kFaultBulkTimeout);

  // The teams' sums in their order; with a cluster each block adds the blocks' sums of its share of
  // the tokens, sent to it, in the order of their ranks. Then the deltas and one rounding.
  if (a.chained) pdl_wait();
  __syncthreads();
  auto finish = [&](int tok, int row, float v) {
    if (a.delta) v = add_deltas(a, v, tok, first_row + row);
    if (MOL_CHECK(first_row + row < a.N, MOL_CHECK_COLUMN, first_row + row))
      a.out[tok * a.out_stride + first_row + row] = __float2bfloat16(v);
  };
  const int total = rows * a.num_tokens;
  if (ranks > 1) cluster_wait();
  for (int i = tid; i < total; i += blockDim.x) {
    const int tok = i / rows, row = i - tok * rows;
    const uint32_t at = 4 * (tok * a.acc_stride + row);
    float v = 0.f;
    for (int c = 0; c < a.teams; ++c) v += ld_sf(all_sums + c * copy_bytes + at);
    if (ranks == 1) {
      finish(tok, row, v);
    } else {  // to the block that adds the token
      remote_store(received + 4 * ((rank * each + tok / ranks) * rows + row), tok % ranks, v);
    }
  }
  if (ranks > 1) {
    cluster_arrive();
    cluster_wait();
    const int mine = (a.num_tokens - rank + ranks - 1) / ranks;  // tokens rank, rank + ranks, ...
    for (int i = tid; i < mine * rows; i += blockDim.x) {
      const int slot_tok = i / rows, row = i - slot_tok * rows;
      float v = 0.f;
      for (int q = 0; q < ranks; ++q) v += ld_sf(received + 4 * ((q * each + slot_tok) * rows + row));
      finish(slot_tok * ranks + rank, row, v);
    }
  }
}

// The launches of one weight format.
template <int G>
struct StreamLaunch {
  template <int MODE, int NT>
  static auto kernel() {
    if constexpr (MODE == kDown) return down_kernel<G, NT>;
    else return stream_kernel<G, MODE, NT>;
  }
  template <int MODE, int NT>
  static cudaError_t one(const StreamArgs& a, int grid, size_t smem, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((MODE == kDown ? kBlockWarps : consumer_warps(NT) + 1) * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, kernel<MODE, NT>(), a);
  }
  template <int MODE>
  static cudaError_t by_tiles(const StreamArgs& a, int grid, size_t smem, cudaStream_t stream) {
    if (a.xrows <= 8) return one<MODE, 1>(a, grid, smem, stream);
    if constexpr (MODE == kLinear) {
      if (a.xrows > 16) return one<MODE, 4>(a, grid, smem, stream);
    }
    return one<MODE, 2>(a, grid, smem, stream);
  }
  static cudaError_t launch(const StreamArgs& a, int mode, int grid, size_t smem,
                            cudaStream_t stream) {
    if (mode == kGateUp) return by_tiles<kGateUp>(a, grid, smem, stream);
    if (mode == kPairs) return by_tiles<kPairs>(a, grid, smem, stream);
    if constexpr (G != 0) {
      if (mode == kLinear) return by_tiles<kLinear>(a, grid, smem, stream);
    }
    return by_tiles<kDown>(a, grid, smem, stream);
  }
  template <int MODE, int NT>
  static cudaError_t prepare_one() {
    cudaError_t e = cudaFuncSetAttribute(kernel<MODE, NT>(),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel<MODE, NT>(), cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    return e;
  }
  template <int MODE>
  static cudaError_t prepare_mode() {
    cudaError_t e = prepare_one<MODE, 1>();
    if (e == cudaSuccess) e = prepare_one<MODE, 2>();
    if constexpr (MODE == kLinear) {
      if (e == cudaSuccess) e = prepare_one<MODE, 4>();
    }
    return e;
  }
  // clusters[i] (may be NULL): how many clusters of 1 << i blocks the device holds at once
  static cudaError_t prepare(int* clusters) {
    cudaError_t e = prepare_mode<kGateUp>();
    if (e == cudaSuccess) e = prepare_mode<kPairs>();
    if (e == cudaSuccess) e = prepare_mode<kDown>();
    if constexpr (G != 0) {
      if (e == cudaSuccess) e = prepare_mode<kLinear>();
    }
    if (!clusters) return e;
    for (int i = 0; i < kClusterSizes && e == cudaSuccess; ++i) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(1 << i);
      cfg.blockDim = dim3(kBlockWarps * 32);
      cfg.dynamicSmemBytes = kSmem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 1 << i;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&clusters[i], kernel<kDown, 1>(), &cfg);
    }
    return e;
  }
  static cudaError_t take_faults(unsigned* out) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_moe_fault_flags, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_moe_fault_flags, &zero, sizeof(unsigned));
  }
  static cudaError_t wait_test(unsigned stall, unsigned long long limit_ns) {
    cudaError_t e = cudaMemcpyToSymbol(g_moe_test_stall, &stall, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_moe_wait_limit_ns, &limit_ns, sizeof(unsigned long long));
  }
  static cudaError_t take_checks(CheckRecord* r) { return take_check_record_here(r); }
};

}  // namespace

// What mol_moe.cu calls, one set for each weight format.
#define MOL_MOE_FORMAT(G)                                                                     \
  template <>                                                                                 \
  cudaError_t stream_launch<G>(const StreamArgs& a, int mode, int grid, size_t smem,          \
                               cudaStream_t stream) {                                         \
    return StreamLaunch<G>::launch(a, mode, grid, smem, stream);                              \
  }                                                                                           \
  template <>                                                                                 \
  cudaError_t stream_prepare<G>(int* clusters) {                                              \
    return StreamLaunch<G>::prepare(clusters);                                                \
  }                                                                                           \
  template <>                                                                                 \
  cudaError_t stream_take_faults<G>(unsigned* out) {                                          \
    return StreamLaunch<G>::take_faults(out);                                                 \
  }                                                                                           \
  template <>                                                                                 \
  cudaError_t stream_wait_test<G>(unsigned stall, unsigned long long limit_ns) {              \
    return StreamLaunch<G>::wait_test(stall, limit_ns);                                       \
  }                                                                                           \
  template <>                                                                                 \
  cudaError_t stream_take_checks<G>(unsigned long long* first, unsigned long long* count) {   \
    CheckRecord r;                                                                            \
    const cudaError_t e = StreamLaunch<G>::take_checks(&r);                                   \
    *first = r.first;                                                                         \
    *count = r.count;                                                                         \
    return e;                                                                                 \
  }

}  // namespace mol
