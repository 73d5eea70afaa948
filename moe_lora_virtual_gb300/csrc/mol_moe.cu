// The experts of a MoE layer for a few tokens and the 4-bit linear (include/mol_block.h).
//
// Mathematics. Both halves of the experts and the linear are products w . x of weight rows with a
// few activation rows, every weight used by the tokens of its expert only (a few), so the time is
// that of reading the taken experts' weights once: 2 bytes (or about half a byte) for 2 n
// operations at n tokens an expert. One streaming loop serves all three:
//
// - A block owns weight rows and walks (expert entry, k) stages: up to 128 weight rows by 256
//   bytes of bf16 (128 inputs) or 128 bytes of 4-bit (256 inputs), and the same inputs of the
//   entry's tokens, copied by all threads with 16-byte cp.async into a ring of stages.
// - A warp multiplies 16 rows with mma.sync m16n8k16: weight rows are the M side, tokens the N
//   side (8 a tile), so one token wastes tensor work and no bandwidth. The contraction's order is
//   free as long as both sides agree: each lane takes 8 neighbouring inputs of its row in one
//   16-byte shared-memory read, for two mma steps. Tokens of one tile are independent columns.
// - 4-bit words become bf16 pairs with a mask and a subtraction that are exact ((128 + q) - 136);
//   a group's products are summed in fp32 first and multiplied by its scale after, so nothing is
//   rounded that fp32 arithmetic would not round.
// - Work is dealt by weight bytes: the gate_up rows of all taken experts form one list that the
//   blocks share evenly, whatever the routing; the down rows are dealt to clusters, whose blocks
//   split the (expert, k) axis and add their fp32 sums through distributed shared memory in the
//   order of their ranks. No atomics on results.
// - Each block groups the (token, slot) pairs by expert itself (at most 1024 of them: match masks,
//   counts in shared memory, one scan), so the layer is two launches, and the down kernel groups the pairs
//   and asks for its first weights while the gate_up kernel's last blocks still run.

#include <type_traits>

#include "mol_block.h"
#include "mol_device.cuh"
#include "mol_internal.h"

namespace mol {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxStages = 8;
constexpr int kExpertsPerThread = MOL_MOE_MAX_EXPERTS / kThreads;
constexpr int kPairsPerThread = MOL_MOE_MAX_PAIRS / kThreads;
// Shared memory of one block: two blocks of this size fit an SM, or one of twice it.
constexpr int kSmemTwo = 112 * 1024;
constexpr int kSmemOne = 224 * 1024;

enum Mode { kGateUp = 0, kDown = 1, kLinear = 2 };

struct StreamArgs {
  const bf16* x;         // activation rows: tokens (gate_up, linear) or pairs (down)
  const int32_t* ids;    // [numel], not for the linear
  const float* weights;  // [numel], down only
  const char* w;
  const bf16* scales;
  const bf16* delta;
  bf16* out;             // act, or the output rows
  int64_t x_stride, delta_stride, out_stride;
  int num_tokens, topk, E;
  int K;                 // contraction width
  int N;                 // outputs of one expert: I, H, or the linear's N
  int xrows;             // tokens of one entry at most: 8, 16, 32, 64
  int rows;              // weight rows of a stage at most, a multiple of 16
  int stages;
  int stage_bytes;
  int acc_stride;        // floats between tokens of the block's sums (down, linear)
};

template <int G>
struct Format {
  static constexpr bool kW4 = G != 0;
  static constexpr int kStageK = kW4 ? 256 : 128;    // inputs of a stage
  static constexpr int kRowBytes = kW4 ? 128 : 256;  // weight bytes of a row in a stage
  static constexpr int kXBytes = kStageK * 2;        // activation bytes of a token in a stage
  static constexpr int kScaleBytes = kW4 ? 2 * (256 / (kW4 ? G : 1)) : 0;  // of a row in a stage
};

template <int G>
constexpr int stage_bytes(int rows, int xrows) {
  using F = Format<G>;
  return rows * (F::kRowBytes + F::kScaleBytes) + xrows * F::kXBytes;
}

// 16-byte chunks of odd rows are stored with bit 2 of their index flipped: the eight lanes of a
// shared-memory phase (two neighbouring rows, four chunks each) then cover all 32 banks.
MOL_DEV int swizzle(int chunk, int row) { return chunk ^ ((row & 1) << 2); }

MOL_DEV void cp_async_small(void* dst, const void* src, int bytes) {  // 4 or 8 bytes
  if (bytes == 4)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

MOL_DEV void wait_stage(int stages) {  // the oldest of stages - 1 groups in flight has landed
  switch (stages) {
    case 2: cp_async_wait_group<0>(); break;
    case 3: cp_async_wait_group<1>(); break;
    case 4: cp_async_wait_group<2>(); break;
    case 5: cp_async_wait_group<3>(); break;
    case 6: cp_async_wait_group<4>(); break;
    case 7: cp_async_wait_group<5>(); break;
    default: cp_async_wait_group<6>(); break;
  }
}

// Tokens of one expert, at most xrows of them: a tile's columns.
struct Entry {
  int e, off, n;
};

// The pairs grouped by expert, in shared memory.
struct Lists {
  uint32_t* order;  // [numel] pair | token << 16, by entry
  float* weight;    // [numel] of the same pairs (down)
  int2* entry;      // x: expert, y: first pair | pairs << 16
  int count;        // entries
  bool repeated;    // some token lists an expert twice
  MOL_DEV Entry get(int a) const {
    const int2 v = entry[a];
    return Entry{v.x, v.y & 0xFFFF, v.y >> 16};
  }
};

// Groups the pairs by expert, in the order of their index: every block finds the same entries, so
// blocks that hold different rows of one expert agree on which entry has which pair. Each warp
// ranks a contiguous run of pairs with match masks and per-warp counts; the counts are then summed
// over the warps, one thread to four experts. `scratch`: 16 E + 4 numel bytes (20 KB at most, and
// the ring it lies in is never smaller), free again afterwards.
MOL_DEV void build_lists(const StreamArgs& a, Lists& l, char* scratch, bool weights) {
  __shared__ int scan[kWarps + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, numel = a.num_tokens * a.topk;
  const int rounds = (numel + kThreads - 1) / kThreads;
  int* ids = reinterpret_cast<int*>(scratch);
  uint16_t* cnt = reinterpret_cast<uint16_t*>(ids + numel);  // [warp][expert]
  int mine[kPairsPerThread], pos[kPairsPerThread];
  const int first = warp * rounds * 32 + lane;
#pragma unroll
  for (int j = 0; j < kPairsPerThread; ++j) {
    const int i = first + j * 32;
    mine[j] = j < rounds && i < numel ? ld_cg_i32(a.ids + i) : -1;
    if (mine[j] >= a.E) mine[j] = -1;
  }
  for (int e = tid; e < a.E * (kWarps / 2); e += kThreads) reinterpret_cast<uint32_t*>(cnt)[e] = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPairsPerThread; ++j) {
    if (j >= rounds) break;
    const int i = first + j * 32;
    if (i < numel) ids[i] = mine[j];
    const unsigned same = __match_any_sync(0xffffffffu, mine[j]);
    const int before = __popc(same & lanemask_lt());
    if (mine[j] >= 0) pos[j] = cnt[warp * a.E + mine[j]] + before;
    __syncwarp();
    if (mine[j] >= 0 && before == 0) cnt[warp * a.E + mine[j]] += (uint16_t)__popc(same);
    __syncwarp();
  }
  __syncthreads();
  bool again = false;
  if (weights) {
#pragma unroll
    for (int j = 0; j < kPairsPerThread; ++j) {
      const int i = first + j * 32;
      if (mine[j] >= 0)
        for (int q = i - i % a.topk; q < i; ++q) again |= ids[q] == mine[j];
    }
  }
  // Counts before each warp's pairs, then (count, entries) offsets of the experts in 16 bits each.
  int c[kExpertsPerThread], sum = 0;
#pragma unroll
  for (int j = 0; j < kExpertsPerThread; ++j) {
    const int e = tid * kExpertsPerThread + j;
    c[j] = 0;
    if (e < a.E) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const int n = cnt[w * a.E + e];
        cnt[w * a.E + e] = (uint16_t)c[j];
        c[j] += n;
      }
    }
    sum += c[j] | ((c[j] + a.xrows - 1) / a.xrows) << 16;
  }
  int total;
  int at = block_exclusive_scan<kThreads>(sum, scan, total);
#pragma unroll
  for (int j = 0; j < kExpertsPerThread; ++j) {
    const int e = tid * kExpertsPerThread + j;
    if (c[j] > 0) {
      const int off = at & 0xFFFF;
      int idx = at >> 16;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) cnt[w * a.E + e] += (uint16_t)off;
      for (int o = 0; o < c[j]; o += a.xrows)
        l.entry[idx++] = make_int2(e, (off + o) | (min(a.xrows, c[j] - o) << 16));
    }
    at += c[j] | ((c[j] + a.xrows - 1) / a.xrows) << 16;
  }
  l.count = total >> 16;
  l.repeated = __syncthreads_or(again);
#pragma unroll
  for (int j = 0; j < kPairsPerThread; ++j) {
    const int i = first + j * 32;
    if (mine[j] >= 0) {
      const int s = cnt[warp * a.E + mine[j]] + pos[j];
      l.order[s] = (uint32_t)i | (uint32_t)(i / a.topk) << 16;
      if (weights) l.weight[s] = a.weights[i];
    }
  }
  __syncthreads();
}

// Where a block is in its work: the stage (entry, first row, rows, k step).
// gate_up: positions are (entry, row pair); a tile is up to rows / 2 row pairs, all of K.
// down, linear: positions are (entry, k step) of the block's share [lo, hi), once for each block
// of at most `rows` output rows of [row, row_end).
template <int MODE>
struct Cursor {
  int lo, hi, pos, ks, ksteps, entry;
  int row, row_end, rows, rows_max;
  int N;
  bool valid;

  MOL_DEV void load() {
    if (MODE == kGateUp) {
      entry = pos / N;
      row = pos - entry * N;
      rows = min(min(rows_max, N - row), hi - pos);
      ks = 0;
    } else {
      entry = pos / ksteps;
      ks = pos - entry * ksteps;
      rows = min(rows_max, row_end - row);
    }
  }
  // rows: row pairs (gate_up) or rows of a tile at most
  MOL_DEV void init(int lo_, int hi_, int ksteps_, int N_, int row_, int row_end_, int rows_) {
    lo = pos = lo_;
    hi = hi_;
    ksteps = ksteps_;
    N = N_;
    row = row_;
    row_end = row_end_;
    rows_max = rows_;
    valid = lo < hi && (MODE == kGateUp || row < row_end);
    if (valid) load();
  }
  MOL_DEV bool tile_ends() const { return ks == ksteps - 1 || (MODE != kGateUp && pos == hi - 1); }
  MOL_DEV bool share_ends() const { return pos == hi - 1; }
  MOL_DEV void next() {
    if (MODE == kGateUp) {
      if (++ks < ksteps) return;
      pos += rows;
      valid = pos < hi;
      if (valid) load();
    } else {
      const bool wrap = ++pos == hi;
      if (wrap) {
        pos = lo;
        row += rows;
        valid = row < row_end;
      }
      if (wrap || ++ks == ksteps) {
        if (valid) load();
      }
    }
  }
};

// Copies the weight rows (and scales) of the cursor's stage.
template <int G, int MODE>
MOL_DEV void copy_weights(const StreamArgs& a, const Cursor<MODE>& c, const Entry& en, char* stage) {
  using F = Format<G>;
  constexpr int kChunks = F::kRowBytes / 16, kStep = kThreads / kChunks;
  const int chunk = threadIdx.x % kChunks, r0 = threadIdx.x / kChunks;
  const int64_t pitch = F::kW4 ? w4_padded(a.K) / 2 : (int64_t)a.K * 2;
  const int koff = c.ks * F::kRowBytes + chunk * 16;
  const bool in_row = koff < pitch;
  // a tile row r: gate_up: eight gate rows, then the eight up rows of the same outputs
  auto source = [&](int r, bool& ok) -> int64_t {
    if (MODE == kGateUp) {
      const int p = (r >> 4) * 8 + (r & 7);
      ok = p < c.rows;
      return (int64_t)en.e * 2 * a.N + c.row + p + ((r & 8) ? a.N : 0);
    }
    ok = r < c.rows;
    return (int64_t)en.e * a.N + c.row + r;
  };
  const int top = MODE == kGateUp ? (c.rows + 7) / 8 * 16 : c.rows;
  for (int r = r0; r < top; r += kStep) {
    bool ok;
    const int64_t row = source(r, ok);
    if (!ok) continue;
    if (!MOL_CHECK(row >= 0 && row < (int64_t)a.E * (MODE == kGateUp ? 2 : 1) * a.N,
                   MOL_CHECK_WEIGHT_ROW, row) ||
        !MOL_CHECK(r < a.rows, MOL_CHECK_SMEM, r))
      continue;
    cp_async16_zfill(stage + r * F::kRowBytes + swizzle(chunk, r) * 16,
                     a.w + row * pitch + (in_row ? koff : 0), in_row ? 16 : 0);
  }
  if constexpr (F::kW4) {
    char* sc = stage + a.rows * F::kRowBytes;
    const int64_t spitch = w4_padded(a.K) / G * 2;
    for (int r = threadIdx.x; r < top; r += kThreads) {
      bool ok;
      const int64_t row = source(r, ok);
      if (!ok) continue;
      const char* src = reinterpret_cast<const char*>(a.scales) + row * spitch +
                        c.ks * F::kScaleBytes;
      if constexpr (F::kScaleBytes == 16)
        cp_async16_zfill(sc + r * 16, src, 16);
      else
        cp_async_small(sc + r * F::kScaleBytes, src, F::kScaleBytes);
    }
  }
}

// Copies the same inputs of the entry's tokens; inputs past K are zeros.
template <int G, int MODE>
MOL_DEV void copy_x(const StreamArgs& a, const Cursor<MODE>& c, const Entry& en, const Lists& l,
                    char* stage) {
  using F = Format<G>;
  constexpr int kChunks = F::kXBytes / 16, kStep = kThreads / kChunks;
  const int chunk = threadIdx.x % kChunks;
  const int k = c.ks * F::kStageK + chunk * 8;
  char* xs = stage + a.rows * (F::kRowBytes + F::kScaleBytes);
  for (int i = threadIdx.x / kChunks; i < en.n; i += kStep) {
    int row = i;
    if (MODE != kLinear) {
      const uint32_t p = l.order[en.off + i];
      row = MODE == kGateUp ? p >> 16 : p & 0xFFFF;
    }
    if (!MOL_CHECK(row < (MODE == kDown ? a.num_tokens * a.topk : a.num_tokens), MOL_CHECK_ROW, row) ||
        !MOL_CHECK(i < a.xrows, MOL_CHECK_SMEM, i))
      continue;
    cp_async16_zfill(xs + i * F::kXBytes + swizzle(chunk, i) * 16,
                     a.x + row * a.x_stride + (k < a.K ? k : 0), k < a.K ? 16 : 0);
  }
}

MOL_DEV uint32_t w4_pair(uint32_t v) {  // two nibbles at bits 0 and 16 -> bf16 pair q - 8, exact
  const uint32_t b = (v & 0x000F000Fu) | 0x43004300u;  // 128 + q
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&b),
                             __nv_bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308)));
  return *reinterpret_cast<uint32_t*>(&r);
}

// One stage's products of a warp's 16 rows with NT tiles of 8 tokens; `part` of `parts` shares of
// the stage's inputs.
template <int G, int NT>
MOL_DEV void multiply(float (&acc)[8][4], const char* wrow, const char* scales, const char* xs,
                      int g, int t, int part, int parts, int k0, int K) {
  using F = Format<G>;
  const int sw = (g & 1) << 2;
  if constexpr (!F::kW4) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if ((b & (parts - 1)) != part) continue;
      const int o = ((b * 4 + t) ^ sw) * 16;
      const uint4 a0 = lds16(wrow + o), a1 = lds16(wrow + 8 * F::kRowBytes + o);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 x = lds16(xs + nt * 8 * F::kXBytes + o);
        mma_16816(acc[nt], a0.x, a1.x, a0.y, a1.y, x.x, x.y);
        mma_16816(acc[nt], a0.z, a1.z, a0.w, a1.w, x.z, x.w);
      }
    }
  } else {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if ((b & (parts - 1)) != part || k0 + b * 128 >= K) continue;
      const int o = ((b * 4 + t) ^ sw) * 16;
      const uint4 a0 = lds16(wrow + o), a1 = lds16(wrow + 8 * F::kRowBytes + o);
      const uint32_t w0[4] = {a0.x, a0.y, a0.z, a0.w}, w1[4] = {a1.x, a1.y, a1.z, a1.w};
      float sum[NT][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i * 32 % G == 0) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            sum[nt][0] = sum[nt][1] = sum[nt][2] = sum[nt][3] = 0.f;
        }
        uint32_t p0[4], p1[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          p0[j] = w4_pair(w0[i] >> (4 * j));
          p1[j] = w4_pair(w1[i] >> (4 * j));
        }
        const int xo = ((b * 16 + i * 4 + t) ^ sw) * 16;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint4 x = lds16(xs + nt * 8 * F::kXBytes + xo);
          mma_16816(sum[nt], p0[0], p1[0], p0[1], p1[1], x.x, x.y);
          mma_16816(sum[nt], p0[2], p1[2], p0[3], p1[3], x.z, x.w);
        }
        if ((i + 1) * 32 % G == 0) {
          // a group wholly past K holds no weights: its scale may be anything
          const int grp = (b * 128 + i * 32) / G;
          const bool in = k0 + grp * G < K;
          const float s0 = in ? __bfloat162float(reinterpret_cast<const bf16*>(scales)[grp]) : 0.f;
          const float s1 =
              in ? __bfloat162float(
                       reinterpret_cast<const bf16*>(scales + 8 * F::kScaleBytes)[grp])
                 : 0.f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            acc[nt][0] = fmaf(s0, sum[nt][0], acc[nt][0]);
            acc[nt][1] = fmaf(s0, sum[nt][1], acc[nt][1]);
            acc[nt][2] = fmaf(s1, sum[nt][2], acc[nt][2]);
            acc[nt][3] = fmaf(s1, sum[nt][3], acc[nt][3]);
          }
        }
      }
    }
  }
}

MOL_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
MOL_DEV uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
MOL_DEV void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
MOL_DEV float remote_f32(uint32_t addr, uint32_t rank) {
  uint32_t p;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(p) : "memory");
  return v;
}

template <int G, int MODE, bool CHAINED>
__global__ void __launch_bounds__(kThreads, 2) stream_kernel(const StreamArgs a) {
  using F = Format<G>;
  extern __shared__ __align__(128) char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int numel = a.num_tokens * a.topk;
  const int ksteps = (a.K + F::kStageK - 1) / F::kStageK;

  // shared memory: stages | sums (down, linear) | lists (the experts)
  char* stages = smem;
  float* sums = reinterpret_cast<float*>(smem + a.stages * a.stage_bytes);
  Lists lists;
  lists.entry = reinterpret_cast<int2*>(sums + (MODE == kGateUp ? 0 : a.num_tokens * a.acc_stride));
  lists.order = reinterpret_cast<uint32_t*>(lists.entry + (MODE == kLinear ? 0 : numel));
  lists.weight = reinterpret_cast<float*>(lists.order + numel);
  lists.count = 1;
  lists.repeated = false;

  if (!CHAINED) {
    pdl_wait();
    pdl_launch_dependents();
  }
  if (MODE != kLinear) build_lists(a, lists, stages, MODE == kDown);
  auto entry_of = [&](int i) {
    return MODE == kLinear ? Entry{0, 0, a.num_tokens} : lists.get(i);
  };

  // this block's share
  Cursor<MODE> cur;
  const uint32_t ranks = MODE == kGateUp ? 1 : cluster_size();
  const uint32_t rank = MODE == kGateUp ? 0 : cluster_rank();
  if (MODE == kGateUp) {
    const int64_t all = (int64_t)lists.count * a.N;
    cur.init((int)(all * blockIdx.x / gridDim.x), (int)(all * (blockIdx.x + 1) / gridDim.x), ksteps,
             a.N, 0, 0, a.rows / 2);
  } else {
    const int clusters = gridDim.x / ranks, cl = blockIdx.x / ranks;
    const int r0 = (int)((int64_t)a.N * cl / clusters), r1 = (int)((int64_t)a.N * (cl + 1) / clusters);
    const int units = lists.count * ksteps;
    const int blocks = (r1 - r0 + a.rows - 1) / a.rows;  // equal blocks of rows
    cur.init((int)((int64_t)units * rank / ranks), (int)((int64_t)units * (rank + 1) / ranks), ksteps,
             a.N, r0, r1, blocks ? (r1 - r0 + blocks - 1) / blocks : 1);
    // a cluster without rows, or a block without stages, still takes part in the sums below
  }

  // warps: 16-row tiles, and shares of a stage's inputs when there are few tiles
  int tiles = kWarps, parts = 1;
  if (MODE != kGateUp) {
    tiles = 1;
    while (tiles * 16 < cur.rows_max) tiles *= 2;
    parts = min(kWarps / tiles, F::kW4 ? 2 : 4);
  }
  const int tile = warp % tiles, part = warp / tiles;

  if (MODE != kGateUp)
    for (int i = tid; i < a.num_tokens * a.acc_stride; i += kThreads) sums[i] = 0.f;

  Cursor<MODE> put = cur;
  const int ahead = a.stages - 1;
  if (CHAINED) {
    // the weights of the first stages, then the wait for the rows that the kernel before writes
    Cursor<MODE> p = put;
    for (int s = 0; s < ahead && p.valid; ++s, p.next())
      copy_weights<G, MODE>(a, p, entry_of(p.entry), stages + s * a.stage_bytes);
    pdl_wait();
    pdl_launch_dependents();
  }
  for (int s = 0; s < ahead; ++s) {
    if (put.valid) {
      const Entry en = entry_of(put.entry);
      if (!CHAINED) copy_weights<G, MODE>(a, put, en, stages + s * a.stage_bytes);
      copy_x<G, MODE>(a, put, en, lists, stages + s * a.stage_bytes);
      put.next();
    }
    cp_async_commit();
  }

  float acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;

  // The sums of a block of rows: over the cluster's ranks in their order, the deltas, one rounding.
  auto write_rows = [&](int row, int rows) {
    if (ranks > 1) cluster_barrier();
    else __syncthreads();
    const int total = rows * a.num_tokens;
    for (int i = tid + rank * kThreads; i < total; i += kThreads * ranks) {
      const int tok = i / rows, r = i - tok * rows;
      const int at = tok * a.acc_stride + r;
      float v = 0.f;
      if (ranks > 1) {
        for (uint32_t q = 0; q < ranks; ++q) v += remote_f32(smem_u32(sums + at), q);
      } else {
        v = sums[at];
      }
      if (MODE == kDown && a.delta) {
        for (int k = 0; k < a.topk; ++k) {
          const int pair = tok * a.topk + k, e = a.ids[pair];
          if (e >= 0 && e < a.E)
            v = fmaf(a.weights[pair], __bfloat162float(a.delta[pair * a.delta_stride + row + r]), v);
        }
      }
      if (MOL_CHECK(row + r < a.N, MOL_CHECK_COLUMN, row + r))
        a.out[tok * a.out_stride + row + r] = __float2bfloat16(v);
    }
    if (ranks > 1) cluster_barrier();
    else __syncthreads();
  };

  if (MODE != kGateUp && !cur.valid) {
    // no stage here: the same barriers as the cluster's other blocks
    for (int row = cur.row; row < cur.row_end; row += cur.rows_max)
      write_rows(row, min(cur.rows_max, cur.row_end - row));
  }
  int slot = 0, put_slot = ahead;
  while (cur.valid) {
    wait_stage(a.stages);
    __syncthreads();
    if (put.valid) {
      const Entry en = entry_of(put.entry);
      copy_weights<G, MODE>(a, put, en, stages + put_slot * a.stage_bytes);
      copy_x<G, MODE>(a, put, en, lists, stages + put_slot * a.stage_bytes);
      put.next();
    }
    cp_async_commit();
    if (++put_slot == a.stages) put_slot = 0;

    const Entry en = entry_of(cur.entry);
    const int ntiles = (en.n + 7) >> 3;
    const bool active =
        part < parts && tile * (MODE == kGateUp ? 8 : 16) < cur.rows;
    if (active) {
      const char* st = stages + slot * a.stage_bytes;
      const char* wrow = st + (tile * 16 + g) * F::kRowBytes;
      const char* sc = st + a.rows * F::kRowBytes + (tile * 16 + g) * F::kScaleBytes;
      const char* xs = st + a.rows * (F::kRowBytes + F::kScaleBytes) + g * F::kXBytes;
      const int k0 = cur.ks * F::kStageK;
      if (ntiles == 1) multiply<G, 1>(acc, wrow, sc, xs, g, t, part, parts, k0, a.K);
      else if (ntiles == 2) multiply<G, 2>(acc, wrow, sc, xs, g, t, part, parts, k0, a.K);
      else if (ntiles <= 4) multiply<G, 4>(acc, wrow, sc, xs, g, t, part, parts, k0, a.K);
      else multiply<G, 8>(acc, wrow, sc, xs, g, t, part, parts, k0, a.K);
    }
    if (++slot == a.stages) slot = 0;

    if (cur.tile_ends()) {
      if (MODE == kGateUp) {
        const int j = tile * 8 + g;
        if (j < cur.rows) {
#pragma unroll
          for (int nt = 0; nt < 8; ++nt) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int col = nt * 8 + 2 * t + h;
              if (col >= en.n) continue;
              const int64_t pair = lists.order[en.off + col] & 0xFFFF;
              if (!MOL_CHECK(pair < numel, MOL_CHECK_ROW, pair)) continue;
              float gate = acc[nt][h], up = acc[nt][2 + h];
              if (a.delta) {
                const bf16* d = a.delta + pair * a.delta_stride + cur.row + j;
                gate += __bfloat162float(d[0]);
                up += __bfloat162float(d[a.N]);
              }
              a.out[pair * a.N + cur.row + j] = __float2bfloat16(gate / (1.f + expf(-gate)) * up);
            }
          }
        }
      } else {
        // add into the block's sums, one share of the inputs after another
        for (int q = 0; q < parts; ++q) {
          if (q > 0) __syncthreads();
          if (active && part == q) {
            // lanes of different columns hold the same token only where a token lists its expert
            // twice: then the four columns of a step take turns
            for (int turn = 0; turn < (lists.repeated ? 4 : 1); ++turn) {
              if (!lists.repeated || t == turn) {
#pragma unroll
                for (int nt = 0; nt < 8; ++nt) {
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    const int col = nt * 8 + 2 * t + h;
                    if (col >= en.n) continue;
                    int tok = col;
                    float wt = 1.f;
                    if (MODE == kDown) {
                      tok = lists.order[en.off + col] >> 16;
                      wt = lists.weight[en.off + col];
                    }
                    float* s = sums + tok * a.acc_stride + tile * 16 + g;
                    if (!MOL_CHECK(tok < a.num_tokens && tile * 16 + g + 8 < a.acc_stride,
                                   MOL_CHECK_SMEM, tok))
                      continue;
                    s[0] = fmaf(wt, acc[nt][h], s[0]);
                    s[8] = fmaf(wt, acc[nt][2 + h], s[8]);
                  }
                }
              }
              __syncwarp();
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    }
    if (MODE != kGateUp && cur.share_ends()) {
      write_rows(cur.row, cur.rows);
      for (int i = tid; i < a.num_tokens * a.acc_stride; i += kThreads) sums[i] = 0.f;
    }
    cur.next();
  }
  cp_async_wait_all();
}

struct Geometry {
  int grid, cluster;
  size_t smem;
};

int g_sm_count = 0;

// The ring that fits beside `fixed` bytes: two blocks per SM when that leaves three stages (their
// barriers and epilogues then overlap), else one block with twice the room.
template <int G>
bool plan_ring(StreamArgs& a, size_t fixed) {
  a.stage_bytes = stage_bytes<G>(a.rows, a.xrows);
  bool two = true;
  int n = ((int)kSmemTwo - (int)fixed) / a.stage_bytes;
  if (n < 3) {
    two = false;
    n = ((int)kSmemOne - (int)fixed) / a.stage_bytes;
  }
  a.stages = n > kMaxStages ? kMaxStages : n;
  return two;
}

// Tokens of an entry: twice the mean of an expert's pairs, so that few experts need a second entry
// (which reads their weights again), and no more room in the ring than the tokens need.
int entry_rows(int num_tokens, int pairs, int experts) {
  int n = 8;
  while (n < 64 && n < num_tokens && n * experts < 2 * pairs) n *= 2;
  return n;
}

constexpr int align_up(int v, int m) { return (v + m - 1) / m * m; }

template <int G, int MODE, bool CHAINED>
cudaError_t launch_stream(const StreamArgs& a, int grid, int cluster, size_t smem,
                          cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = MODE == kGateUp ? 1 : 2;
  count_launch();
  return cudaLaunchKernelEx(&cfg, stream_kernel<G, MODE, CHAINED>, a);
}

// Clusters of eight blocks (two to an SM) or of four (one to an SM) that fit the device at once.
int g_clusters_two = 0, g_clusters_one = 0;

// down, linear: rows over clusters, (entry, k) over a cluster's blocks.
template <int G, int MODE, bool CHAINED>
cudaError_t launch_rows(StreamArgs a, size_t lists, cudaStream_t stream) {
  auto fit = [&](int clusters) {
    const int per = (a.N + clusters - 1) / clusters;
    const int blocks = (per + 127) / 128;
    a.rows = align_up((per + blocks - 1) / blocks, 16);
    int tiles = 1;
    while (tiles * 16 < a.rows) tiles *= 2;
    a.acc_stride = tiles * 16 + 8;
    return (size_t)a.num_tokens * a.acc_stride * 4 + lists;
  };
  size_t fixed = fit(g_clusters_two);
  int clusters = g_clusters_two, size = 8;
  if (!plan_ring<G>(a, fixed)) {
    clusters = g_clusters_one;
    size = 4;
    fixed = fit(clusters);
    plan_ring<G>(a, fixed);
  }
  if (a.stages < 2) return cudaErrorInvalidConfiguration;
  return launch_stream<G, MODE, CHAINED>(a, clusters * size, size,
                                         a.stages * a.stage_bytes + fixed, stream);
}

template <typename F>
cudaError_t by_group(int group, F f) {
  if (group == 0) return f(std::integral_constant<int, 0>{});
  if (group == 32) return f(std::integral_constant<int, 32>{});
  if (group == 64) return f(std::integral_constant<int, 64>{});
  return f(std::integral_constant<int, 128>{});
}

StreamArgs common_args(const MoeShape& s, const void* x, int64_t x_stride, const int32_t* ids,
                       const WeightRows& w, const void* delta, int64_t delta_stride, void* out,
                       int64_t out_stride) {
  StreamArgs a = {};
  a.x = static_cast<const bf16*>(x);
  a.ids = ids;
  a.w = static_cast<const char*>(w.data);
  a.scales = static_cast<const bf16*>(w.scales);
  a.delta = static_cast<const bf16*>(delta);
  a.out = static_cast<bf16*>(out);
  a.x_stride = x_stride;
  a.delta_stride = delta_stride;
  a.out_stride = out_stride;
  a.num_tokens = s.num_tokens;
  a.topk = s.topk;
  a.E = s.num_experts;
  a.K = w.K;
  a.xrows = entry_rows(s.num_tokens, s.num_tokens * s.topk, s.num_experts);
  return a;
}

}  // namespace

cudaError_t launch_moe_gate_up(const MoeShape& s, const void* x, int64_t x_stride,
                               const int32_t* topk_ids, const WeightRows& w, const void* delta,
                               int64_t delta_stride, void* act, cudaStream_t stream) {
  StreamArgs a = common_args(s, x, x_stride, topk_ids, w, delta, delta_stride, act, s.inter);
  a.N = s.inter;
  const int numel = s.num_tokens * s.topk;
  return by_group(w.group, [&](auto gc) {
    constexpr int G = decltype(gc)::value;
    // the tallest tile: a block's share of the row pairs when every pair takes its own expert
    const int grid = 2 * g_sm_count;
    const int64_t most = (int64_t)numel * s.inter;
    const int64_t share = (most + grid - 1) / grid;
    a.rows = (int)(share >= 64 ? 128 : align_up((int)share, 8) * 2);
    const size_t lists = (size_t)numel * (sizeof(int2) + 4);
    const bool two = plan_ring<G>(a, lists);
    return launch_stream<G, kGateUp, false>(a, two ? grid : g_sm_count, 1,
                                            a.stages * a.stage_bytes + lists, stream);
  });
}

cudaError_t launch_moe_down(const MoeShape& s, const void* act, const int32_t* topk_ids,
                            const float* topk_weights, const WeightRows& w, const void* delta,
                            int64_t delta_stride, void* out, int64_t out_stride, bool chained,
                            cudaStream_t stream) {
  StreamArgs a = common_args(s, act, s.inter, topk_ids, w, delta, delta_stride, out, out_stride);
  a.weights = topk_weights;
  a.N = s.hidden;
  const size_t lists = (size_t)s.num_tokens * s.topk * (sizeof(int2) + 8);
  return by_group(w.group, [&](auto gc) {
    constexpr int G = decltype(gc)::value;
    return chained ? launch_rows<G, kDown, true>(a, lists, stream)
                   : launch_rows<G, kDown, false>(a, lists, stream);
  });
}

cudaError_t launch_w4_linear(const void* x, int64_t x_stride, int num_tokens, int N,
                             const WeightRows& w, void* out, int64_t out_stride,
                             cudaStream_t stream) {
  const MoeShape s{num_tokens, 1, 1, N, w.K};
  StreamArgs a = common_args(s, x, x_stride, nullptr, w, nullptr, 0, out, out_stride);
  a.N = N;
  a.xrows = num_tokens <= 8 ? 8 : num_tokens <= 16 ? 16 : num_tokens <= 32 ? 32 : 64;
  if (w.group == 32) return launch_rows<32, kLinear, false>(a, 0, stream);
  if (w.group == 64) return launch_rows<64, kLinear, false>(a, 0, stream);
  return launch_rows<128, kLinear, false>(a, 0, stream);
}

namespace {

template <int G, int MODE, bool CHAINED>
cudaError_t prepare_one() {
  cudaError_t e = cudaFuncSetAttribute(stream_kernel<G, MODE, CHAINED>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemOne);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(stream_kernel<G, MODE, CHAINED>,
                             cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  return e;
}

template <int G>
cudaError_t prepare_group() {
  cudaError_t e = prepare_one<G, kGateUp, false>();
  if (e == cudaSuccess) e = prepare_one<G, kDown, false>();
  if (e == cudaSuccess) e = prepare_one<G, kDown, true>();
  if constexpr (G != 0) {
    if (e == cudaSuccess) e = prepare_one<G, kLinear, false>();
  }
  return e;
}

cudaError_t max_clusters(int size, int smem, int* out) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(out, stream_kernel<0, kDown, false>, &cfg);
}

}  // namespace

cudaError_t prepare_moe_kernels() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&g_sm_count, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = prepare_group<0>();
  if (e == cudaSuccess) e = prepare_group<32>();
  if (e == cudaSuccess) e = prepare_group<64>();
  if (e == cudaSuccess) e = prepare_group<128>();
  if (e == cudaSuccess) e = max_clusters(8, kSmemTwo, &g_clusters_two);
  if (e == cudaSuccess) e = max_clusters(4, kSmemOne, &g_clusters_one);
  if (e == cudaSuccess && (g_clusters_two < 1 || g_clusters_one < 1)) e = cudaErrorInvalidConfiguration;
  return e;
}

cudaError_t take_moe_checks(unsigned long long* first, unsigned long long* count) {
  CheckRecord r;
  const cudaError_t e = take_check_record_here(&r);
  *first = r.first;
  *count = r.count;
  return e;
}

}  // namespace mol
