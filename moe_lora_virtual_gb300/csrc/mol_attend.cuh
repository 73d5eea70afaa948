// What the attention kernels share: sequences, their row blocks and key ranges, the joining of parts.
#pragma once

#include "mol_attend.h"
#include "mol_device.cuh"

namespace mol {
namespace attn {

// A NaN or an infinity among eight bf16 values: an exponent of ones carries into the sign's place.
MOL_DEV bool not_finite(const uint4& q) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) c |= (w[i] & 0x7F807F80u) + 0x00800080u;
  return (c & 0x80008000u) != 0;
}

MOL_DEV float ex2(float x) {  // 2^x, within 2^-22 of it; 0 for -infinity
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One sequence of the call: its first row of q, its rows, its cached tokens. Whatever the caller's
// arrays hold, rows stay within the call's and tokens within the page table.
struct Seq {
  int start, n, kv;
};
MOL_DEV int seq_start(const AttnArgs& a, int b) {
  if (!a.q_starts) return b;
  return min(max(__ldg(a.q_starts + b), 0), a.num_tokens);
}
MOL_DEV Seq sequence(const AttnArgs& a, int b) {
  Seq s;
  s.start = seq_start(a, b);
  s.n = a.q_starts ? max(seq_start(a, b + 1) - s.start, 0) : 1;
  s.kv = min(max(__ldg(a.kv_lens + b), 0), a.max_pages * a.page_size);
  return s;
}

// A sequence's rows (new tokens x the group's query heads, row = token * group + head) are cut into
// blocks of `rows`. A block and the tiles of `tile` cached tokens that one of its rows sees:
struct Block {
  int b, r;         // sequence, block of it
  Seq s;
  int row0, nrows;  // first row within the sequence, rows
  int lo, hi;       // tokens that some row sees lie in [lo, hi)
  int t0, tiles;    // tiles of them (one, with nothing in it, where there are none)
};
// Blocks of a sequence; none where it is another launch's.
MOL_DEV int num_blocks(const AttnArgs& a, const Seq& s, int rows) {
  const int total = s.n * a.group;
  return total < a.min_rows || total > a.max_rows ? 0 : (total + rows - 1) / rows;
}
MOL_DEV Block block_of(const AttnArgs& a, int b, const Seq& s, int r, int rows, int tile) {
  Block k;
  k.b = b;
  k.r = r;
  k.s = s;
  k.row0 = r * rows;
  k.nrows = min(s.n * a.group - k.row0, rows);
  const int i0 = k.row0 / a.group, i1 = (k.row0 + k.nrows - 1) / a.group;
  const int shift = s.kv - s.n;
  k.hi = max(shift + i1 + 1, 0);
  k.lo = a.window > 0 ? max(shift + i0 - a.window + 1, 0) : 0;
  k.t0 = k.lo / tile;
  k.tiles = max((k.hi + tile - 1) / tile - k.t0, 1);
  return k;
}

// What a launch does is counted in units: a block's tiles and `extra` more for what it takes to begin
// and to end one. All units of the launch, in the order (sequence, block, head, unit), are dealt in
// even runs to its thread blocks.
struct Place {  // where a thread block's run begins
  Block k;
  int h, unit;
};
struct Run {
  int64_t total, from, to;  // units of the launch, this thread block's
  int64_t share, longer;    // units a thread block; the first `longer` ones have one more
  bool any;
  MOL_DEV int64_t begin(int64_t c) const { return c * share + min(c, longer); }
  // The thread block that has unit u.
  MOL_DEV int owner(int64_t u) const {
    const int64_t split = longer * (share + 1);
    return (int)(u < split ? u / (share + 1) : longer + (u - split) / share);
  }
};

// Every thread of a thread block of THREADS calls it; `sh` holds THREADS / 32 + 1 ints. *place is
// written where the run is not empty. A thread a sequence: one round trip for their lengths.
template <int THREADS>
MOL_DEV Run deal(const AttnArgs& a, int rows, int tile, int extra, int* sh, Place* place) {
  if (threadIdx.x == 0) place->k.tiles = 0;
  Run run;
  Seq s = {};
  int blocks = 0, before = 0, sum = 0, n = 0;
  auto units = [&](int b) {
    n = blocks = 0;
    if (b >= a.num_seqs) return;
    s = sequence(a, b);
    blocks = num_blocks(a, s, rows);
    for (int r = 0; r < blocks; ++r) n += block_of(a, b, s, r, rows, tile).tiles + extra;
  };
  run.total = 0;
  for (int b0 = 0; b0 < a.num_seqs; b0 += THREADS) {
    units(b0 + threadIdx.x);
    before = block_exclusive_scan<THREADS>(n, sh, sum);
    run.total += sum;
  }
  run.total *= a.kv_heads;
  const int64_t c = blockIdx.x, grid = gridDim.x;
  if (run.total < (int64_t)1 << 31) {  // (a division of 64 bits takes a few times as long)
    run.share = (uint32_t)run.total / (uint32_t)grid;
    run.longer = (uint32_t)run.total % (uint32_t)grid;
  } else {
    run.share = run.total / grid;
    run.longer = run.total % grid;
  }
  run.from = run.begin(c);
  run.to = run.begin(c + 1);
  run.any = run.from < run.to;
  if (!run.any) return run;
  int64_t passed = 0;
  for (int b0 = 0; b0 < a.num_seqs && passed * a.kv_heads <= run.from; b0 += THREADS) {
    if (a.num_seqs > THREADS) {  // (else as above)
      units(b0 + threadIdx.x);
      before = block_exclusive_scan<THREADS>(n, sh, sum);
    }
    int64_t at = run.from - (passed + before) * a.kv_heads;
    if (at >= 0 && at < (int64_t)n * a.kv_heads) {
      for (int r = 0; r < blocks; ++r) {
        const Block k = block_of(a, b0 + threadIdx.x, s, r, rows, tile);
        const int u = k.tiles + extra;
        if (at < (int64_t)u * a.kv_heads) {
          place->k = k;
          place->h = (int)(at / u);
          place->unit = (int)(at - (int64_t)place->h * u);
          break;
        }
        at -= (int64_t)u * a.kv_heads;
      }
    }
    passed += sum;
  }
  __syncthreads();
  return run;
}

// A walk over a thread block's run, a block's head at a time.
template <int TILE, int EXTRA>
struct Walk {
  Block k;
  int rows, h;
  int first, count;  // tiles of the block in the run
  int unit;
  int64_t left;      // units of the run from here on
  MOL_DEV void start(const AttnArgs& a, const Place& p, int rows_, const Run& run) {
    k = p.k;
    rows = rows_;
    h = p.h;
    unit = p.unit;
    left = k.tiles > 0 ? run.to - run.from : 0;  // (0: starts that decrease; sums of units may mislead)
    if (left == 0) return;
    cut();
    if (count == 0) next(a);
  }
  MOL_DEV void cut() {
    const int n = (int)min((int64_t)(k.tiles + EXTRA - unit), left);
    first = max(unit - EXTRA, 0);
    count = max(unit + n - EXTRA, 0) - first;
  }
  MOL_DEV bool more() const { return left > 0; }
  MOL_DEV bool ends() const { return first + count >= k.tiles; }
  // On to the next head or block; ones that the run has no tile of are passed by.
  MOL_DEV void next(const AttnArgs& a) {
    do {
      left -= k.tiles + EXTRA - unit;
      if (left <= 0) return;
      unit = 0;
      if (++h == a.kv_heads) {
        h = 0;
        int b = k.b, r = k.r + 1;
        Seq s = k.s;
        while (r >= num_blocks(a, s, rows)) {
          if (++b >= a.num_seqs) {
            left = 0;
            return;
          }
          s = sequence(a, b);
          r = 0;
        }
        k = block_of(a, b, s, r, rows, TILE);
      }
      cut();
    } while (count == 0);
  }
  // The last thread block that has a tile of this block, which the run begins and does not end.
  MOL_DEV int last(const Run& r) const { return r.owner(r.to + (k.tiles - first - count) - 1); }
};

// Parts of blocks that several thread blocks share. Thread block c leaves the part that continues its
// predecessor's block in slot 2c, the one that it begins and does not end in slot 2c + 1 with a
// record of it: last thread block of it (-1: there is none), the sequence's first row of q, first row
// within it, rows, head.
struct Record {
  int last, start, row0, nrows, h, pad[3];
};
struct Parts {
  float* sums;   // [slot][rows][D], not divided
  float2* tops;  // [slot][rows]: largest scaled score (base 2), sum of the weights
  Record* records;
};
__host__ __device__ inline size_t parts_bytes(int grid, int rows, int D) {
  return (size_t)grid * 2 * rows * (D * 4 + 8) + (size_t)grid * sizeof(Record);
}
__host__ __device__ inline Parts parts(void* p, int grid, int rows, int D) {
  Parts r;
  char* c = static_cast<char*>(p);
  r.sums = reinterpret_cast<float*>(c);
  c += (size_t)grid * 2 * rows * D * 4;
  r.tops = reinterpret_cast<float2*>(c);
  c += (size_t)grid * 2 * rows * 8;
  r.records = reinterpret_cast<Record*>(c);
  return r;
}

// Joins the parts of every record: out = sum_p f_p sums_p / sum_p f_p weights_p with f_p = 2^(top_p - top),
// in an order that the timing does not change.
cudaError_t launch_join(const AttnArgs& a, int grid, int rows, const Parts& p, cudaStream_t stream);

// The device's SMs, at most 152.
int sms();

// Many rows: sequences of at least a.min_rows rows (mol_attend_tc.cu). Whether its tiles can be loaded from
// pages of this size, for heads of this width.
bool many_fits(int page_size, int head_dim);
size_t many_bytes(int group, int head_dim);
cudaError_t prepare_many();
cudaError_t launch_many(const AttnArgs& a, cudaStream_t stream);

}  // namespace attn
}  // namespace mol
