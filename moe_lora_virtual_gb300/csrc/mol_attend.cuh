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
// blocks of `rows`. Block numbers: sequence b's begin at start * group / rows + b, which leaves each
// sequence room for its own without a sum over those before it. Some numbers are nobody's.
MOL_DEV int first_block(const AttnArgs& a, int b, int rows) {
  return a.q_starts ? (int)((int64_t)seq_start(a, b) * a.group / rows) + b
                    : b * ((a.group + rows - 1) / rows);
}
__host__ __device__ inline int num_blocks(const AttnArgs& a, int rows) {
  return a.q_starts ? (int)((int64_t)a.num_tokens * a.group / rows) + a.num_seqs
                    : a.num_seqs * ((a.group + rows - 1) / rows);
}
// The sequence that block number v falls to.
MOL_DEV int block_seq(const AttnArgs& a, int v, int rows) {
  if (!a.q_starts) return v / ((a.group + rows - 1) / rows);
  int lo = 0, hi = a.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first_block(a, mid, rows) <= v)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// A block of rows and the tiles of `tile` cached tokens that one of its rows sees.
struct Block {
  int b;
  Seq s;
  int row0, nrows;  // first row within the sequence, rows
  int lo, hi;       // tokens that some row sees lie in [lo, hi)
  int t0, tiles;    // tiles of them (one, with nothing in it, where there are none); 0: nobody's
};
MOL_DEV Block block_of(const AttnArgs& a, int v, int b, int rows, int tile) {
  Block k;
  k.b = b;
  k.s = sequence(a, b);
  k.row0 = (v - first_block(a, b, rows)) * rows;
  const int total = k.s.n * a.group;
  k.nrows = min(total - k.row0, rows);
  k.lo = k.hi = k.t0 = k.tiles = 0;
  if (k.row0 < 0 || k.nrows <= 0 || total < a.min_rows || total > a.max_rows) return k;
  const int i0 = k.row0 / a.group, i1 = (k.row0 + k.nrows - 1) / a.group;
  const int shift = k.s.kv - k.s.n;
  k.hi = max(shift + i1 + 1, 0);
  k.lo = a.window > 0 ? max(shift + i0 - a.window + 1, 0) : 0;
  k.t0 = k.lo / tile;
  k.tiles = max((k.hi + tile - 1) / tile - k.t0, 1);
  return k;
}

// What a launch does is counted in units: a block's tiles and `extra` more for what it takes to begin
// and to end one. All units of the launch, in the order (block, head, unit), are dealt in even runs to
// its thread blocks.
struct Place {  // where a thread block's run begins
  Block k;
  int v, h, unit;
};
struct Run {
  int64_t total, grid, from, to;  // units of the launch, thread blocks that get some, this one's
};
MOL_DEV int block_units(const Block& k, int extra) { return k.tiles > 0 ? k.tiles + extra : 0; }

// Every thread of a thread block of THREADS calls it; `sh` holds THREADS / 32 + 1 ints. *place is
// written where the run is not empty.
template <int THREADS>
MOL_DEV Run deal(const AttnArgs& a, int rows, int tile, int extra, int* sh, Place* place) {
  const int nv = num_blocks(a, rows);
  Run run;
  Block k = {};
  int before = 0, sum = 0, n = 0;
  run.total = 0;
  for (int v0 = 0; v0 < nv; v0 += THREADS) {
    const int v = v0 + threadIdx.x;
    n = 0;
    if (v < nv) {
      k = block_of(a, v, block_seq(a, v, rows), rows, tile);
      n = block_units(k, extra);
    }
    before = block_exclusive_scan<THREADS>(n, sh, sum);
    run.total += sum;
  }
  run.total *= a.kv_heads;
  run.grid = min((int64_t)gridDim.x, run.total);
  const int64_t c = blockIdx.x;
  run.from = run.to = 0;
  if (c >= run.grid) return run;
  run.from = c * run.total / run.grid;
  run.to = (c + 1) * run.total / run.grid;
  int64_t passed = 0;
  for (int v0 = 0; v0 < nv && passed * a.kv_heads <= run.from; v0 += THREADS) {
    const int v = v0 + threadIdx.x;
    if (nv > THREADS) {  // (else as above)
      n = 0;
      if (v < nv) {
        k = block_of(a, v, block_seq(a, v, rows), rows, tile);
        n = block_units(k, extra);
      }
      before = block_exclusive_scan<THREADS>(n, sh, sum);
    }
    const int64_t first = (passed + before) * a.kv_heads, at = run.from - first;
    if (n > 0 && at >= 0 && at < (int64_t)n * a.kv_heads) {
      place->k = k;
      place->v = v;
      place->h = (int)(at / n);
      place->unit = (int)(at % n);
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
  int rows, v, h;
  int first, count;  // tiles of the block in the run
  int unit;
  int64_t left;      // units of the run from here on
  MOL_DEV void start(const Place& p, int rows_, int64_t n) {
    k = p.k;
    rows = rows_;
    v = p.v;
    h = p.h;
    unit = p.unit;
    left = n;
    cut();
  }
  MOL_DEV void cut() {
    const int n = (int)min((int64_t)(k.tiles + EXTRA - unit), left);
    first = max(unit - EXTRA, 0);
    count = max(unit + n - EXTRA, 0) - first;
  }
  MOL_DEV bool more() const { return left > 0; }
  MOL_DEV bool ends() const { return first + count >= k.tiles; }
  // On to the next head or block; ones that the run has no tile of are passed by.
  MOL_DEV void next(const AttnArgs& a, int nv) {
    do {
      left -= k.tiles + EXTRA - unit;
      if (left <= 0) return;
      unit = 0;
      if (++h == a.kv_heads) {
        h = 0;
        int b = k.b;
        do {
          if (++v >= nv) {
            left = 0;
            return;
          }
          while (b + 1 < a.num_seqs && first_block(a, b + 1, rows) <= v) ++b;
          k = block_of(a, v, b, rows, TILE);
        } while (k.tiles == 0);
      }
      cut();
    } while (count == 0);
  }
  // The last thread block that has a tile of this block, which the run begins and does not end.
  MOL_DEV int last(const Run& r) const {
    const int64_t end = r.to + (k.tiles - first - count);
    return (int)((end * r.grid + r.total - 1) / r.total) - 1;
  }
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
