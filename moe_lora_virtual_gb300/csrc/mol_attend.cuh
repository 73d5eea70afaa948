// What the attention kernels share: sequences, their row blocks and key ranges, the joining of parts.
#pragma once

#include "mol_attend.h"
#include "mol_device.cuh"

namespace mol {
namespace attn {

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

// Where a part of the tiles begins: block number, head, tile of it.
struct Place {
  int v, h, tile;
};

// All tiles of the launch, in the order (block, head, tile), are dealt in even runs. total: tiles of
// one head. Every thread of a thread block of THREADS calls these; `sh` holds THREADS / 32 + 1 ints.
template <int THREADS>
MOL_DEV int64_t count_tiles(const AttnArgs& a, int rows, int tile, int* sh) {
  const int nv = num_blocks(a, rows);
  int64_t total = 0;
  for (int v0 = 0; v0 < nv; v0 += THREADS) {
    const int v = v0 + threadIdx.x;
    const int n = v < nv ? block_of(a, v, block_seq(a, v, rows), rows, tile).tiles : 0;
    int here;
    block_exclusive_scan<THREADS>(n, sh, here);
    total += here;
  }
  return total;
}
template <int THREADS>
MOL_DEV void find_tile(const AttnArgs& a, int rows, int tile, int64_t at, int* sh, Place* out) {
  const int nv = num_blocks(a, rows);
  int64_t passed = 0;
  for (int v0 = 0; v0 < nv && passed * a.kv_heads <= at; v0 += THREADS) {
    const int v = v0 + threadIdx.x;
    const int n = v < nv ? block_of(a, v, block_seq(a, v, rows), rows, tile).tiles : 0;
    int total;
    const int before = block_exclusive_scan<THREADS>(n, sh, total);
    const int64_t first = (passed + before) * a.kv_heads;
    if (n > 0 && at >= first && at < first + (int64_t)n * a.kv_heads) {
      out->v = v;
      out->h = (int)((at - first) / n);
      out->tile = (int)((at - first) % n);
    }
    passed += total;
  }
  __syncthreads();
}

// A walk over a thread block's run of tiles.
template <int TILE>
struct Walk {
  Block k;
  int rows, v, h, tile;
  int64_t left;  // tiles of the run from here on
  MOL_DEV void start(const AttnArgs& a, int rows_, const Place& p, int64_t n) {
    rows = rows_;
    v = p.v;
    h = p.h;
    tile = p.tile;
    left = n;
    k = block_of(a, v, block_seq(a, v, rows), rows, TILE);
  }
  // On to the next tile; true where that is another block's or head's, or none.
  MOL_DEV bool next(const AttnArgs& a, int nv) {
    if (--left <= 0) return true;
    if (++tile < k.tiles) return false;
    advance(a, nv);
    return true;
  }
  // On to the first tile of the next block or head.
  MOL_DEV void advance(const AttnArgs& a, int nv) {
    tile = 0;
    if (++h < a.kv_heads) return;
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
};

// Parts of blocks that several thread blocks share. Thread block c leaves the part that continues its
// predecessor's block in slot 2c, the one that it begins and does not end in slot 2c + 1 with a
// record of it: {last thread block of it, sequence, first row, head}, {-1} where there is none.
struct Record {
  int last, b, row0, h;
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
