// What the attention kernels share: sequences, their row blocks and key ranges, the joining of parts.
#pragma once

#include "mol_attend.h"
#include "mol_device.cuh"

namespace mol {

MOL_DEV int divide(int n, const Divider& d) {
  const uint32_t t = __umulhi(d.mul, (uint32_t)n);
  return (int)((t + (((uint32_t)n - t) >> d.s1)) >> d.s2);
}

namespace attn {

// A NaN or an infinity among eight bf16 values: an exponent of ones carries into the sign's place.
MOL_DEV bool not_finite(const uint4& q) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) c |= (w[i] & 0x7F807F80u) + 0x00800080u;
  return (c & 0x80008000u) != 0;
}

MOL_DEV void ldsm4(const void* p, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p))
               : "memory");
}
MOL_DEV void ldsm4_t(const void* p, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p))
               : "memory");
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
// Metadata and queries are read past L1: the kernel before may have written them while this one was already
// on the multiprocessor.
MOL_DEV int load_int(const int32_t* p) { return ld_cg_i32(p); }
MOL_DEV uint4 load_16(const void* p) {
  uint4 r;
  asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
}

// What the caller's arrays say of a sequence.
struct Given {
  int start, end, kv;
  MOL_DEV bool operator!=(const Given& o) const { return start != o.start || end != o.end || kv != o.kv; }
};
MOL_DEV Given given(const AttnArgs& a, int b) {
  Given g = {b, 0, 0};
  if (b >= a.num_seqs) return g;
  g.kv = load_int(a.kv_lens + b);
  if (a.q_starts) {
    g.start = load_int(a.q_starts + b);
    g.end = load_int(a.q_starts + b + 1);
  }
  return g;
}
// From its first row and what the arrays say of its end and its tokens. (Fewer than no rows: it ends before it
// begins, and has no blocks.)
MOL_DEV Seq sequence(const AttnArgs& a, int start, int end, int kv) {
  Seq s;
  s.start = start;
  s.n = a.q_starts ? min(max(end, 0), a.num_tokens) - start : 1;
  s.kv = min(max(kv, 0), a.max_pages * a.page_size);
  return s;
}
MOL_DEV Seq sequence(const AttnArgs& a, const Given& g) {
  return sequence(a, a.q_starts ? min(max(g.start, 0), a.num_tokens) : g.start, g.end, g.kv);
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
MOL_DEV int num_blocks(const AttnArgs& a, const Seq& s, int rows) {
  return (s.n * a.group + rows - 1) / rows;
}
MOL_DEV Block block_of(const AttnArgs& a, int b, const Seq& s, int r, int rows, int tile) {
  Block k;
  k.b = b;
  k.r = r;
  k.s = s;
  k.row0 = r * rows;
  k.nrows = min(s.n * a.group - k.row0, rows);
  const int i0 = divide(k.row0, a.by_group), i1 = divide(k.row0 + k.nrows - 1, a.by_group);
  const int shift = s.kv - s.n;
  k.hi = max(shift + i1 + 1, 0);
  k.lo = a.window > 0 ? max(shift + i0 - a.window + 1, 0) : 0;
  k.t0 = k.lo / tile;
  k.tiles = max((k.hi + tile - 1) / tile - k.t0, 1);
  return k;
}

// What a launch does is counted in units: a block's tiles and `extra` more for what it takes to begin
// and to end one; or blocks, where these go undivided. All units of the launch, in the order (sequence,
// block, head, unit), are dealt in even runs to its thread blocks.
MOL_DEV int units_of(const AttnArgs& a, const Block& k, int extra) { return a.whole ? 1 : k.tiles + extra; }

struct Place {  // where a thread block's run begins
  Block k;
  int h, unit;
};
struct Run {
  int64_t total, from, to;  // units of the launch, this thread block's
  int64_t share;            // units a thread block; the first `longer` ones have one more
  int longer;
  bool any;
  MOL_DEV int64_t begin(int c) const { return c * share + min(c, longer); }
  // The thread block that has the unit x behind this one's run.
  MOL_DEV int owner(uint32_t x) const {
    const int c = blockIdx.x + 1;
    const uint32_t one = (uint32_t)min(share, (int64_t)0x7fffffff);  // (more than any x)
    const int64_t span = c < longer ? (int64_t)(longer - c) * (share + 1) : 0;
    return x < span ? c + (int)(x / (one + 1)) : max(c, longer) + (int)((x - (uint32_t)span) / one);
  }
};

// Every thread of a thread block of THREADS calls it, with what the arrays said of the thread's sequence (whose
// blocks it goes through one by one: 2400 cycles for sequences of a block, 26 K for a prompt of 8192 tokens of
// 8 heads a key head in 256 blocks, 47 K for the 512 blocks of the form for 256 values);
// `sh` holds THREADS / 32 + 1 ints. *place is written where the run is not empty. A thread a sequence: one
// round trip for their lengths. (The kernels' code comes from memory when they start, so what is not hot is
// kept small.)
template <int THREADS>
MOL_DEV Run deal(const AttnArgs& a, const Given& mine, int rows, int tile, int extra, int* sh, Place* place) {
  if (threadIdx.x == 0) place->k.tiles = 0;
  Run run;
  Seq s = {};
  int blocks = 0, before = 0, sum = 0, n = 0;
  int64_t passed = 0;
  bool falls = false;
  run.total = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {  // the sum of all units, then where the run begins
#pragma unroll 1
    for (int b0 = 0; b0 < a.num_seqs; b0 += THREADS) {
      const int b = b0 + threadIdx.x;
      if (pass == 0 || a.num_seqs > THREADS) {
        n = blocks = 0;
        if (b < a.num_seqs) {
          s = sequence(a, a.num_seqs > THREADS ? given(a, b) : mine);
          falls |= s.n < 0;
          blocks = num_blocks(a, s, rows);
#pragma unroll 1
          for (int r = 0; r < blocks; ++r) n += units_of(a, block_of(a, b, s, r, rows, tile), extra);
        }
        before = block_exclusive_scan<THREADS>(n, sh, sum);
      }
      if (pass == 0) {
        run.total += sum;
        continue;
      }
      int64_t at = run.from - (passed + before) * a.kv_heads;
      passed += sum;
      if (at < 0 || at >= (int64_t)n * a.kv_heads) continue;
#pragma unroll 1
      for (int r = 0; r < blocks; ++r) {
        const Block k = block_of(a, b, s, r, rows, tile);
        const int u = units_of(a, k, extra);
        if (at < (int64_t)u * a.kv_heads) {
          place->k = k;
          place->h = at >> 32 ? (int)(at / u) : (int)((uint32_t)at / (uint32_t)u);
          place->unit = (int)(at - (int64_t)place->h * u);
          break;
        }
        at -= (int64_t)u * a.kv_heads;
      }
    }
    if (pass == 0) {
      // Starts that decrease: sequences overlap here and not in the walk, which goes on from where the last
      // one ended, so parts would be left to thread blocks past the last. Such a call has no units.
      if (a.q_starts && __syncthreads_or(falls)) run.total = 0;
      run.total *= a.kv_heads;  // (below 2^47; thread blocks below 2^9)
      const int high = divide((int)(run.total >> 20), a.by_grid);
      const int rest = ((int)(run.total >> 20) - high * (int)gridDim.x) << 20 | (int)(run.total & 0xfffff);
      const int low = divide(rest, a.by_grid);
      run.share = ((int64_t)high << 20) + low;
      run.longer = rest - low * (int)gridDim.x;
      run.from = run.begin(blockIdx.x);
      run.to = run.begin(blockIdx.x + 1);
      run.any = run.from < run.to;
      if (!run.any) break;
    }
  }
  __syncthreads();
  return run;
}

// The thread block's run, behind the wait for the kernel before. Short calls, whose blocks go undivided, deal
// already before it, from lengths that are most often what they will be, and read these again behind it:
// 4.5 us against 5.7 for 18 requests of a few tokens, one after the other. (Calls with parts lost where they
// follow each other: the kernel before is then a join, too short to hide it; 24 requests of up to 8191 tokens
// 20.2 us against 19.2. Behind another kernel, as the append in a layer, they were not timed.)
template <int THREADS>
MOL_DEV Run wait_and_deal(const AttnArgs& a, int rows, int tile, int extra, int* sh, Place* place) {
  bool waited = !a.whole || a.num_seqs > THREADS;
  if (waited) pdl_wait();
  Given mine = given(a, threadIdx.x);
  Run run;
#pragma unroll 1
  while (true) {
    run = deal<THREADS>(a, mine, rows, tile, extra, sh, place);
    if (waited) break;
    pdl_wait();
    waited = true;
    const Given now = given(a, threadIdx.x);
    if (!__syncthreads_or(now != mine)) break;
    mine = now;
  }
  pdl_launch_dependents();
  return run;
}

// Asks L2 for the page table, a line a thread over all thread blocks, while the runs are dealt: the first
// copies wait for their pages, which come from memory otherwise. (Of a larger table its beginning.)
template <int THREADS>
MOL_DEV void prefetch_table(const AttnArgs& a) {
  const int64_t at = ((int64_t)blockIdx.x * THREADS + threadIdx.x) * 32;
  const int64_t all = a.max_pages > 0 ? (int64_t)(a.num_seqs - 1) * a.table_stride + a.max_pages : 0;
  if (at < all) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.page_table + at));
}

// Cached tokens whose products one sum takes. A matrix instruction cuts what does not fit its fp32 sum, so a
// sum of like signs falls short by 2^-24 or so an instruction of 16 tokens: 2^-8.5 a million, more than half of
// a bf16 step. Behind 2^16 (2^-12.5) the sum goes to memory and a fresh one is begun, to be added in fp32.
constexpr int kStretch = 1 << 16;
// Whether a block may see more, for which the kernels have a form of their own: with what it takes to go on
// and to add, the others would be slower (a prompt of 8192 434 us against 425, mixed batches 104 against 99).
bool beyond_a_stretch(const AttnArgs& a, int rows, int tile);

// A walk over a thread block's run, a block's head at a time, with LONG of a long block a stretch at a time.
template <bool LONG>
struct Walk {
  Block k;
  int h;
  int first, count;  // tiles of the block, or of a stretch of it
  int from;          // the block's first tile in the run (LONG)
  int unit;
  int64_t left;      // units of the run from here on
  int kv1, end1;     // what the caller's arrays say of the sequence behind this one, asked for ahead
  MOL_DEV bool more() const { return left > 0; }
  MOL_DEV bool begins() const { return (LONG ? from : first) == 0; }
  MOL_DEV bool ends() const { return first + count >= k.tiles; }
  MOL_DEV bool joins() const { return LONG && first > from; }  // a stretch behind another one
  MOL_DEV int taken(int extra) const { return first + count + extra - unit; }  // units of the stretch
  MOL_DEV bool stays(int extra) const { return LONG && !ends() && left > taken(extra); }  // another one behind it
  // The last thread block that has a tile of this block, which the run begins and does not end.
  MOL_DEV int last(const Run& r) const { return r.owner((uint32_t)(k.tiles - first - count) - 1); }
};
template <bool LONG>
MOL_DEV void cut(const AttnArgs& a, Walk<LONG>& w, int tile, int extra) {
  if (a.whole) {
    w.first = 0;
    w.count = w.k.tiles;
    return;
  }
  const int n = (int)min((int64_t)(w.k.tiles + extra - w.unit), w.left);
  w.first = max(w.unit - extra, 0);
  w.count = max(w.unit + n - extra, 0) - w.first;
  if (LONG) w.count = min(w.count, kStretch / tile);
}
template <bool LONG>
MOL_DEV void peek(const AttnArgs& a, Walk<LONG>& w) {
  w.kv1 = w.end1 = 0;
  if (w.k.b + 1 >= a.num_seqs) return;
  w.kv1 = load_int(a.kv_lens + w.k.b + 1);
  if (a.q_starts) w.end1 = load_int(a.q_starts + w.k.b + 2);
}
// On to the next stretch, head or block; ones that the run has no tile of are passed by.
template <bool LONG>
MOL_DEV void go_on(const AttnArgs& a, Walk<LONG>& w, int rows, int tile, int extra) {
  if (w.stays(extra)) {
    const int n = w.taken(extra);
    w.left -= n;
    w.unit += n;
    cut(a, w, tile, extra);
    return;
  }
  w.from = 0;
#pragma unroll 1
  do {
    w.left -= units_of(a, w.k, extra) - w.unit;
    if (w.left <= 0) return;
    w.unit = 0;
    if (++w.h == a.kv_heads) {
      w.h = 0;
      int r = w.k.r + 1;
#pragma unroll 1
      while (r >= num_blocks(a, w.k.s, rows)) {
        if (++w.k.b >= a.num_seqs) {
          w.left = 0;
          return;
        }
        w.k.s = sequence(a, w.k.s.start + w.k.s.n, w.end1, w.kv1);
        peek(a, w);
        r = 0;
      }
      w.k = block_of(a, w.k.b, w.k.s, r, rows, tile);
    }
    cut(a, w, tile, extra);
  } while (w.count == 0);
}
template <bool LONG>
MOL_DEV void begin(const AttnArgs& a, Walk<LONG>& w, const Place& p, const Run& run, int rows, int tile,
                   int extra) {
  w.k = p.k;
  w.h = p.h;
  w.unit = p.unit;
  w.left = p.k.tiles > 0 ? run.to - run.from : 0;  // (0: lengths that changed under the call)
  if (w.left == 0) return;
  peek(a, w);
  cut(a, w, tile, extra);
  w.from = w.first;
  if (w.count == 0) go_on(a, w, rows, tile, extra);
}

// Parts of blocks that several thread blocks share. Thread block c leaves the part that continues its
// predecessor's block in slot 2c, the one that it begins and does not end in slot 2c + 1 (its last one, so until
// then the stretches of others that it begins meet there) with a record of it: last thread block of it (-1: there is none), the sequence's first row of q, first row
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

// Whether blocks go undivided, which needs no join: where none has more than `tiles` tiles.
bool undivided(const AttnArgs& a, int rows, int tile, int tiles);

// The device's SMs, at most 152, and the most thread blocks that a launch's parts are laid out for.
int sms();
constexpr int kMaxGrid = 2 * 152;

// Many rows a sequence (mol_attend_tc.cu): 64 or 128 values a head.
size_t many_bytes(int group, int head_dim);
cudaError_t prepare_many();
cudaError_t launch_many(const AttnArgs& a, cudaStream_t stream);
// Many rows a sequence of 256 values a head (mol_attend_wide.cu).
size_t wide_bytes();
cudaError_t prepare_wide();
cudaError_t launch_wide(const AttnArgs& a, cudaStream_t stream);

}  // namespace attn
}  // namespace mol
