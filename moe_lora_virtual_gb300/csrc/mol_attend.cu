// Attention of few new tokens over the paged cache (include/mol_attn.h).

#include <algorithm>

#include "mol_attend.cuh"
#include "mol_internal.h"

namespace mol {
namespace {

using attn::Block;
using attn::Parts;
using attn::Place;
using attn::Record;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kExtra = 1;             // units that a block takes beside its tiles

using attn::ldsm4;
using attn::ldsm4_t;

template <int D, int MT>
struct Geo {
  static constexpr int kRows = 16 * MT;
  static constexpr int kStep = D == 64 ? 32 : 16;        // tokens a warp takes at a time
  static constexpr int kTile = kWarps * kStep;
  static constexpr int kStages = 3;
  static constexpr int kTileBytes = kStep * D * 2;       // keys, or values, of a step
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr size_t kSmem = (size_t)kRing + kRows * D * 2;  // and the queries
  // A warp's sums go to the ring stage it has just taken, for the others to add.
  static_assert(kRows * D * 4 <= kStageBytes, "sums that meet");
  static constexpr int kPerSM = kSmem <= 113 * 1024 ? 2 : 1;
  static constexpr bool kQueriesInRegisters = MT * D <= 128;
};

// Few rows (new tokens x group) against long runs of keys: the cache is read once, and that is what
// bounds it. All tiles of 64 tokens (128 for 64 values a head) of the launch, over sequences, heads and row
// blocks, are one list dealt in even runs to thread blocks, so sequences of any lengths fill the GPU alike;
// a block whose tiles fall to several leaves parts that launch_join adds in order. In a tile each warp has 16
// (32) tokens of its own, with a cp.async ring of its own that runs on across the blocks' borders (keys and
// values asked for two steps ahead, no barrier between warps), its own maximum, sum and fp32
// accumulators; the warps meet where a block ends. Scores: mma.sync with the rows as the 16-row side.
// Tokens that lie on no page, or past the sequence, are zero in shared memory, whatever memory
// holds; where a row does not see a token that another one sees, the step's values are looked
// through, and summed without the tensor cores should one not be finite (0 * NaN is NaN there). LONG: blocks
// that may see more than kStretch tokens, their stretches added up in the slot of the block's part.
// 4 sequences of 131072, one new token each, 64 heads of 128 on 8: 322 us, 6.67 TB/s (0.98 of a copy's rate);
// 24 of up to 8191, 16 heads on 2: 19.7 us, 3.3 TB/s. What a call takes beside its stream: the deal 1.7 us,
// pages and first copies 1.2, their data 1.3, a step 0.7, the warps' sums 0.8, the join 2.3.
template <int D, int MT, bool LONG>
__global__ void __launch_bounds__(kThreads, Geo<D, MT>::kPerSM)
    attend_few_kernel(const __grid_constant__ AttnArgs a) {
  using G = Geo<D, MT>;
  constexpr int kChunks = D / 8;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int s_scan[kWarps + 1];
  __shared__ Place s_place;
  __shared__ uint32_t s_held[kWarps][G::kStages];
  __shared__ float2 s_top[kWarps][G::kRows];
  __shared__ float2 s_met[LONG ? 2 : 1][G::kRows];  // maxima and sums of a block's stretches so far, of even and odd ones
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* ring = smem + warp * (G::kStages * G::kStageBytes);
  unsigned char* shared = smem + G::kRing;

  attn::prefetch_table<kThreads>(a);
  const attn::Run run = attn::wait_and_deal<kThreads>(a, G::kRows, G::kTile, kExtra, s_scan, &s_place);
  const Parts parts = attn::parts(a.workspace, gridDim.x, G::kRows, D);
  const int64_t c = blockIdx.x;
  if (!run.any) {
    if (tid == 0) parts.records[c].last = -1;
    return;
  }
  constexpr int kStep = G::kStep;
  attn::Walk<LONG> load, work;  // over the run, of the copies and of the products
  attn::begin(a, load, s_place, run, G::kRows, G::kTile, kExtra);
  work = load;
  int load_tile = 0;  // of load.count

  // Where this lane's token of a step lies: its page is asked for two steps before its copies are.
  struct Token {
    int page, offset, h;  // (page -1: no row sees the token)
  };
  auto look = [&]() {
    Token t = {-1, 0, load.h};
    if (!load.more()) return t;
    const int j = (load.k.t0 + load.first + load_tile) * G::kTile + warp * kStep + lane % kStep;
    if (j >= load.k.lo && j < load.k.hi) {
      const int p = divide(j, a.by_page);
      if (MOL_CHECK(p >= 0 && p < a.max_pages, MOL_CHECK_COLUMN, p))
        t.page = attn::load_int(a.page_table + load.k.b * a.table_stride + p);
      t.offset = j - p * a.page_size;
    }
    if (++load_tile == load.count) {
      attn::go_on(a, load, G::kRows, G::kTile, kExtra);
      load_tile = 0;
    }
    return t;
  };
  Token ahead[2] = {{-1, 0, 0}, {-1, 0, 0}};
  // Asks for the next step into ring stage s; for a negative one only for its pages.
  auto fetch = [&](int s) {
    const Token t = ahead[0];
    ahead[0] = ahead[1];
    ahead[1] = look();
    if (s < 0) return;
    const bool held = t.page >= 0 && t.page < a.num_pages;
    const int64_t at = held ? t.page * a.page_stride + t.offset * a.token_stride + t.h * a.head_stride : 0;
    const uint32_t mask = __ballot_sync(0xffffffffu, held);
    if (lane == 0) s_held[warp][s] = mask;
    unsigned char* st = ring + s * G::kStageBytes;
#pragma unroll
    for (int i = 0; i < kStep * kChunks / 32; ++i) {
      const int idx = i * 32 + lane, row = idx / kChunks, ch = idx % kChunks;
      const int64_t from_row = __shfl_sync(0xffffffffu, at, row) + ch * 8;
      const uint32_t n = (mask >> row) & 1 ? 16u : 0u;
      unsigned char* d = st + row * (D * 2) + ((ch ^ (row & 7)) << 4);
      cp_async16_zfill(d, a.k + from_row, n);
      cp_async16_zfill(d + G::kTileBytes, a.v + from_row, n);
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int s = -2; s < G::kStages - 1; ++s) fetch(s);

  const int g = lane >> 2, t4 = lane & 3;
  int stage = 0;
  // A block's queries are asked for while the block before it ends.
  constexpr int kQueries = G::kRows * kChunks / kThreads;
  uint4 query[kQueries];
  auto ask_queries = [&](const Block& k, int h) {
#pragma unroll
    for (int i = 0; i < kQueries; ++i) {
      const int row = (i * kThreads + tid) / kChunks, ch = (i * kThreads + tid) % kChunks;
      query[i] = make_uint4(0, 0, 0, 0);
      if (row < k.nrows) {
        const int r = k.row0 + row, token = divide(r, a.by_group);
        if (MOL_CHECK(k.s.start + token < a.num_tokens, MOL_CHECK_ROW, k.s.start + token))
          query[i] = attn::load_16(a.q + (int64_t)(k.s.start + token) * a.q_token_stride +
                                   (int64_t)(h * a.group + r - token * a.group) * a.q_head_stride + ch * 8);
      }
    }
  };
  auto put_queries = [&]() {
#pragma unroll
    for (int i = 0; i < kQueries; ++i) {
      const int row = (i * kThreads + tid) / kChunks, ch = (i * kThreads + tid) % kChunks;
      *reinterpret_cast<uint4*>(shared + row * (D * 2) + ((ch ^ (row & 7)) << 4)) = query[i];
    }
  };
  Record record = {};
  record.last = -1;
  if (work.more()) ask_queries(work.k, work.h);
#pragma unroll 1
  while (work.more()) {
    // ------------------------------------------------------------ a block of rows and a head
    const Block k = work.k;
    const int h = work.h, first = work.first, count = work.count;
    put_queries();
    __syncthreads();
    auto load_q = [&](int mt, int kk, uint32_t (&r)[4]) {
      const int row = mt * 16 + (lane & 15), ch = 2 * kk + (lane >> 4);
      ldsm4(shared + row * (D * 2) + ((ch ^ (row & 7)) << 4), r);
    };
    uint32_t qf[G::kQueriesInRegisters ? MT : 1][G::kQueriesInRegisters ? D / 16 : 1][4];
    if constexpr (G::kQueriesInRegisters) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) load_q(mt, kk, qf[mt][kk]);
    }
    // the positions of this lane's rows; of the block's first and last row
    int pos[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        pos[mt][i] = k.s.kv - k.s.n + divide(k.row0 + min(mt * 16 + g + 8 * i, k.nrows - 1), a.by_group);
    const int pos_first = k.s.kv - k.s.n + divide(k.row0, a.by_group);
    const int pos_last = k.s.kv - k.s.n + divide(k.row0 + k.nrows - 1, a.by_group);

    float o[MT][D / 8][4];
    float top[MT][2], sum[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      top[mt][0] = top[mt][1] = -INFINITY;
      sum[mt][0] = sum[mt][1] = 0.f;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.f;
    }
#pragma unroll 1
    for (int tile = first; tile < first + count; ++tile) {
      cp_async_wait_group<G::kStages - 2>();
      __syncwarp();  // the step has landed, and the stage before it is free, for every lane
      fetch(stage == 0 ? G::kStages - 1 : stage - 1);
      const unsigned char* kt = ring + stage * G::kStageBytes;
      const unsigned char* vt = kt + G::kTileBytes;
      constexpr uint32_t kAll = kStep == 32 ? 0xffffffffu : (1u << kStep) - 1;
      constexpr int kNT = kStep / 8;
      const uint32_t mask = s_held[warp][stage] & kAll;
      const int j0 = (k.t0 + tile) * G::kTile + warp * kStep;
      if (mask != 0) {
        float s[MT][kNT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < kNT; ++n) s[mt][n][0] = s[mt][n][1] = s[mt][n][2] = s[mt][n][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t b[kNT / 2][4];
#pragma unroll
          for (int n = 0; n < kNT / 2; ++n) {
            const int row = n * 16 + (lane & 7) + ((lane >> 4) << 3), ch = 2 * kk + ((lane >> 3) & 1);
            ldsm4(kt + row * (D * 2) + ((ch ^ (row & 7)) << 4), b[n]);
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t q[4];
            if constexpr (G::kQueriesInRegisters) {
#pragma unroll
              for (int i = 0; i < 4; ++i) q[i] = qf[mt][kk][i];
            } else {
              load_q(mt, kk, q);
            }
#pragma unroll
            for (int n = 0; n < kNT; ++n)
              mma_16816(s[mt][n], q[0], q[1], q[2], q[3], b[n / 2][n % 2 * 2], b[n / 2][n % 2 * 2 + 1]);
          }
        }
        // every row sees every token of the step, or not
        const bool edge = mask != kAll || j0 + kStep - 1 > pos_first ||
                          (a.window > 0 && j0 <= pos_last - a.window);
        auto sees = [&](int j, int p) {
          return ((mask >> (j - j0)) & 1) && j <= p && (a.window == 0 || j > p - a.window);
        };
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < kNT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s[mt][n][e] *= a.scale_log2;
              if (edge && !sees(j0 + n * 8 + 2 * t4 + (e & 1), pos[mt][e >> 1])) s[mt][n][e] = -INFINITY;
            }
        uint32_t p[MT][kStep / 16][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float m = s[mt][0][2 * i];
#pragma unroll
            for (int n = 0; n < kNT; ++n) m = fmaxf(m, fmaxf(s[mt][n][2 * i], s[mt][n][2 * i + 1]));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const float was = top[mt][i];
            if (__any_sync(0xffffffffu, m > was)) {
              const float now = fmaxf(was, m);
              const float f = was == now ? 1.f : attn::ex2(was - now);  // (-inf before the first)
              top[mt][i] = now;
              sum[mt][i] *= f;
#pragma unroll
              for (int n = 0; n < D / 8; ++n) {
                o[mt][n][2 * i] *= f;
                o[mt][n][2 * i + 1] *= f;
              }
            }
            // a row that has seen nothing yet keeps weights of 0: 2^-inf
            const float base = top[mt][i] == -INFINITY ? 0.f : top[mt][i];
#pragma unroll
            for (int n = 0; n < kNT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float w = attn::ex2(s[mt][n][2 * i + e] - base);
                s[mt][n][2 * i + e] = w;
                sum[mt][i] += w;
              }
          }
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            p[mt][n / 2][n % 2 * 2] = pack_bf16x2(s[mt][n][0], s[mt][n][1]);
            p[mt][n / 2][n % 2 * 2 + 1] = pack_bf16x2(s[mt][n][2], s[mt][n][3]);
          }
        }
        bool plain = false;
        if (edge) {
          bool bad = false;
#pragma unroll 4
          for (int i = lane; i < kStep * kChunks; i += 32) {
            bad |= attn::not_finite(lds16(vt + i * 16));
          }
          plain = __any_sync(0xffffffffu, bad);
        }
        if (!plain) {
#pragma unroll
          for (int x = 0; x < kStep / 16; ++x)
#pragma unroll
            for (int n2 = 0; n2 < D / 16; ++n2) {
              uint32_t b[4];
              const int row = x * 16 + (lane & 15), ch = 2 * n2 + (lane >> 4);
              ldsm4_t(vt + row * (D * 2) + ((ch ^ (row & 7)) << 4), b);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                const uint32_t(&w)[4] = p[mt][x];
                mma_16816(o[mt][2 * n2], w[0], w[1], w[2], w[3], b[0], b[1]);
                mma_16816(o[mt][2 * n2 + 1], w[0], w[1], w[2], w[3], b[2], b[3]);
              }
            }
        } else {
#pragma unroll
          for (int x = 0; x < kStep / 16; ++x)
#pragma unroll 1
            for (int i = 0; i < 16; ++i) {
              const int at = x * 16 + i, j = j0 + at, from_lane = (lane & ~3) | ((i & 7) >> 1);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                float w[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  const uint32_t pair = i < 8 ? p[mt][x][r] : p[mt][x][2 + r];
                  const uint32_t got = __shfl_sync(0xffffffffu, pair, from_lane);
                  w[r] = i & 1 ? bf16_hi(got) : bf16_lo(got);
                }
                const bool see[2] = {sees(j, pos[mt][0]), sees(j, pos[mt][1])};
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                  const uint32_t v = *reinterpret_cast<const uint32_t*>(vt + at * (D * 2) +
                                                                        ((n ^ (at & 7)) << 4) + 4 * t4);
                  const float v0 = bf16_lo(v), v1 = bf16_hi(v);
#pragma unroll
                  for (int r = 0; r < 2; ++r)
                    if (see[r]) {
                      o[mt][n][2 * r] += w[r] * v0;
                      o[mt][n][2 * r + 1] += w[r] * v1;
                    }
                }
              }
            }
        }
      }
      stage = stage + 1 == G::kStages ? 0 : stage + 1;
    }

    // ------------------------------------------------------------ the warps' sums become one
    const bool begins = work.begins(), joins = work.joins(), stays = work.stays(kExtra);
    const bool part = stays || !begins || !work.ends();
    const int slot = (int)(2 * c) + (begins ? 1 : 0);
    const int odd = LONG ? (first - work.from) / (attn::kStretch / G::kTile) & 1 : 0;
    const int start = k.s.start, row0 = k.row0, nrows = k.nrows;
    if (begins && part && !stays && tid == 0) record = {work.last(run), start, row0, nrows, h, {}};
    attn::go_on(a, work, G::kRows, G::kTile, kExtra);
    if (work.more()) ask_queries(work.k, work.h);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float l = sum[mt][i];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (t4 == 0) s_top[warp][mt * 16 + g + 8 * i] = make_float2(top[mt][i], l);
      }
    // Each in the stage that the next copies go to; the 32-byte pieces of a row in another order for
    // each row, so that a store's rows do not fall on the same banks.
    const int free_stage = stage == 0 ? G::kStages - 1 : stage - 1;
    unsigned char* mine = ring + free_stage * G::kStageBytes;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          *reinterpret_cast<float2*>(mine + (mt * 16 + g + 8 * i) * (D * 4) + ((n ^ g) << 5) +
                                     t4 * 8) = make_float2(o[mt][n][2 * i], o[mt][n][2 * i + 1]);
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < G::kRows * (D / 4); i += kThreads) {
      const int row = i / (D / 4), col = i % (D / 4) * 4;
      if (row >= nrows) break;
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_top[w][row].x);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {  // (in this order, whatever the timing)
        const float2 t = s_top[w][row];
        const float f = t.x == -INFINITY ? 0.f : attn::ex2(t.x - m);
        const float4 y = *reinterpret_cast<const float4*>(
            smem + (w * G::kStages + free_stage) * G::kStageBytes + row * (D * 4) +
            (((col >> 3) ^ (row & 7)) << 5) + (col & 4) * 4);
        l += f * t.y;
        x.x += f * y.x;
        x.y += f * y.y;
        x.z += f * y.z;
        x.w += f * y.w;
      }
      float4* const met = reinterpret_cast<float4*>(parts.sums + ((int64_t)slot * G::kRows + row) * D + col);
      if (joins) {  // (the thread's own values of the stretch before)
        const float2 t = s_met[odd ^ 1][row];
        const float4 y = *met;
        const float most = fmaxf(m, t.x), base = most == -INFINITY ? 0.f : most;
        const float f = attn::ex2(t.x - base), own = attn::ex2(m - base);
        m = most;
        l = f * t.y + own * l;
        x = make_float4(f * y.x + own * x.x, f * y.y + own * x.y, f * y.z + own * x.z, f * y.w + own * x.w);
      }
      if (kChecked && !MOL_CHECK(start + divide(row0 + row, a.by_group) < a.num_tokens, MOL_CHECK_ROW,
                                 start + divide(row0 + row, a.by_group)))
        continue;
      if (part) {
        *met = x;
        if (col == 0) (stays ? s_met[odd][row] : parts.tops[slot * G::kRows + row]) = make_float2(m, l);
      } else {
        const int r = row0 + row, token = divide(r, a.by_group);
        const float inv = m == -INFINITY ? 0.f : 1.f / l;
        *reinterpret_cast<uint2*>(a.out + (int64_t)(start + token) * a.out_token_stride +
                                  (int64_t)(h * a.group + r - token * a.group) * a.out_head_stride +
                                  col) =
            make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
      }
    }
    __syncthreads();
  }
  cp_async_wait_all();
  if (tid == 0) parts.records[c] = record;
}

constexpr int kJoinWarps = 8;

// WAYS warps a row, its columns over their lanes: each takes every WAYS-th part, and the first adds what
// they have. Every part is read once; a launch and two round trips (record, parts) are what it costs.
template <int D, int WAYS>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(AttnArgs a, int rows, Parts p) {
  constexpr int kPer = D / 32;  // columns a lane
  constexpr int kRows = kJoinWarps / WAYS;
  __shared__ float s_sum[WAYS > 1 ? kRows : 1][WAYS][D];
  __shared__ float2 s_top[kRows][WAYS];
  pdl_wait();
  pdl_launch_dependents();
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int local = warp / WAYS, way = warp % WAYS, row = blockIdx.y * kRows + local;
  const Record rec = p.records[c];
  if (rec.last >= 0)
    (void)MOL_CHECK(rec.last > c && rec.last < (int)gridDim.x, MOL_CHECK_ROW, rec.last);
  if (rec.last < 0 || (int)blockIdx.y * kRows >= rec.nrows) return;
  const bool has = row < rec.nrows;
  float x[kPer], l = 0.f, m = -INFINITY;
#pragma unroll
  for (int e = 0; e < kPer; ++e) x[e] = 0.f;
  if (has) {
    // (maxima and sums of four parts asked for together)
#pragma unroll 1
    for (int i0 = c + way; i0 <= rec.last; i0 += 4 * WAYS) {
      float2 t[4], v[4][kPer / 2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + j * WAYS;
        const int64_t at = (int64_t)(2 * i + (i == c)) * rows + row;
        t[j] = i <= rec.last ? p.tops[at] : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < kPer / 2; ++e)
          v[j][e] = i <= rec.last ? reinterpret_cast<const float2*>(p.sums + at * D + lane * kPer)[e]
                                  : make_float2(0.f, 0.f);
      }
      float now = m;
#pragma unroll
      for (int j = 0; j < 4; ++j) now = fmaxf(now, t[j].x);
      const float base = now == -INFINITY ? 0.f : now, f = attn::ex2(m - base);
      m = now;
      l *= f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) x[e] *= f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float fj = attn::ex2(t[j].x - base);
        l += fj * t[j].y;
#pragma unroll
        for (int e = 0; e < kPer / 2; ++e) {
          x[2 * e] += fj * v[j][e].x;
          x[2 * e + 1] += fj * v[j][e].y;
        }
      }
    }
  }
  if constexpr (WAYS > 1) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) s_sum[local][way][lane * kPer + e] = x[e];
    if (lane == 0) s_top[local][way] = make_float2(m, l);
    __syncthreads();
    if (way > 0) return;
#pragma unroll
    for (int w = 0; w < WAYS; ++w) m = fmaxf(m, s_top[local][w].x);
    const float base = m == -INFINITY ? 0.f : m;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) x[e] = 0.f;
#pragma unroll
    for (int w = 0; w < WAYS; ++w) {
      const float f = attn::ex2(s_top[local][w].x - base);
      l += f * s_top[local][w].y;
#pragma unroll
      for (int e = 0; e < kPer; ++e) x[e] += f * s_sum[local][w][lane * kPer + e];
    }
  }
  if (!has) return;
  const int r = rec.row0 + row, token = divide(r, a.by_group);
  const float inv = m == -INFINITY ? 0.f : 1.f / l;
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + (int64_t)(rec.start + token) * a.out_token_stride +
                                              (int64_t)(rec.h * a.group + r - token * a.group) *
                                                  a.out_head_stride) + lane * (kPer / 2);
#pragma unroll
  for (int e = 0; e < kPer; e += 2) dst[e / 2] = pack_bf16x2(x[e] * inv, x[e + 1] * inv);
}

template <int D, int MT>
cudaError_t attend_few(const AttnArgs& args, cudaStream_t stream) {
  using G = Geo<D, MT>;
  const int grid = attn::sms() * G::kPerSM;
  AttnArgs a = args;
  a.by_grid = divider(grid);
  // Up to four tiles (two of wide heads) one after the other take no longer than parts and their join: one
  // request of 120 tokens, 16 heads of 128 on 2, 5.8 us against 8.5, of 250 7.7 against 8.7.
  a.whole = attn::undivided(a, G::kRows, G::kTile, D == 256 ? 2 : 4);
  auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(grid), dim3(kThreads), G::kSmem, stream, a); };
  const cudaError_t e = attn::beyond_a_stretch(a, G::kRows, G::kTile) ? go(attend_few_kernel<D, MT, true>)
                                                                     : go(attend_few_kernel<D, MT, false>);
  if (e != cudaSuccess || a.whole) return e;
  return attn::launch_join(a, grid, G::kRows, attn::parts(a.workspace, grid, G::kRows, D), stream);
}

template <int D, int MT>
cudaError_t prepare() {
  auto set = [](auto kernel) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Geo<D, MT>::kSmem);
  };
  const cudaError_t e = set(attend_few_kernel<D, MT, false>);
  return e != cudaSuccess ? e : set(attend_few_kernel<D, MT, true>);
}

}  // namespace

int attn::sms() {
  static const int n = [] {
    int dev = 0, v = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0)
      v = 152;
    return std::min(v, 152);
  }();
  return n;
}

// Cached tokens that a block's rows see together, at most.
static int64_t most_tokens(const AttnArgs& a, int rows, int tile) {
  const int64_t tokens = (int64_t)a.max_pages * a.page_size;
  // (a window's rows see so many, and a tile's beginning is theirs by chance)
  return a.window > 0 ? std::min<int64_t>(tokens, (int64_t)a.window + rows / a.group + tile) : tokens;
}
bool attn::undivided(const AttnArgs& a, int rows, int tile, int tiles) {
  return most_tokens(a, rows, tile) <= (int64_t)tiles * tile;
}
bool attn::beyond_a_stretch(const AttnArgs& a, int rows, int tile) {
  return most_tokens(a, rows, tile) > kStretch;
}

cudaError_t attn::launch_join(const AttnArgs& a, int grid, int rows, const Parts& p,
                              cudaStream_t stream) {
  // Few rows come in many parts (a sequence of 128 K tokens: 38), many rows in two or three.
  constexpr int kWays = 4;
  const bool few = rows <= 32;
  const int per = few ? kJoinWarps / kWays : kJoinWarps;
  const dim3 g(grid, (rows + per - 1) / per), block(kJoinWarps * 32);
  auto go = [&](auto kernel) { return launch_pdl(kernel, g, block, 0, stream, a, rows, p); };
  if (a.head_dim == 64) return few ? go(join_kernel<64, kWays>) : go(join_kernel<64, 1>);
  if (a.head_dim == 128) return few ? go(join_kernel<128, kWays>) : go(join_kernel<128, 1>);
  return few ? go(join_kernel<256, kWays>) : go(join_kernel<256, 1>);
}

cudaError_t prepare_attn_kernels() {
  cudaError_t e = prepare<64, 1>();
  if (e == cudaSuccess) e = prepare<64, 2>();
  if (e == cudaSuccess) e = prepare<128, 1>();
  if (e == cudaSuccess) e = prepare<256, 1>();
  if (e == cudaSuccess) e = attn::prepare_many();
  if (e == cudaSuccess) e = attn::prepare_wide();
  return e;
}

// The form for the rows (new tokens x group) that a sequence has on average, all that the host knows: one
// launch for all sequences, whatever each has. Measured with 8 key heads, group 1 to 8, 4 to 100 sequences
// (us for attend_few in blocks of 16 rows | of 32 | attend_many; 16 sequences of 4000 tokens):
//   64 values a head:  12 rows 32 | 40 | 54, 16 rows 33 | 40 | 54, 24 rows 49 | 41 | 54, 48 rows 65 | 68 | 55
//   128 values:        12 rows 52 | 66 | 61, 16 rows 52 | 66 | 61, 24 rows 91 | 68 | 61, 48 rows 131 | 119 | 62
// A call with both of decoding sequences and prompts pays: 200 rows of one sequence in blocks of 16 read its
// keys 13 times (from L2). 256 requests of 1000 to 4315 tokens and a chunk of 512 over 30000, 32 heads of 128 on
// 8, take 2014 us (12 rows on average), in two calls 419 + 183; with 100 requests the average is 24 rows and the
// call takes 313. 256 values a head, 2 key heads (us for attend_few | attend_wide): one sequence of
// 2000 tokens, 32 rows 15 | 22, 128 rows 20 | 32; 8 of them, 32 rows each 25 | 29, 64 rows 37 | 34, 128 rows
// 60 | 45; 200 new of 300 tokens, 1600 rows 31 | 24; 2048 tokens 590 | 202.
enum class Form { kFew16, kFew32, kMany, kWide };
static Form form(int64_t num_seqs, int64_t rows, int head_dim) {
  if (rows <= 16 * num_seqs) return Form::kFew16;
  if (head_dim == 256) return rows <= std::max<int64_t>(64 * num_seqs, 256) ? Form::kFew16 : Form::kWide;
  return head_dim == 64 && rows <= 32 * num_seqs ? Form::kFew32 : Form::kMany;
}

static size_t bytes_of(Form f, int group, int head_dim) {
  return f == Form::kMany   ? attn::many_bytes(group, head_dim)
         : f == Form::kWide ? attn::wide_bytes()
                          : attn::parts_bytes(attn::kMaxGrid, f == Form::kFew32 ? 32 : 16, head_dim);
}
size_t attn_workspace_bytes(int64_t num_seqs, int64_t num_tokens, int group, int head_dim) {
  if (num_seqs <= 0 || num_tokens <= 0) return 0;
  return bytes_of(form(num_seqs, num_tokens * group, head_dim), group, head_dim);
}
// A form for more rows takes more scratch, and of at most so many sequences and tokens it is one sequence
// with all the tokens that has the most rows.
size_t attn_workspace_most(int64_t num_tokens, int group, int head_dim) {
  if (num_tokens <= 0) return 0;
  return bytes_of(form(1, num_tokens * group, head_dim), group, head_dim);
}

cudaError_t launch_attention(const AttnArgs& a, cudaStream_t stream) {
  switch (form(a.num_seqs, (int64_t)a.num_tokens * a.group, a.head_dim)) {
    case Form::kMany:
      return attn::launch_many(a, stream);
    case Form::kWide:
      return attn::launch_wide(a, stream);
    case Form::kFew32:
      return attend_few<64, 2>(a, stream);
    default:
      return a.head_dim == 64    ? attend_few<64, 1>(a, stream)
             : a.head_dim == 128 ? attend_few<128, 1>(a, stream)
                                 : attend_few<256, 1>(a, stream);
  }
}

cudaError_t take_attn_checks(unsigned long long* first, unsigned long long* count) {
  CheckRecord r;
  const cudaError_t e = take_check_record_here(&r);
  *first = r.first;
  *count = r.count;
  return e;
}

}  // namespace mol
