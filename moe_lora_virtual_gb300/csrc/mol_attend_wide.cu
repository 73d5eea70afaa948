// Attention of many new tokens with 256 values a head over the paged cache (include/mol_attn.h).

#include "mol_attend.cuh"
#include "mol_internal.h"

namespace mol {
namespace {

using attn::Block;
using attn::ldsm4;
using attn::ldsm4_t;
using attn::Parts;
using attn::Place;
using attn::Record;

constexpr int kD = 256;
constexpr int kChunks = kD / 8;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = kWarps * 16;
constexpr int kTile = 32;                     // tokens
constexpr int kStages = 3;
constexpr int kTileBytes = kTile * kD * 2;    // keys, or values
constexpr int kRing = kStages * 2 * kTileBytes;
constexpr size_t kSmem = kRing + kRows * kD * 2;  // and the queries
constexpr int kExtra = 4;                     // units that a block takes beside its tiles
constexpr int kWhole = 8;                     // most tiles of blocks that go undivided

// The simple form, on mma.sync (on tcgen05 one tile's sums would take half of tensor memory and two tiles of
// scores the other half, so that the softmax of one overlaps the products of the next; that form is not
// built): 128 rows a thread block, 16 a warp, which all read one ring of 32-token tiles (cp.async, three
// stages, a barrier a tile). A row's scores, maximum, sum and 256 columns of sums stay with four lanes. Bound by shared memory: a warp reads its
// queries (8 KB, no registers are left for them) and the tile (32 KB) for 2 x 16 x 32 x 256 products, which
// at 128 bytes a cycle allows 470 TFLOP/s; 16 query heads of 2 key heads reach 233 on 8 prompts of 8192
// tokens and 195 on 8 of 2048 (attend_few: 74), the rest waits, as two warps a scheduler hide little.
// Tiles are dealt, what a row does not see is treated, and long blocks are summed by stretches (LONG), as in
// attend_few.
template <bool LONG>
__global__ void __launch_bounds__(kThreads, 1) attend_wide_kernel(const __grid_constant__ AttnArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int s_scan[kWarps + 1];
  __shared__ Place s_place;
  __shared__ uint32_t s_held[kWarps][kStages];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* shared = smem + kRing;

  attn::prefetch_table<kThreads>(a);
  const attn::Run run = attn::wait_and_deal<kThreads>(a, kRows, kTile, kExtra, s_scan, &s_place);
  const Parts parts = attn::parts(a.workspace, gridDim.x, kRows, kD);
  const int64_t c = blockIdx.x;
  if (!run.any) {
    if (tid == 0) parts.records[c].last = -1;
    return;
  }
  attn::Walk<LONG> load, work;  // over the run, of the copies and of the products
  attn::begin(a, load, s_place, run, kRows, kTile, kExtra);
  work = load;
  int load_tile = 0;  // of load.count

  // Where token `lane` of a tile lies: its page is asked for two tiles before its copies are.
  struct Token {
    int page, offset, h;  // (page -1: no row sees the token)
  };
  auto look = [&]() {
    Token t = {-1, 0, load.h};
    if (!load.more()) return t;
    const int j = (load.k.t0 + load.first + load_tile) * kTile + lane;
    if (j >= load.k.lo && j < load.k.hi) {
      const int p = divide(j, a.by_page);
      if (MOL_CHECK(p >= 0 && p < a.max_pages, MOL_CHECK_COLUMN, p))
        t.page = attn::load_int(a.page_table + load.k.b * a.table_stride + p);
      t.offset = j - p * a.page_size;
    }
    if (++load_tile == load.count) {
      attn::go_on(a, load, kRows, kTile, kExtra);
      load_tile = 0;
    }
    return t;
  };
  Token ahead[2] = {{-1, 0, 0}, {-1, 0, 0}};
  // Asks for this warp's rows of the next tile into ring stage s; for a negative one only for its pages.
  auto fetch = [&](int s) {
    const Token t = ahead[0];
    ahead[0] = ahead[1];
    ahead[1] = look();
    if (s < 0) return;
    const bool held = t.page >= 0 && t.page < a.num_pages;
    const int64_t at = held ? t.page * a.page_stride + t.offset * a.token_stride + t.h * a.head_stride : 0;
    const uint32_t mask = __ballot_sync(0xffffffffu, held);
    if (lane == 0) s_held[warp][s] = mask;
#pragma unroll
    for (int i = 0; i < kTile / kWarps; ++i) {
      const int row = i * kWarps + warp;
      const int64_t from_row = __shfl_sync(0xffffffffu, at, row) + lane * 8;
      const uint32_t n = (mask >> row) & 1 ? 16u : 0u;
      unsigned char* d = smem + s * 2 * kTileBytes + row * (kD * 2) + ((lane ^ (row & 7)) << 4);
      cp_async16_zfill(d, a.k + from_row, n);
      cp_async16_zfill(d + kTileBytes, a.v + from_row, n);
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int s = -2; s < kStages - 1; ++s) fetch(s);

  const int g = lane >> 2, t4 = lane & 3;
  int stage = 0;
  Record record = {};
  record.last = -1;
#pragma unroll 1
  while (work.more()) {
    // ------------------------------------------------------------ a block of rows and a head
    const Block k = work.k;
    const int h = work.h, first = work.first, count = work.count;
#pragma unroll 4
    for (int i = tid; i < kRows * kChunks; i += kThreads) {
      const int row = i / kChunks, ch = i % kChunks;
      uint4 q = make_uint4(0, 0, 0, 0);
      if (row < k.nrows) {
        const int r = k.row0 + row, token = divide(r, a.by_group);
        if (MOL_CHECK(k.s.start + token < a.num_tokens, MOL_CHECK_ROW, k.s.start + token))
          q = attn::load_16(a.q + (int64_t)(k.s.start + token) * a.q_token_stride +
                            (int64_t)(h * a.group + r - token * a.group) * a.q_head_stride + ch * 8);
      }
      *reinterpret_cast<uint4*>(shared + row * (kD * 2) + ((ch ^ (row & 7)) << 4)) = q;
    }
    // the positions of this lane's rows; of the warp's first and last row
    const int row_w = warp * 16, rows_w = min(k.nrows - row_w, 16), shift = k.s.kv - k.s.n;
    int pos[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      pos[i] = shift + divide(k.row0 + min(row_w + g + 8 * i, k.nrows - 1), a.by_group);
    const int pos_first = shift + divide(k.row0 + min(row_w, k.nrows - 1), a.by_group);
    const int pos_last = shift + divide(k.row0 + min(row_w + 15, k.nrows - 1), a.by_group);

    float o[kD / 8][4], top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < kD / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
#pragma unroll 1
    for (int tile = first; tile < first + count; ++tile) {
      cp_async_wait_group<kStages - 2>();
      __syncthreads();  // the tile has landed (the queries too), the stage before it is free, for every warp
      fetch(stage == 0 ? kStages - 1 : stage - 1);
      const unsigned char* kt = smem + stage * 2 * kTileBytes;
      const unsigned char* vt = kt + kTileBytes;
      const uint32_t mask = s_held[warp][stage];
      const int j0 = (k.t0 + tile) * kTile;
      // (what no row of the warp sees is passed by)
      if (mask != 0 && rows_w > 0 && j0 <= pos_last && (a.window == 0 || j0 + kTile > pos_first - a.window + 1)) {
        float s[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
          uint32_t q[4], b[2][4];
          const int q_row = row_w + (lane & 15), q_ch = 2 * kk + (lane >> 4);
          ldsm4(shared + q_row * (kD * 2) + ((q_ch ^ (q_row & 7)) << 4), q);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int row = n * 16 + (lane & 7) + ((lane >> 4) << 3), ch = 2 * kk + ((lane >> 3) & 1);
            ldsm4(kt + row * (kD * 2) + ((ch ^ (row & 7)) << 4), b[n]);
          }
#pragma unroll
          for (int n = 0; n < 4; ++n)
            mma_16816(s[n], q[0], q[1], q[2], q[3], b[n / 2][n % 2 * 2], b[n / 2][n % 2 * 2 + 1]);
        }
        const bool edge = mask != 0xffffffffu || j0 + kTile - 1 > pos_first ||
                          (a.window > 0 && j0 <= pos_last - a.window);
        auto sees = [&](int j, int p) {
          return ((mask >> (j - j0)) & 1) && j <= p && (a.window == 0 || j > p - a.window);
        };
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[n][e] *= a.scale_log2;
            if (edge && !sees(j0 + n * 8 + 2 * t4 + (e & 1), pos[e >> 1])) s[n][e] = -INFINITY;
          }
        uint32_t p[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float m = s[0][2 * i];
#pragma unroll
          for (int n = 0; n < 4; ++n) m = fmaxf(m, fmaxf(s[n][2 * i], s[n][2 * i + 1]));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          const float was = top[i];
          if (__any_sync(0xffffffffu, m > was)) {
            const float now = fmaxf(was, m);
            const float f = was == now ? 1.f : attn::ex2(was - now);  // (-inf before the first)
            top[i] = now;
            sum[i] *= f;
#pragma unroll
            for (int n = 0; n < kD / 8; ++n) {
              o[n][2 * i] *= f;
              o[n][2 * i + 1] *= f;
            }
          }
          // a row that has seen nothing yet keeps weights of 0: 2^-inf
          const float base = top[i] == -INFINITY ? 0.f : top[i];
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float w = attn::ex2(s[n][2 * i + e] - base);
              s[n][2 * i + e] = w;
              sum[i] += w;
            }
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          p[n / 2][n % 2 * 2] = pack_bf16x2(s[n][0], s[n][1]);
          p[n / 2][n % 2 * 2 + 1] = pack_bf16x2(s[n][2], s[n][3]);
        }
        bool plain = false;
        if (edge) {
          bool bad = false;
#pragma unroll 4
          for (int i = lane; i < kTile * kChunks; i += 32) bad |= attn::not_finite(lds16(vt + i * 16));
          plain = __any_sync(0xffffffffu, bad);
        }
        if (!plain) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int n2 = 0; n2 < kD / 16; ++n2) {
              uint32_t b[4];
              const int row = x * 16 + (lane & 15), ch = 2 * n2 + (lane >> 4);
              ldsm4_t(vt + row * (kD * 2) + ((ch ^ (row & 7)) << 4), b);
              mma_16816(o[2 * n2], p[x][0], p[x][1], p[x][2], p[x][3], b[0], b[1]);
              mma_16816(o[2 * n2 + 1], p[x][0], p[x][1], p[x][2], p[x][3], b[2], b[3]);
            }
        } else {
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll 1
            for (int i = 0; i < 16; ++i) {
              const int at = x * 16 + i, j = j0 + at, from_lane = (lane & ~3) | ((i & 7) >> 1);
              float w[2];
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const uint32_t pair = i < 8 ? p[x][r] : p[x][2 + r];
                const uint32_t got = __shfl_sync(0xffffffffu, pair, from_lane);
                w[r] = i & 1 ? bf16_hi(got) : bf16_lo(got);
              }
              const bool see[2] = {sees(j, pos[0]), sees(j, pos[1])};
#pragma unroll
              for (int n = 0; n < kD / 8; ++n) {
                const uint32_t v =
                    *reinterpret_cast<const uint32_t*>(vt + at * (kD * 2) + ((n ^ (at & 7)) << 4) + 4 * t4);
                const float v0 = bf16_lo(v), v1 = bf16_hi(v);
#pragma unroll
                for (int r = 0; r < 2; ++r)
                  if (see[r]) {
                    o[n][2 * r] += w[r] * v0;
                    o[n][2 * r + 1] += w[r] * v1;
                  }
              }
            }
        }
      }
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }

    // ------------------------------------------------------------ the rows, or a part of them
    const bool begins = work.begins(), stays = work.stays(kExtra), joins = work.joins();
    const bool part = stays || !begins || !work.ends();
    const int slot = (int)(2 * c) + (begins ? 1 : 0);
    if (begins && part && !stays && tid == 0) record = {work.last(run), k.s.start, k.row0, k.nrows, h, {}};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float l = sum[i];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      const int row = row_w + g + 8 * i;
      float was = 0.f, own = 1.f;  // factors of the stretches before and of this one
      if (joins) {
        float2 met = t4 == 0 ? parts.tops[(int64_t)slot * kRows + row] : make_float2(0.f, 0.f);
        met.x = __shfl_sync(0xffffffffu, met.x, lane & ~3);
        met.y = __shfl_sync(0xffffffffu, met.y, lane & ~3);
        const float most = fmaxf(top[i], met.x), base = most == -INFINITY ? 0.f : most;
        was = attn::ex2(met.x - base);
        own = attn::ex2(top[i] - base);
        top[i] = most;
        l = was * met.y + own * l;
      }
      if (row >= k.nrows) continue;
      const int r = k.row0 + row, token = divide(r, a.by_group);
      if (!MOL_CHECK(k.s.start + token < a.num_tokens, MOL_CHECK_ROW, k.s.start + token)) continue;
      float2* sums = reinterpret_cast<float2*>(parts.sums + ((int64_t)slot * kRows + row) * kD + 2 * t4);
      if (joins) {  // (with what the lane itself left there)
#pragma unroll
        for (int n = 0; n < kD / 8; ++n) {
          const float2 y = sums[n * 4];
          sums[n * 4] = make_float2(was * y.x + own * o[n][2 * i], was * y.y + own * o[n][2 * i + 1]);
        }
      } else if (part) {
#pragma unroll
        for (int n = 0; n < kD / 8; ++n) sums[n * 4] = make_float2(o[n][2 * i], o[n][2 * i + 1]);
      }
      if (part) {
        if (t4 == 0) parts.tops[(int64_t)slot * kRows + row] = make_float2(top[i], l);
      } else {
        const float inv = top[i] == -INFINITY ? 0.f : 1.f / l;
        uint16_t* dst = a.out + (int64_t)(k.s.start + token) * a.out_token_stride +
                        (int64_t)(h * a.group + r - token * a.group) * a.out_head_stride + 2 * t4;
        if (joins) {
#pragma unroll 4
          for (int n = 0; n < kD / 8; ++n)
            *reinterpret_cast<uint32_t*>(dst + n * 8) = pack_bf16x2(sums[n * 4].x * inv, sums[n * 4].y * inv);
        } else {
#pragma unroll
          for (int n = 0; n < kD / 8; ++n)
            *reinterpret_cast<uint32_t*>(dst + n * 8) = pack_bf16x2(o[n][2 * i] * inv, o[n][2 * i + 1] * inv);
        }
      }
    }
    attn::go_on(a, work, kRows, kTile, kExtra);
    __syncthreads();  // every warp has read its queries
  }
  cp_async_wait_all();
  if (tid == 0) parts.records[c] = record;
}

}  // namespace

size_t attn::wide_bytes() { return attn::parts_bytes(kMaxGrid / 2, kRows, kD); }

cudaError_t attn::prepare_wide() {
  auto set = [](auto kernel) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  };
  const cudaError_t e = set(attend_wide_kernel<false>);
  return e != cudaSuccess ? e : set(attend_wide_kernel<true>);
}

cudaError_t attn::launch_wide(const AttnArgs& args, cudaStream_t stream) {
  const int grid = attn::sms();
  AttnArgs a = args;
  a.by_grid = divider(grid);
  a.whole = attn::undivided(a, kRows, kTile, kWhole);
  auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(grid), dim3(kThreads), kSmem, stream, a); };
  const cudaError_t e = attn::beyond_a_stretch(a, kRows, kTile) ? go(attend_wide_kernel<true>)
                                                               : go(attend_wide_kernel<false>);
  if (e != cudaSuccess || a.whole) return e;
  return attn::launch_join(a, grid, kRows, attn::parts(a.workspace, grid, kRows, kD), stream);
}

cudaError_t take_wide_checks(unsigned long long* first, unsigned long long* count) {
  CheckRecord r;
  const cudaError_t e = take_check_record_here(&r);
  *first = r.first;
  *count = r.count;
  return e;
}

}  // namespace mol
