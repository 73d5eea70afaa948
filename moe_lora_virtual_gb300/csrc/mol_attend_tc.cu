// Attention of many new tokens over the paged cache on the fifth-generation tensor cores
// (include/mol_attn.h).

#include <algorithm>
#include <mutex>

#include "mol_attend.cuh"
#include "mol_internal.h"
#include "mol_tc.cuh"

namespace mol {

__device__ unsigned int g_many_fault_flags;
// Test controls of the bounded waits, set only through mol_debug_wait_test.
__device__ unsigned int g_many_test_stall;
__device__ unsigned long long g_many_wait_limit_ns = kWaitLimitNs;

namespace {

using attn::Block;
using attn::ex2;
using attn::Parts;
using attn::Place;
using attn::Record;

constexpr int kM = 128;                       // rows of a query tile, tokens of a key tile
constexpr int kThreads = 12 * 32;
// Registers a thread: 384 threads are launched with 168; the last four warps give theirs up to the
// softmax warps, 256 * 200 + 128 * 96 <= 384 * 168.
constexpr int kSoftmaxRegs = 200, kOtherRegs = 96;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * 168, "registers");
constexpr uint32_t kPolls = 1u << 22;
constexpr int kHeldRing = 8;                  // more tiles than the loader is ever ahead
// Most tiles of blocks that go undivided: 200 tokens over 500, 16 heads of 128 on 2, 14.6 us against 19.9 in parts.
constexpr int kWhole = 4;
constexpr int kExtra = 2;                     // units that a block takes beside its tiles
constexpr float kLazy = 8.f;                  // log2 of how far weights may pass 1

template <int D>
struct Geo {
  static constexpr int kHalf = kM * 128;        // bytes of 64 columns of a tile
  static constexpr int kTileBytes = kHalf * (D / 64);
  static constexpr int kSlots = D == 128 ? 5 : 10;
  static constexpr size_t kSmem = 1024 + (size_t)(2 + kSlots) * kTileBytes;
  // Tensor memory: the scores of both query tiles, their sums, and the weights: in columns of their own
  // where there are any left (64 values a head), else over the first half of the scores.
  static constexpr bool kApart = D == 64;
  static constexpr uint32_t kS = 0, kO = 2 * kM, kP = kApart ? kO + 2 * D : kS, kPStep = kApart ? kM / 2 : kM;
  static constexpr uint32_t kCols = 512;
};

// A whole warp's bounded wait, whose lanes agree on its outcome.
MOL_DEV bool warp_wait(uint64_t* bar, uint32_t parity, unsigned long long limit_ns) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, kPolls, limit_ns));
}

MOL_DEV void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
// Shared-memory operands: low word of their descriptor (address and, for rows that are the contraction, the
// distance of their 64-column atoms in the upper half) and the high word that all have: 8-row groups
// 1024 bytes apart, 128-byte swizzle.
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
MOL_DEV uint32_t desc_low(uint32_t saddr) { return (saddr & 0x3FFFFu) >> 4; }
// D += A * B by one lane of the converged warp: A and B with the contraction along their rows.
MOL_DEV void umma_ss(uint32_t leader, uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc,
                     uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " mov.b64 a, {%1, %6};\n mov.b64 b, {%2, %6};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_low | 1u << 16), "r"(b_low | 1u << 16), "r"(idesc), "r"(accumulate), "r"(leader), "r"(kDescHigh)
      : "memory");
}
// The same with A (bf16) in tensor memory and B's rows the contraction, its atoms `atom` 16-byte units apart.
MOL_DEV void umma_ts(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low, uint32_t atom,
                     uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " mov.b64 b, {%2, %6};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_low | atom << 16), "r"(idesc), "r"(accumulate), "r"(leader), "r"(kDescHigh)
      : "memory");
}
MOL_DEV void arrive(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n @q mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(
          smem_u32(bar)),
      "r"(leader)
      : "memory");
}
MOL_DEV void commit(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          smem_u32(bar)),
      "r"(leader)
      : "memory");
}
MOL_DEV void tmem_ld_x32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// The same and the largest of the 32 (NaN aside).
MOL_DEV void tmem_ld_max_x32(uint32_t taddr, uint32_t* r, float& m) {
  uint32_t w;
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, %32, [%33];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(w)
      : "r"(taddr)
      : "memory");
  m = __uint_as_float(w);  // (to be read behind the wait, like the others)
}
MOL_DEV void tmem_st_x32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
MOL_DEV void tmem_ld_x16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
MOL_DEV void tmem_st_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
MOL_DEV uint32_t tmem_ld_x1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
  return r;
}
MOL_DEV void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
MOL_DEV void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 values at a time.
MOL_DEV float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
MOL_DEV float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}


// Which of a tile's tokens lie in the cache: bit p for those of page p of the tile, or a bit a token and
// whether all do. (Copied page by page, 64 values a head are faster with the second, mixed batch 98 us
// against 104, and 128 with the first, chunk of 509 tokens 182 against 200.)
template <bool TOKENS>
struct Held {
  uint32_t pages;
  MOL_DEV bool all(int per) const { return pages == (uint32_t)(((uint64_t)1 << (kM / per)) - 1); }
  MOL_DEV uint32_t columns(int w, int per) const {  // 32 w .. 32 w + 31
    uint32_t c = 0xffffffffu;
    const int log_per = 31 - __clz(per);
#pragma unroll
    for (int b = 0; b < 4; ++b)
      if (!((pages >> ((32 * w + 8 * b) >> log_per)) & 1)) c &= ~(0xffu << (8 * b));
    return c;
  }
};
template <>
struct Held<true> {
  uint32_t tokens[4];
  uint32_t whole;
  MOL_DEV bool all(int) const { return whole != 0; }
  MOL_DEV uint32_t columns(int w, int) const { return tokens[w]; }
};
// Of a tile's columns 32 w .. 32 w + 31 those that lie in (lo, hi] and whose token is held.
template <typename H>
MOL_DEV uint32_t columns_seen(int w, int lo, int hi, const H& held, int per) {
  const int first = max(lo + 1 - 32 * w, 0), last = min(hi - 32 * w, 31);
  if (first > 31 || last < first) return 0u;
  return (0xffffffffu << first) & (0xffffffffu >> (31 - last)) & held.columns(w, per);
}
// M = 128, N = 128, both operands with the contraction along their rows.
constexpr uint32_t kScores = IDesc<kM, kM>::kValue;
// N = D, the second operand's rows are the contraction.
template <int D>
constexpr uint32_t kValues = IDesc<kM, D>::kValue | (1u << 16);

// Two query tiles of 128 rows (new tokens x the group's heads, so the group shares each key) against
// tiles of 128 cached tokens, the whole chain in tensor memory: scores = queries . keys^T in fp32,
// weights in bf16 written over them, sums += weights . values. tcgen05.mma bounds it: 4 * D operations a
// score, against one exponential; while one tile's softmax runs, the tensor cores have the other
// tile's products.
//   warps 0-3, 4-7  softmax of query tile 0, 1: a thread a row, 128 scores in registers, maximum and sum
//                   without a shuffle. The maximum that weights refer to moves only when one would
//                   pass 2^8 (bf16 and fp32 lose nothing to that), so sums are hardly ever rescaled
//   warp 8          issues the products: P0 V, Q0 K', P1 V, Q1 K' (K' the next keys); Q0 K', Q1 K', P0 V, P1 V
//                   for 64 values a head, whose weights need not wait for the scores' place. TWO: the
//                   scores' products alone, those of the weights are issued by warp 10
//   warp 9          copies the queries and, page by page, keys and values (TMA, 128-byte swizzle) into a
//                   ring of tiles; token by token (cp.async) from pages whose tokens make no such copies
//   warps 10, 11    look through the values of tiles that some row does not see all of: values that are
//                   not finite are zeroed where no row sees them; where another row does, the tile's
//                   softmax warps sum its products without the tensor cores, for which 0 * NaN is NaN
// Tiles are dealt as in attend_few, long blocks summed by stretches (LONG); parts of blocks join in
// launch_join. Pages outside the cache are zeros (the copy's fill); what a row does not see is replaced among
// its scores.
// 509 tokens over 30001, 32 heads of 128 on 4: 183 us, 1360 TFLOP/s (0.71 of the measured rate), a prompt of
// 8192 426 us, 1290. A pair of tiles takes 3200 cycles: a query tile's own products 1340, its softmax 1525,
// hand-overs 380, against 2680 of both tiles' products.
template <int D, bool GATHER, bool TWO, bool LONG>
__global__ void __launch_bounds__(kThreads, 1)
    attend_many_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, AttnArgs a, int tile_tokens) {
  using G = Geo<D>;
  constexpr bool kTokens = GATHER || D == 64;
  static_assert(!TWO || (G::kApart && !GATHER), "a free warp, and weights apart from the scores");
  // tokens that are gathered, or a second issuing warp, leave one to look through values
  constexpr int kLookers = GATHER || TWO ? 1 : 2;
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t q_full, q_empty, all_done, full[G::kSlots], empty[G::kSlots], seen[G::kSlots], s_full[2],
      p_full[2], o_full[2], s_read[2];
  __shared__ Held<kTokens> s_held[kHeldRing];
  __shared__ uint32_t s_tmem, s_skip[2], s_bad[G::kSlots];
  __shared__ int s_scan[kThreads / 32 + 1];
  __shared__ Place s_place;
  __shared__ attn::Run s_run;
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char* ring = smem + 2 * G::kTileBytes;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    mbar_init(&all_done, TWO ? 2 : 1);
    for (int s = 0; s < G::kSlots; ++s) {
      mbar_init(&full[s], GATHER ? 32 : 1);
      mbar_init(&empty[s], 1 + kLookers);  // the last products' commit, and the warps that look through values
      mbar_init(&seen[s], kLookers);
      s_bad[s] = 0;
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 2);  // the products' commit, and the issuing thread for what it has seen
      mbar_init(&p_full[t], 4);  // a warp each
      mbar_init(&o_full[t], 1);
      mbar_init(&s_read[t], TWO ? 5 : 4);  // and the values' issuing warp, for the products of before
    }
    fence_mbar_init();
  }
  if (warp == 8) tmem_alloc(&s_tmem, G::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  const int tile_rows = tile_tokens * a.group, rows = 2 * tile_rows;
  {
    const attn::Run run = attn::wait_and_deal<kThreads>(a, rows, kM, kExtra, s_scan, &s_place);
    if (tid == 0) s_run = run;
    __syncthreads();
  }
  auto held_at = [&](uint32_t n) {
    Held<kTokens> h;
    const volatile Held<kTokens>* at = &s_held[n % kHeldRing];
    if constexpr (kTokens) {
      for (int x = 0; x < 4; ++x) h.tokens[x] = at->tokens[x];
      h.whole = at->whole;
    } else {
      h.pages = at->pages;
    }
    return h;
  };
  bool fault = false;
  const unsigned long long limit = g_many_wait_limit_ns;
  // (each role begins its own, from shared memory: nothing of it is held in registers before)
  using Walk = attn::Walk<LONG>;
  auto begin = [&](Walk& w) {
    w.left = 0;
    if (s_run.any) attn::begin(a, w, s_place, s_run, rows, kM, kExtra);
  };
  auto next = [&](Walk& w) { attn::go_on(a, w, rows, kM, kExtra); };

  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == 9 || (GATHER && warp == 10)) {
    // ------------------------------------------------------------ copies
    uint32_t u = 0, n = 0, seg = 0;  // ring slots used, tiles, blocks
    if constexpr (!GATHER) {
      const int per = a.page_size < kM ? a.page_size : kM;  // tokens a copy
      const int copies = kM / per;
      Walk w;
      for (begin(w); w.more() && !fault && !(g_many_test_stall & 1); next(w)) {
        const Block& k = w.k;
        const int32_t* pages = a.page_table + k.b * a.table_stride;
        // lane p: page p of the block's i-th tile, asked for a tile ahead
        auto look = [&](int i) {
          const int j = (k.t0 + w.first + i) * kM + lane * per;
          if (i >= w.count || lane >= copies || j + per <= k.lo || j >= k.hi) return -1;
          const int p = divide(j, a.by_page);
          return MOL_CHECK(p >= 0 && p < a.max_pages, MOL_CHECK_COLUMN, p) ? attn::load_int(pages + p) : -1;
        };
        int page = look(0);
        for (int i = 0; i < w.count && !fault; ++i, ++n) {
          const int next_page = look(i + 1);
          const bool held = page >= 0 && page < a.num_pages;
          const uint32_t mask = __ballot_sync(0xffffffffu, held);
          if (!held) page = a.num_pages;  // past the end: zeros
          const int j = (k.t0 + w.first + i) * kM + lane * per;
          const int offset = j - divide(j, a.by_page) * a.page_size;
          (void)MOL_CHECK(lane >= copies || (offset >= 0 && offset + per <= a.page_size), MOL_CHECK_TMA_COORD,
                          offset);
          if constexpr (kTokens) {
            const Held<false> by_page{mask};
            if (lane < 4) *(volatile uint32_t*)&s_held[n % kHeldRing].tokens[lane] = by_page.columns(lane, per);
            if (lane == 0) *(volatile uint32_t*)&s_held[n % kHeldRing].whole = by_page.all(per);
            __syncwarp();
          } else {
            if (lane == 0) *(volatile uint32_t*)&s_held[n % kHeldRing].pages = mask;
          }
          for (int kv = 0; kv < 2 && !fault; ++kv, ++u) {
            const int s = (int)(u % G::kSlots);
            if (!warp_wait(&empty[s], ((u / G::kSlots) & 1) ^ 1, limit)) {
              fault = true;
              break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)G::kTileBytes);
            __syncwarp();
            if (lane < copies)
              for (int x = 0; x < D / 64; ++x)
                tma_load_4d(ring + s * G::kTileBytes + x * G::kHalf + lane * per * 128, kv ? &map_v : &map_k,
                            x * 64, offset, w.h, page, &full[s]);
            if (i + kv == 0) {  // the queries behind the first keys, which need not wait for the block before
              if (seg > 0 && !warp_wait(&q_empty, (seg - 1) & 1, limit)) {
                fault = true;
                ++u;
                break;
              }
              const bool two = k.nrows > tile_rows;
              if (lane == 0) {
                mbar_arrive_expect_tx(&q_full, (uint32_t)(tile_rows * 128 * (D / 64) * (two ? 2 : 1)));
                for (int t = 0; t < (two ? 2 : 1); ++t)
                  for (int x = 0; x < D / 64; ++x)
                    tma_load_4d(smem + t * G::kTileBytes + x * G::kHalf, &map_q, x * 64, 0, w.h,
                                k.s.start + divide(k.row0, a.by_group) + t * tile_tokens, &q_full);
              }
              ++seg;
            }
          }
          page = next_page;
        }
      }
    } else {
      // token by token, 16 bytes a lane: keys by one warp, values by the other
      constexpr int kChunks = D / 8;
      const int kv = warp - 9;
      const uint16_t* src = kv ? a.v : a.k;
      u = kv;
      Walk w;
      for (begin(w); w.more() && !fault && !(g_many_test_stall & 1); next(w)) {
        const Block& k = w.k;
        const int32_t* pages = a.page_table + k.b * a.table_stride;
        // lane l: the pages of tokens l, 32 + l, 64 + l, 96 + l of the block's i-th tile
        int page[4], next_page[4];
        auto look = [&](int i, int (&to)[4]) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int j = (k.t0 + w.first + i) * kM + 32 * x + lane;
            const int p = divide(max(j, 0), a.by_page);
            to[x] = i < w.count && j >= k.lo && j < k.hi && MOL_CHECK(p < a.max_pages, MOL_CHECK_COLUMN, p)
                        ? attn::load_int(pages + p) : -1;
          }
        };
        look(0, page);
        for (int i = 0; i < w.count && !fault; ++i, ++n, u += 2) {
          look(i + 1, next_page);
          int64_t at[4];
          uint32_t held[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int j = (k.t0 + w.first + i) * kM + 32 * x + lane;
            const bool in = page[x] >= 0 && page[x] < a.num_pages;
            at[x] = in ? page[x] * a.page_stride + (j - divide(j, a.by_page) * a.page_size) * a.token_stride +
                             w.h * a.head_stride : 0;
            held[x] = __ballot_sync(0xffffffffu, in);
            page[x] = next_page[x];
          }
          if (kv == 0 && lane == 0) {
            volatile Held<kTokens>* to = &s_held[n % kHeldRing];
            for (int x = 0; x < 4; ++x) to->tokens[x] = held[x];
            to->whole = (held[0] & held[1] & held[2] & held[3]) == 0xffffffffu;
          }
          __syncwarp();
          const int s = (int)(u % G::kSlots);
          if (!warp_wait(&empty[s], ((u / G::kSlots) & 1) ^ 1, limit)) {
            fault = true;
            break;
          }
          unsigned char* tile = ring + s * G::kTileBytes;
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll 8
            for (int y = 0; y < kChunks; ++y) {
              const int row = (y * 32 + lane) / kChunks, ch = (y * 32 + lane) % kChunks;
              cp_async16_zfill(tile + (ch >> 3) * G::kHalf + (32 * x + row) * 128 + (((ch & 7) ^ (row & 7)) << 4),
                               src + __shfl_sync(0xffffffffu, at[x], row) + ch * 8,
                               (held[x] >> row) & 1 ? 16u : 0u);
            }
          cp_async_arrive_noinc(&full[s]);
          if (i == 0 && kv == 0) {
            if (seg > 0 && !warp_wait(&q_empty, (seg - 1) & 1, limit)) {
              fault = true;
              break;
            }
            const bool two = k.nrows > tile_rows;
            if (lane == 0) {
              mbar_arrive_expect_tx(&q_full, (uint32_t)(tile_rows * 128 * (D / 64) * (two ? 2 : 1)));
              for (int t = 0; t < (two ? 2 : 1); ++t)
                for (int x = 0; x < D / 64; ++x)
                  tma_load_4d(smem + t * G::kTileBytes + x * G::kHalf, &map_q, x * 64, 0, w.h,
                              k.s.start + divide(k.row0, a.by_group) + t * tile_tokens, &q_full);
            }
            ++seg;
          }
        }
      }
      cp_async_wait_all();
    }
    if (fault) {  // nothing left in flight (gathered tokens are not, by now)
      for (uint32_t i = u > (uint32_t)G::kSlots ? u - G::kSlots : 0; !GATHER && i < u; ++i)
        (void)warp_wait(&full[i % G::kSlots], (i / G::kSlots) & 1, limit);
      if (seg > 0) (void)warp_wait(&q_full, (seg - 1) & 1, limit);
    }
  } else if (warp >= 12 - kLookers) {
    // ------------------------------------------------------------ values that not every row sees
    uint32_t u = 0, n = 0;
    const int per = a.page_size < kM ? a.page_size : kM;
    Walk w;
    for (begin(w); w.more() && !fault; next(w)) {
      const Block& k = w.k;
      const int shift = k.s.kv - k.s.n;
      const int pos_first = shift + divide(k.row0, a.by_group);
      const int pos_last = shift + divide(k.row0 + k.nrows - 1, a.by_group);
      for (int i = 0; i < w.count && !fault; ++i, ++n)
        for (int kv = 0; kv < 2; ++kv, ++u) {
          const int s = (int)(u % G::kSlots);
          if (!warp_wait(&full[s], (u / G::kSlots) & 1, limit)) {
            fault = true;
            break;
          }
          const int j0 = (k.t0 + w.first + i) * kM;
          if (kv && (!held_at(n).all(per) || j0 + kM - 1 > pos_first ||
                     (a.window > 0 && j0 <= pos_last - a.window))) {
            unsigned char* v = ring + s * G::kTileBytes;
            // 0 times a value is NaN where it is not finite, and stays so in the sum
            uint32_t zeros = 0;
#pragma unroll 8
            for (int x = tid - (12 - kLookers) * 32; x < G::kTileBytes / 16; x += kLookers * 32) {
              const uint4 q = lds16(v + x * 16);
              for (uint32_t two : {q.x, q.y, q.z, q.w})
                asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(zeros) : "r"(two), "r"(0u));
            }
            bool bad = false;
            if (zeros & 0x7fff7fffu) {
#pragma unroll 1
              for (int x = tid - (12 - kLookers) * 32; x < G::kTileBytes / 16; x += kLookers * 32)
                if (attn::not_finite(lds16(v + x * 16))) {
                  const int j = j0 + (x >> 3) % kM;
                  if (j < k.lo || j >= k.hi)
                    *reinterpret_cast<uint4*>(v + x * 16) = make_uint4(0, 0, 0, 0);
                  else
                    bad = true;
                }
            }
            fence_proxy_async_smem();
            if (bad) *(volatile uint32_t*)&s_bad[s] = u + 1;
            __syncwarp();
          }
          if (lane == 0) {
            mbar_arrive(&seen[s]);
            mbar_arrive(&empty[s]);
          }
        }
    }
  } else {
    // ------------------------------------------------------------ products
    // The whole warp goes through it, so that what the products take lies in registers that the warp shares;
    // one lane issues them.
    uint32_t u = 0, seg = 0, np[2] = {0, 0};
    const uint32_t leader = lane == 0;
    const uint32_t q_at = desc_low(smem_u32(smem)), ring_at = desc_low(smem_u32(ring));
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!warp_wait(bar, parity, limit)) fault = true;
      return !fault;
    };
    // (what came token by token is the generic proxy's; the products read through the async one)
    auto wait_slot = [&](uint32_t i) {
      const bool ok = wait(&full[i % G::kSlots], (i / G::kSlots) & 1);
      if (GATHER) fence_proxy_async_smem();
      return ok;
    };
    // Two barriers with one vote where both have completed (a wait is some 100 cycles without a product).
    auto wait_two = [&](uint64_t* a0, uint32_t p0, uint64_t* a1, uint32_t p1) {
      const bool one = mbar_try_wait(a0, p0), other = mbar_try_wait(a1, p1);
      return __all_sync(0xffffffffu, one && other) || (wait(a0, p0) && wait(a1, p1));
    };
    auto scores = [&](int t, uint32_t slot) {
      const uint32_t q = q_at + t * (G::kTileBytes >> 4);
      const uint32_t k = ring_at + (slot % G::kSlots) * (G::kTileBytes >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk / 4) * G::kHalf + (kk % 4) * 32) >> 4;
        umma_ss(leader, tmem + G::kS + t * kM, q + off, k + off, kScores, kk != 0);
      }
      commit(leader, &s_full[t]);
      arrive(leader, &s_full[t]);
    };
    // false where the weights do not come
    auto sums = [&](int t, uint32_t slot, bool begun) {
      if (!wait(&p_full[t], np[t] & 1)) return false;
      tc_fence_after();
      ++np[t];
      if (!*(volatile uint32_t*)&s_skip[t]) {
        const uint32_t v = ring_at + (slot % G::kSlots) * (G::kTileBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < kM / 16; ++kk)
          umma_ts(leader, tmem + G::kO + t * D, tmem + G::kP + t * G::kPStep + kk * 8, v + (kk * 16 * 128 >> 4),
                  G::kHalf >> 4, kValues<D>, begun || kk != 0);
      }
      return true;
    };
    Walk w;
    if constexpr (TWO) {
      // One warp's waits while the other's products run; the scores go on into the next block. A tile's next
      // scores are issued behind the products of the weights before, which their softmax waits for first.
      if (warp == 10) {
        arrive(leader, &s_read[0]);
        arrive(leader, &s_read[1]);
      }
      for (begin(w); w.more() && !fault; next(w)) {
        const int tiles = w.k.nrows > tile_rows ? 2 : 1, count = w.count;
        ++seg;
        if (warp == 8 && !wait(&q_full, (seg - 1) & 1)) break;
        for (int i = 0; i < count && !fault; ++i, u += 2) {
          const uint32_t slot = warp == 8 ? u : u + 1;
          if (!wait_slot(slot)) break;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t == tiles) break;
            if (warp == 8) {  // as soon as the scores before these have been read
              if (np[t] > 0 && !wait(&s_read[t], (np[t] - 1) & 1)) break;
              tc_fence_after();
              ++np[t];
              scores(t, slot);
            } else {
              if (!sums(t, slot, i > 0)) break;
              commit(leader, &o_full[t]);
              arrive(leader, &s_read[t]);
            }
          }
          commit(leader, &empty[slot % G::kSlots]);
          if (warp == 8 && i + 1 == count) commit(leader, &q_empty);
        }
      }
    } else {
      for (begin(w); w.more() && !fault; next(w)) {
        const int tiles = w.k.nrows > tile_rows ? 2 : 1, count = w.count;
        ++seg;
        if (!wait(&q_full, (seg - 1) & 1) || !wait_slot(u)) break;
        scores(0, u);
        if (tiles == 2) scores(1, u);
        commit(leader, &empty[u % G::kSlots]);
        if (count == 1) commit(leader, &q_empty);  // (with the block's last scores)
        bool begun[2] = {false, false};
        for (int i = 0; i < count && !fault; ++i) {
          // slot u: the tile's keys (done with), u + 1: its values, u + 2: the next tile's keys
          const bool more = i + 1 < count;
          const uint32_t k1 = more ? u + 2 : u + 1;
          if (!wait_two(&full[(u + 1) % G::kSlots], ((u + 1) / G::kSlots) & 1, &full[k1 % G::kSlots],
                        (k1 / G::kSlots) & 1))
            break;
          if (GATHER) fence_proxy_async_smem();
          // the next tile's scores as soon as these have been read, where the weights lie apart
          if (G::kApart && more) {
            const bool both = tiles == 2;
            if (!wait_two(&s_read[0], np[0] & 1, &s_read[both], (both ? np[1] : np[0]) & 1)) break;
            tc_fence_after();
            scores(0, u + 2);
            if (both) scores(1, u + 2);
            commit(leader, &empty[(u + 2) % G::kSlots]);
            if (i + 2 == count) commit(leader, &q_empty);
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t == tiles || !sums(t, u + 1, begun[t])) break;
            begun[t] = true;
            if (t == tiles - 1) commit(leader, &empty[(u + 1) % G::kSlots]);
            if (G::kApart || !more) commit(leader, &o_full[t]);
            if (!G::kApart && more) {
              scores(t, u + 2);
              if (t == tiles - 1) {
                commit(leader, &empty[(u + 2) % G::kSlots]);
                if (i + 2 == count) commit(leader, &q_empty);
              }
            }
          }
          u += 2;
        }
      }
    }
    // the products are done, and their commits have arrived
    commit(leader, &all_done);
    if (!warp_wait(&all_done, 0, limit)) fault = true;
  }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int t = warp >> 2, quarter = warp & 3;
    const int local = quarter * 32 + lane;  // row of the tile
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t ts = tmem + lanes + G::kS + t * kM, to_ = tmem + lanes + G::kO + t * D;
    const uint32_t tp = tmem + lanes + G::kP + t * G::kPStep;
    uint32_t ns = 0, n = 0, u = 0, no = 0;  // scores waited for, tiles, ring slots, sums waited for
    Record record = {};
    record.last = -1;
    Walk w;
    for (begin(w); w.more() && !fault; next(w)) {
      const Block& k = w.k;
      const int count = w.count;
      const bool begins = w.begins(), stays = w.stays(kExtra), part = stays || !begins || !w.ends();
      const int in_tile = min(k.nrows - t * tile_rows, tile_rows);  // rows of this query tile
      if (in_tile > 0) {
        const int shift = k.s.kv - k.s.n, row = k.row0 + t * tile_rows;
        const int pos = shift + divide(row + min(local, in_tile - 1), a.by_group);
        const int pos_first = shift + divide(row, a.by_group);
        const int pos_last = shift + divide(row + in_tile - 1, a.by_group);
        float top = -INFINITY, sum = 0.f;
        for (int i = 0; i < count; ++i) {
          const int j0 = (k.t0 + w.first + i) * kM;
          if (!warp_wait(&s_full[t], ns & 1, limit)) {
            fault = true;
            break;
          }
          ++ns;
          tc_fence_after();
          const Held<kTokens> held = held_at(n + i);
          const int per = a.page_size < kM ? a.page_size : kM;
          const bool edge = !held.all(per) || j0 + kM - 1 > pos_first ||
                            (a.window > 0 && j0 <= pos_last - a.window);
          const int hi = pos - j0, lo = a.window > 0 ? hi - a.window : -1;  // seen: lo < column <= hi
          uint32_t r[kM];
          float m4[kM / 32];
#pragma unroll
          for (int x = 0; x < kM / 32; ++x) tmem_ld_max_x32(ts + x * 32, r + x * 32, m4[x]);
          tmem_wait_ld();
          if (G::kApart) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_read[t]);
          }
          if (edge) {
#pragma unroll
            for (int x = 0; x < kM / 32; ++x) {
              const uint32_t sees = columns_seen(x, lo, hi, held, per);
              if (__all_sync(0xffffffffu, sees == 0xffffffffu)) continue;  // (its maximum stands)
              m4[x] = -INFINITY;
#pragma unroll
              for (int y = 0; y < 32; ++y) {
                if (!((sees >> y) & 1)) r[32 * x + y] = __float_as_uint(-INFINITY);
                m4[x] = fmaxf(m4[x], __uint_as_float(r[32 * x + y]));
              }
            }
          }
          const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * a.scale_log2;
          // the products before these weights are done (where these lie over scores, those came behind them)
          if (G::kApart && ns > 1) {
            if (!warp_wait(&o_full[t], ns & 1, limit)) {
              fault = true;
              break;
            }
            tc_fence_after();
          }
          const bool moves = m > top + kLazy || (top == -INFINITY && m > top);
          if (__any_sync(0xffffffffu, moves)) {
            const float f = moves ? ex2(top - m) : 1.f;
            if (moves) top = m;
            sum *= f;
            if (i > 0) {
#pragma unroll 1
              for (int x = 0; x < D; x += 16) {
                uint32_t o[16];
                tmem_ld_x16(to_ + x, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st_x16(to_ + x, o);
              }
            }
          }
          const float base = top == -INFINITY ? 0.f : top;
          const float2 sc = make_float2(a.scale_log2, a.scale_log2), nb = make_float2(-base, -base);
          float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          uint32_t p[kM / 2];
#pragma unroll
          for (int x = 0; x < kM / 2; ++x) {
            float2 e = fma2(make_float2(__uint_as_float(r[2 * x]), __uint_as_float(r[2 * x + 1])), sc, nb);
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            s2[x & 1] = add2(s2[x & 1], e);
            p[x] = pack_bf16x2(e.x, e.y);
          }
          sum += (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
          tmem_st_x32(tp, p);
          tmem_st_x32(tp + 32, p + 32);
          tmem_wait_st();
          const uint32_t slot = u + 2 * i + 1;  // of the tile's values
          bool plain = false;
          if (edge) {  // they have been looked through
            if (!warp_wait(&seen[slot % G::kSlots], (slot / G::kSlots) & 1, limit)) {
              fault = true;
              break;
            }
            plain = *(volatile uint32_t*)&s_bad[slot % G::kSlots] == slot + 1;
          }
          if (plain) {
            // the row's weights come back from tensor memory two at a time
            const unsigned char* v = ring + (slot % G::kSlots) * G::kTileBytes;
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
              uint32_t o[32];
              if (i > 0) {
                tmem_ld_x32(to_ + x, o);
                tmem_wait_ld();
              } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0u;
              }
#pragma unroll 1
              for (int y = 0; y < kM; ++y) {
                const uint32_t pair = tmem_ld_x1(tp + (y >> 1));
                tmem_wait_ld();
                const float wt = y & 1 ? bf16_hi(pair) : bf16_lo(pair);
                const bool sees = (columns_seen(y >> 5, lo, hi, held_at(n + i), per) >> (y & 31)) & 1;
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                  const int ch = ((x & 63) + e) >> 3;
                  const uint4 q = lds16(v + (x >> 6) * G::kHalf + y * 128 + ((ch ^ (y & 7)) << 4));
                  const uint32_t q4[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                  for (int z = 0; z < 4; ++z) {
                    const float a0 = __uint_as_float(o[e + 2 * z]), a1 = __uint_as_float(o[e + 2 * z + 1]);
                    o[e + 2 * z] = __float_as_uint(sees ? fmaf(wt, bf16_lo(q4[z]), a0) : a0);
                    o[e + 2 * z + 1] = __float_as_uint(sees ? fmaf(wt, bf16_hi(q4[z]), a1) : a1);
                  }
                }
                __syncwarp();
              }
              tmem_st_x32(to_ + x, o);
            }
            tmem_wait_st();
          }
          if (quarter == 0 && lane == 0) *(volatile uint32_t*)&s_skip[t] = plain;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[t]);
        }
        if (fault || !warp_wait(&o_full[t], (G::kApart ? ns - 1 : no) & 1, limit)) {
          fault = true;
          break;
        }
        ++no;
        tc_fence_after();
        // ---------------------------------------------------------- the rows, or a part of them
        const int slot = 2 * (int)blockIdx.x + (begins ? 1 : 0);
        const int at = t * tile_rows + local, r = k.row0 + at, token = divide(r, a.by_group);
        const bool mine = local < in_tile && MOL_CHECK(k.s.start + token < a.num_tokens, MOL_CHECK_ROW,
                                                       k.s.start + token);
        const Parts parts = attn::parts(a.workspace, gridDim.x, rows, D);
        float* part_dst = parts.sums + ((int64_t)slot * rows + at) * D;
        float was = 0.f, own = 1.f;  // factors of the stretches before and of this one
        if (w.joins() && mine) {
          const float2 met = parts.tops[(int64_t)slot * rows + at];
          const float most = fmaxf(top, met.x), base = most == -INFINITY ? 0.f : most;
          was = ex2(met.x - base);
          own = ex2(top - base);
          top = most;
          sum = was * met.y + own * sum;
        }
        const float inv = top == -INFINITY ? 0.f : 1.f / sum;
        uint16_t* dst = a.out + (int64_t)(k.s.start + token) * a.out_token_stride +
                        (int64_t)(w.h * a.group + r - token * a.group) * a.out_head_stride;
#pragma unroll 1
        for (int x = 0; x < D; x += 32) {
          uint32_t o[32];
          tmem_ld_x32(to_ + x, o);
          tmem_wait_ld();
          if (w.joins() && mine) {  // (what the thread itself left there)
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 y = *reinterpret_cast<const float4*>(part_dst + x + e);
              o[e] = __float_as_uint(was * y.x + own * __uint_as_float(o[e]));
              o[e + 1] = __float_as_uint(was * y.y + own * __uint_as_float(o[e + 1]));
              o[e + 2] = __float_as_uint(was * y.z + own * __uint_as_float(o[e + 2]));
              o[e + 3] = __float_as_uint(was * y.w + own * __uint_as_float(o[e + 3]));
            }
          }
          if (mine && part) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(part_dst + x + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          } else if (mine) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t b[4];
#pragma unroll
              for (int z = 0; z < 4; ++z)
                b[z] = pack_bf16x2(__uint_as_float(o[e + 2 * z]) * inv, __uint_as_float(o[e + 2 * z + 1]) * inv);
              *reinterpret_cast<uint4*>(dst + x + e) = make_uint4(b[0], b[1], b[2], b[3]);
            }
          }
          __syncwarp();
        }
        if (part && mine) parts.tops[(int64_t)slot * rows + at] = make_float2(top, sum);
        tc_fence_before();
      }
      if (begins && part && !stays) record = {w.last(s_run), k.s.start, k.row0, k.nrows, w.h, {}};
      n += count;
      u += 2 * count;
    }
    if (tid == 0) attn::parts(a.workspace, gridDim.x, rows, D).records[blockIdx.x] = record;
  }

  if (fault) atomicOr(&g_many_fault_flags, kFaultBulkTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, G::kCols);
}

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;
cudaError_t g_encode_status = cudaSuccess;

// A bf16 tensor of four dimensions, copied 64 values of the innermost at a time.
bool encode(CUtensorMap* map, const void* p, const cuuint64_t (&dims)[4], const int64_t (&strides)[3],
            const cuuint32_t (&box)[4]) {
  cuuint64_t bytes[3];
  // (the stride of a dimension of one means nothing, but has to be one)
  for (int i = 0; i < 3; ++i) bytes[i] = dims[i + 1] > 1 ? (cuuint64_t)strides[i] * 2 : dims[0] * 2;
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p), dims, bytes, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pages that tensor copies can take a tile from: parts of 8 tokens (a swizzle's rows) or more, or whole tiles.
bool in_copies(const AttnArgs& a) {
  return a.num_pages > 0 && (a.page_size % kM == 0 || (a.page_size >= 8 && kM % a.page_size == 0));
}

template <int D, bool GATHER, bool TWO>
cudaError_t many(AttnArgs a, cudaStream_t stream) {
  const int tokens = kM / a.group, per = std::min(a.page_size, kM);
  CUtensorMap q, k, v;
  const cuuint64_t page_dims[4] = {(cuuint64_t)D, (cuuint64_t)a.page_size, (cuuint64_t)a.kv_heads,
                                   (cuuint64_t)a.num_pages};
  const int64_t page_strides[3] = {a.token_stride, a.head_stride, a.page_stride};
  if (!encode(&q, a.q, {(cuuint64_t)D, (cuuint64_t)a.group, (cuuint64_t)a.kv_heads, (cuuint64_t)a.num_tokens},
              {a.q_head_stride, a.q_head_stride * a.group, a.q_token_stride},
              {64, (cuuint32_t)a.group, 1, (cuuint32_t)tokens}))
    return cudaErrorInvalidValue;
  k = v = q;  // (not read where tokens are gathered)
  if (!GATHER && (!encode(&k, a.k, page_dims, page_strides, {64, (cuuint32_t)per, 1, 1}) ||
                  !encode(&v, a.v, page_dims, page_strides, {64, (cuuint32_t)per, 1, 1})))
    return cudaErrorInvalidValue;
  const int grid = attn::sms(), rows = 2 * tokens * a.group;
  a.by_grid = divider(grid);
  a.whole = attn::undivided(a, rows, kM, kWhole);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3(grid), dim3(kThreads), Geo<D>::kSmem, stream, q, k, v, a, tokens);
  };
  const cudaError_t e = attn::beyond_a_stretch(a, rows, kM) ? go(attend_many_kernel<D, GATHER, TWO, true>)
                                                           : go(attend_many_kernel<D, GATHER, TWO, false>);
  if (e != cudaSuccess || a.whole) return e;
  return attn::launch_join(a, grid, rows, attn::parts(a.workspace, grid, rows, D), stream);
}

template <int D, bool GATHER, bool TWO>
cudaError_t prepare() {
  auto set = [](auto kernel) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Geo<D>::kSmem);
  };
  const cudaError_t e = set(attend_many_kernel<D, GATHER, TWO, false>);
  return e != cudaSuccess ? e : set(attend_many_kernel<D, GATHER, TWO, true>);
}

}  // namespace

size_t attn::many_bytes(int group, int head_dim) {
  return attn::parts_bytes(kMaxGrid / 2, 2 * (kM / group) * group, head_dim);
}

cudaError_t attn::prepare_many() {
  std::call_once(g_encode_once, [] {
    cudaDriverEntryPointQueryResult q;
    g_encode_status = cudaGetDriverEntryPointByVersion(
        "cuTensorMapEncodeTiled", reinterpret_cast<void**>(&g_encode), 12000, cudaEnableDefault, &q);
    if (g_encode_status == cudaSuccess && (q != cudaDriverEntryPointSuccess || !g_encode))
      g_encode_status = cudaErrorNotSupported;
  });
  if (g_encode_status != cudaSuccess) return g_encode_status;
  cudaError_t e = prepare<64, false, false>();
  if (e == cudaSuccess) e = prepare<64, false, true>();
  if (e == cudaSuccess) e = prepare<64, true, false>();
  if (e == cudaSuccess) e = prepare<128, false, false>();
  if (e == cudaSuccess) e = prepare<128, true, false>();
  return e;
}

// 64 values a head are bound by the issue of products, 24 small ones a pair of tiles with the waits before
// them. Two issuing warps hide those, where both query tiles have rows and few tiles are cut by a mask
// (us with one | two, 32 heads on 8: 512 tokens over 30000 169 | 144, a prompt of 8192 384 | 351, 16 times 64
// tokens over 3000 54.5 | 51.7; but one query tile, 16 times 20 tokens over 3000, 39.6 | 40.6, and with a window of
// 1024 the prompt 140 | 143, a batch of prompts and single tokens 99 | 101, for which one warp then looks
// through the values).
cudaError_t attn::launch_many(const AttnArgs& a, cudaStream_t stream) {
  const bool copies = in_copies(a);
  if (a.head_dim == 128) return copies ? many<128, false, false>(a, stream) : many<128, true, false>(a, stream);
  if (!copies) return many<64, true, false>(a, stream);
  const bool two = a.window == 0 && (int64_t)a.num_tokens * a.group > (int64_t)kM * a.num_seqs;
  return two ? many<64, false, true>(a, stream) : many<64, false, false>(a, stream);
}

cudaError_t take_attn_faults(unsigned* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_many_fault_flags, sizeof(unsigned));
  if (e != cudaSuccess) return e;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_many_fault_flags, &zero, sizeof(unsigned));
}

cudaError_t set_attn_wait_test(unsigned stall, unsigned long long limit_ns) {
  const cudaError_t e = cudaMemcpyToSymbol(g_many_test_stall, &stall, sizeof(unsigned));
  return e != cudaSuccess ? e : cudaMemcpyToSymbol(g_many_wait_limit_ns, &limit_ns, sizeof(limit_ns));
}

cudaError_t take_many_checks(unsigned long long* first, unsigned long long* count) {
  CheckRecord r;
  const cudaError_t e = take_check_record_here(&r);
  *first = r.first;
  *count = r.count;
  return e;
}

}  // namespace mol
