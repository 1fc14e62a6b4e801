// Tensor-core attention over a paged latent||rope cache: one token, a row of
// drafted tokens, a tree of them or a prompt chunk per batch row (bf16, 128 or
// 64 heads, rank 512, rope 64, pages of a multiple of 8 rows).
//
// Like the window decode (tc_decode.cu), a cluster of two CTAs owns a stream of
// (query row, 64-key tile) work: each CTA scores half of the 576 features of a
// tile, the fp16 halves cross by st.async, and each CTA accumulates the context
// over its 256 latent dims in TMEM.  What differs:
//  * Pages.  A tile is 64 / box_rows boxes, each inside one page.  The pool is
//    mapped as [pages][groups of 8 rows][8 chunks of 64 dims][8 rows][64 dims],
//    so that one copy brings a box of all the CTA's dims: groups of 8 rows x 4
//    chunks of 1024 bytes, 128-byte swizzle, which both MMAs read through their
//    descriptors' strides (scores: 4096 bytes between groups of 8 keys; P.V:
//    1024 between chunks of 64 dims).
//  * Three groups of four softmax warps take the tiles in turn.  A tile's scores
//    are summed and their maximum taken before the reference that the tile
//    before left is known; the reference is handed on before the exponentials,
//    so these phases of the tiles overlap.  Each group keeps its own sum, and
//    they are joined at the end of a segment, whose context each stores a
//    part of.
//  * kPair: two tokens of 64 heads share the MMA's 128 rows.
//  * Masks.  A tile that a token sees in part has its scores masked; rows that no
//    token of the query row sees are cleared before the scores (a probability
//    of 0 must not meet what another token, or nobody, left there).  With two
//    tokens, a key that only one of them sees may not be cleared: its elements
//    that are not finite are replaced by 0 and the token that does see it gets
//    NaN.
//
// Measured, in bursts: 32 rows of 1024 to 32768 keys 120 to 127 us (5.0 TB/s;
// window decode 138), 8 x 4 tokens of 65536 367 us (1.6 PFLOP/s; 387 to 403 over
// pages of 16 rows), 8 trees of 64 nodes behind 8000 to 15000 keys 1073 to 1110
// (1.5 PFLOP/s), one row of 4096 15.7.  With many tokens per key it is bound by
// the tensor cores (busy in 68 % of the cycles) and, in a loop of a second, by
// the power limit: verify over pages of 16 rows 430, the trees 1281.  Single
// tokens read at 75 % of the copy rate, in a loop at 70; neither memory nor the
// tensor cores bind them.  The instructions of the softmax do not bind it: 96
// fewer of some 900 that a scheduler issues per tile changed nothing but the
// clock under that limit (1 %).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "mla_internal.h"
#include "tc_common.cuh"
#include "tc_host.h"
#include "tc_split.cuh"

namespace mla {
namespace {

using namespace tc;

constexpr int STAGES = 5;
// A stage: 8 groups of 8 keys, each 4 chunks of [8 keys x 64 latent dims], then [64 keys x 32 rope dims] (64-byte swizzle).
constexpr int GROUP_BYTES = 4 * 1024;
constexpr int LATENT_BYTES = 8 * GROUP_BYTES;
constexpr int STAGE_BYTES = LATENT_BYTES + BN * 64;
// The query of a segment comes through the ring ahead of its tiles, as two fills: latent chunks 0, 1 and 2, 3 of 64
// dims, each [128 rows x 128 bytes] (128-byte swizzle), with the rope dims of rows 0..63 and 64..127 (64-byte swizzle).
constexpr int QCHUNK_BYTES = 128 * 128;
static_assert(2 * QCHUNK_BYTES == LATENT_BYTES, "two query chunks take a stage's place");
constexpr int XH_BYTES = 128 * BN * 2;    // fp16 partial scores of one tile
constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 2 * XH_BYTES;
constexpr uint32_t TM_O = 0, TM_Q = 256, TM_S = 400, TM_P = 464;  // TMEM columns (Q: 128 + 16)
// Warpgroups: the softmax groups, and the issuers (loads, score MMA, P.V MMA, L2 prefetch).
constexpr uint32_t kGroups = 3;
constexpr uint32_t kSlots = 2 * kGroups;   // of masks handed from the score warp to the groups
constexpr int THREADS = 128 * (kGroups + 1);
constexpr int kLoadWarp = 4 * kGroups, kScoreWarp = kLoadWarp + 1, kPvWarp = kLoadWarp + 2, kPrefetchWarp = kLoadWarp + 3;
// Registers per thread of each warpgroup; their sum fits the launch's.
constexpr int kRegsLaunch = 128;
__host__ __device__ constexpr int regs_softmax(bool pair) { return pair ? 136 : 152; }
__host__ __device__ constexpr int regs_issue(bool pair) { return pair ? 104 : 56; }
static_assert(kGroups * regs_softmax(false) + regs_issue(false) <= (kGroups + 1) * kRegsLaunch &&
                  kGroups * regs_softmax(true) + regs_issue(true) <= (kGroups + 1) * kRegsLaunch,
              "more registers than the launch has");
// Up to this many query rows of a batch row go in lockstep, each with a cluster, so that they read a tile at the same
// time.  By 1, 2, 4, 8 rows: verify of 8 x 4 tokens of 65536 438, 395, 377, 378 us; 8 trees of 64 nodes behind 8000 to
// 15000 keys 1146, 1110, 1118, 1120; trees of 20 nodes in 4 rows of 20000 332, 307, 300, 309 (eight leave four of 76
// clusters idle).  Units are cut from the flat list of query rows, and a cluster whose row has no keys waits for the
// others: 32 rows of 1024 to 32768 keys take 396 us with four tokens each, 381 with one of four (120 in a call of one
// token), and with 5, 6 and 8 tokens, of which the first two straddle batch rows, 583, 661 and 805.
constexpr int kLockstep = 4;
// A unit's start is charged as this many tiles where the ranges are at least so long (the query waits for the last
// scores of the unit before, and its context is stored): one tree of 16 nodes behind 4050 keys 33.2 -> 29.8 us, of 64
// nodes 76 -> 72, of 20 nodes in 4 rows of 20000 309 -> 297; between 3 and 14 the charge itself moves them by 2 %.
constexpr int kStartCharge = 7, kChargeSpan = 8;
// Tiles that a row alone pulls into L2 ahead of their load (32 ragged rows 125 us, without 128).  Rows in lockstep read
// each tile four times as it is, and at the power limit every further request costs clock: verify of 8 x 4 tokens of
// 65536 in a loop of a second 436 us, 8 ahead 457, 8 ahead by one of the four in turn 441.
constexpr int kPrefetchAheadGroup = 0, kPrefetchAheadRow = 3;

__device__ __forceinline__ void tma_load_5d(void* dst, const void* tmap, uint64_t* bar, int x, int y, int z, int w, int v) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_l2_5d(const void* tmap, int x, int y, int z, int w, int v) {
  asm volatile("cp.async.bulk.prefetch.tensor.5d.L2.global.tile [%0, {%1, %2, %3, %4, %5}];"
               ::"l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v)
               : "memory");
}

// Two values in fp16, those beyond its range +-65504 (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_f16x2_sat(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

// (a0 * b0 + c0, a1 * b1 + c1) as one packed f32x2 operation.
__device__ __forceinline__ float2 fma_f32x2(float2 a, float2 b, float2 c) {
  uint64_t x, y, z, r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(r));
  return d;
}

// bf16 pairs with infinities and NaN replaced by 0; `found` is set if there was one.
__device__ __forceinline__ uint32_t finite_pair(uint32_t w, bool& found) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u, found = true;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu, found = true;
  return w;
}

template <int kPrefetchAhead, bool kPair>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    tc_paged_kernel(const __grid_constant__ CUtensorMap lat_map, const __grid_constant__ CUtensorMap rope_map,
                    const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap qrope_map,
                    const __grid_constant__ TcDecodeArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if ((smem_u32(smem_raw) & 1023u) != 0) {   // the same in every CTA: nothing waits on anything yet
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, MLA_DEVICE_LAYOUT);
    return;
  }
  uint8_t* stages = smem_raw;
  // The peer's halves of the scores, [8][128 rows][16 B] in fp16, tiles in turn.
  uint8_t* xin = smem_raw + STAGES * STAGE_BYTES;

  __shared__ __align__(8) uint64_t full_bar[STAGES], empty_bar[STAGES];
  __shared__ __align__(8) uint64_t p_full, q_full, o_free, mma_drain, pv_drain, seg_done;
  // One barrier per softmax group: its waits then follow its own tiles, whatever the others' progress.
  __shared__ __align__(8) uint64_t s_full[kGroups], s_free[kGroups], x_full[kGroups], x_free[kGroups];
  __shared__ __align__(8) uint64_t ref_full[kGroups][4];   // per lane quarter: the group's reference is in ref_s
  __shared__ __align__(8) uint64_t poison_full[kSlots];    // kPair
  __shared__ uint64_t poison_s[kSlots];
  __shared__ float ref_s[kGroups][128], sum_s[kGroups][128], sum_ref_s[kGroups][128];
  __shared__ uint32_t tmem_base_s;
  __shared__ volatile int abort_s, loaded_s;   // loaded_s: tiles whose loads have been issued
  __shared__ int32_t plan_keys_s[kMaxRowsInKernelPlan], plan_prefix_s[kMaxRowsInKernelPlan + 2];
  __shared__ int32_t row_first_s[kMaxRowsInKernelPlan], limit_s[2 * kMaxRowsInKernelPlan];
  auto aborted = [&]() -> bool { return __any_sync(0xffffffffu, abort_s != 0); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t peer = rank ^ 1u;
  const int dim_base = 256 * (int)rank;     // first latent dim of this CTA
  const int cluster = blockIdx.x >> 1;
  const int group = cluster / a.width, member = cluster % a.width;
  constexpr int kTokens = kPair ? 2 : 1;

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&lat_map);
    tma_prefetch_desc(&rope_map);
    tma_prefetch_desc(&q_map);
    tma_prefetch_desc(&qrope_map);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(&p_full, 4);      // one arrival per warp of the tile's group
    mbar_init(&q_full, 4);      // a group has written this segment's query into TMEM
    mbar_init(&o_free, 4 * kGroups);
    mbar_init(&seg_done, 4 * kGroups);   // the sums are published
    for (uint32_t b = 0; b < kGroups; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&s_free[b], 4);   // the group has read S
      mbar_init(&x_full[b], 1);   // the peer's bytes of the group's tile, announced by one of its threads
      mbar_init(&x_free[b], 4);   // the peer's group has read them
      for (int q = 0; q < 4; ++q) mbar_init(&ref_full[b][q], 1);
    }
    for (uint32_t k = 0; k < kSlots; ++k) mbar_init(&poison_full[k], 1);
    mbar_init(&mma_drain, 1);
    mbar_init(&pv_drain, 1);
    abort_s = 0;
    loaded_s = 0;
    fence_mbar_init();
  }
  if (warp == kScoreWarp) {
    tmem_alloc(&tmem_base_s, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // peer barriers initialised before any remote arrive
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  pdl_wait();

  const int32_t* keys_p = a.keys;
  const int32_t* prefix_p = a.prefix;
  if (a.plan_in_kernel) {
    plan_rows<true>(a, plan_keys_s, plan_prefix_s, blockIdx.x == 0, row_first_s, limit_s);
    keys_p = plan_keys_s;
    prefix_p = plan_prefix_s;
  }
  WorkIter it;
  it.init(a, prefix_p, group);

  auto fail = [&]() {
    abort_s = 1;
    if (a.status) atomicOr(a.status, MLA_DEVICE_TIMEOUT);
  };
  // What token k of query row n sees: keys [0, limit), in a tree from `first` on by its mask.  A token that sees nothing
  // beside one that does is scored like that one (and its result dropped).
  auto limit_of = [&](int n, int k) {
    return a.plan_in_kernel ? limit_s[kTokens * n + k] : token_limit(a, n / a.s_q, (n % a.s_q) * kTokens + k);
  };
  auto seen_of = [&](int n, int k, int t) -> uint64_t {   // of the keys of tile t
    int limit = limit_of(n, k);
    if (kPair && limit == 0) limit = limit_of(n, k ^= 1);
    const int b = n / a.s_q, i = (n % a.s_q) * kTokens + k;
    const uint64_t* mask = i < a.tok_q ? tree_of(a, b * a.tok_q + i) : nullptr;
    return paged_seen(t * BN, limit, !mask ? limit : a.plan_in_kernel ? row_first_s[n] : paged_first(a, b), mask, a.tree_words);
  };
  // One token per row: what it sees, kept in registers (looked up again in a row's last tiles, as with two tokens, the
  // loop over the tiles came out 5 % slower; kept for two tokens, 10 %).
  struct Sight {
    int limit, first;
    const uint64_t* mask;
  };
  auto sight_of = [&](int n) {
    const int b = n / a.s_q;
    Sight s;
    s.limit = limit_of(n, 0);
    s.mask = tree_of(a, b * a.tok_q + n % a.s_q);
    s.first = !s.mask ? s.limit : a.plan_in_kernel ? row_first_s[n] : paged_first(a, b);
    return s;
  };
  auto seen_of_one = [&](const Sight& s, int t) {
    return (t + 1) * BN <= min(s.limit, s.first) ? ~0ull : paged_seen(t * BN, s.limit, s.first, s.mask, a.tree_words);
  };
  // Two tokens: the first tiles of row n, which both see in whole.
  auto whole_of = [&](int n) {
    const int keys0 = limit_of(n, 0), keys1 = limit_of(n, 1);
    int keys = keys0 == 0 ? keys1 : keys1 == 0 ? keys0 : min(keys0, keys1);
    if (a.tree) keys = min(keys, a.plan_in_kernel ? row_first_s[n] : paged_first(a, n / a.s_q));
    return max(keys, 0) / BN;
  };

  if (warp >= kLoadWarp) {
    reg_dealloc<regs_issue(kPair)>();
    if (warp == kLoadWarp || warp == kPrefetchWarp) {
      // ============================================================ loads, and L2 prefetch a few tiles ahead of them
      const bool loads = warp == kLoadWarp;
      int stage = 0;
      uint32_t phase = 0;
      int fills = 0;   // the ring's first STAGES fills need no free slot
      int tiles = 0;
      auto wait_empty = [&]() { return fills < STAGES || mbar_wait_warp(&empty_bar[stage], phase ^ 1u, kWaitLimit); };
      auto next_stage = [&]() {
        ++fills;
        if (++stage == STAGES) stage = 0, phase ^= 1u;
      };
      const int boxes = BN / a.box_rows;   // 1, 2, 4 or 8 of a tile, one per lane
      const int groups = a.box_rows >> 3;
      int u, n, t0, t1;
      bool whole;
      while (!aborted() && it.next(u, t0, t1, whole)) {
        if (!member_segment<true>(a, keys_p, u, member, n, t0, t1)) continue;
        const int keys = keys_p[n];
        const int32_t* table = a.table + (n / a.s_q) * a.table_stride;
        // Lane l holds the page (-1: no key in the box) and first row there of box 32 * block + l, and of the
        // block behind it.
        int block = -2, page = -1, row = 0, page_next = -1, row_next = 0;
        auto fetch = [&](int blk, int& pg, int& rw) {
          const int key = (32 * blk + lane) * a.box_rows, at = key / a.page_size;
          rw = key - at * a.page_size;
          pg = key < keys ? __ldg(table + at) : -1;
          if (key < keys && (pg < 0 || pg >= a.num_pages)) {   // flagged, and read as zeros: no such page in the map
            pg = a.num_pages;
            if (a.status && rank == 0) atomicOr(a.status, MLA_DEVICE_INDEX_OUT_OF_RANGE);
          }
        };
        auto box_of = [&](int t, int& pg, int& rw) {   // this lane's box of tile t
          const int blk = (t * boxes) >> 5;
          if (blk != block) {
            if (blk == block + 1) page = page_next, row = row_next; else fetch(blk, page, row);
            fetch(blk + 1, page_next, row_next);
            block = blk;
          }
          const int from = (t * boxes + lane) & 31;
          pg = __shfl_sync(0xffffffffu, page, from);
          rw = __shfl_sync(0xffffffffu, row, from);
          if (lane >= boxes) pg = -1;
        };
        auto prefetch_tile = [&](int t) {
          int pg, rw;
          box_of(t, pg, rw);
          if (pg >= 0 && pg < a.num_pages) {
            tma_prefetch_l2_5d(&lat_map, 0, 0, 4 * (int)rank, rw >> 3, pg);
            tma_prefetch_l2_3d(&rope_map, 32 * (int)rank, rw, pg);
          }
          __syncwarp();
        };
        // the query: MMA rows 0..63 and 64..127 are heads 0.. and 64.. of a token, or two tokens (heads or a token that
        // are not there read as zeros: no such coordinate in the map)
        if (loads) {
          const int b = n / a.s_q, i = (n % a.s_q) * kTokens, token = b * a.tok_q + i;
          const int head2 = kPair ? 0 : 64, token2 = !kPair ? token : i + 1 < a.tok_q ? token + 1 : a.n_tokens;
          for (int half = 0; half < 2; ++half) {
            if (!wait_empty()) { fail(); break; }
            if (lane == 0) {
              uint8_t* dst = stages + stage * STAGE_BYTES;
              mbar_arrive_expect_tx(&full_bar[stage], STAGE_BYTES);
              for (int c = 0; c < 2; ++c) {
                tma_load_3d(dst + c * QCHUNK_BYTES, &q_map, &full_bar[stage], dim_base + 64 * (2 * half + c), 0, token);
                tma_load_3d(dst + c * QCHUNK_BYTES + 64 * 128, &q_map, &full_bar[stage], dim_base + 64 * (2 * half + c), head2, token2);
              }
              tma_load_3d(dst + LATENT_BYTES, &qrope_map, &full_bar[stage], RANK + 32 * (int)rank, half ? head2 : 0, half ? token2 : token);
            }
            __syncwarp();
            next_stage();
          }
          if (aborted()) break;
        }
        for (int t = t0; t < t1 && !aborted(); ++t) {
          if (loads) {
            int pg, rw;
            box_of(t, pg, rw);
            const uint32_t there = __ballot_sync(0xffffffffu, pg >= 0);
            if (!wait_empty()) { fail(); break; }
            if (lane == 0) mbar_arrive_expect_tx(&full_bar[stage], __popc(there) * a.box_rows * (STAGE_BYTES / BN));
            __syncwarp();
            if (pg >= 0) {
              uint8_t* dst = stages + stage * STAGE_BYTES;
              tma_load_5d(dst + lane * groups * GROUP_BYTES, &lat_map, &full_bar[stage], 0, 0, 4 * (int)rank, rw >> 3, pg);
              tma_load_3d(dst + LATENT_BYTES + lane * a.box_rows * 64, &rope_map, &full_bar[stage], 32 * (int)rank, rw, pg);
            }
            __syncwarp();
            next_stage();
            if (lane == 0) loaded_s = tiles + 1;
          } else {
            // with the loads of tile t, or at once if those are farther already (a counter, not the stage's barrier: a
            // late reader of a barrier's parity could miss a phase)
            const long long begin = clock64();
            while (loaded_s <= tiles && !abort_s && clock64() - begin < kWaitLimit) __nanosleep(100);
            __syncwarp();
            if (kPrefetchAhead > 0 && t + kPrefetchAhead < t1) prefetch_tile(t + kPrefetchAhead);
            if (t == (t1 - kQueryPrefetchTiles > t0 ? t1 - kQueryPrefetchTiles : t0) && lane == 0) {
              // the next segment's query
              WorkIter peek = it;
              int un, nn, tn0, tn1;
              bool wn;
              while (peek.next(un, tn0, tn1, wn)) {
                if (!member_segment<true>(a, keys_p, un, member, nn, tn0, tn1)) continue;
                const int i = (nn % a.s_q) * kTokens, token = (nn / a.s_q) * a.tok_q + i;
                const int head2 = kPair ? 0 : 64, token2 = kPair ? token + 1 : token;
                for (int c = 0; c < 4; ++c) {
                  tma_prefetch_l2_3d(&q_map, dim_base + 64 * c, 0, token);
                  if (kPair ? i + 1 < a.tok_q : a.heads > 64) tma_prefetch_l2_3d(&q_map, dim_base + 64 * c, head2, token2);
                }
                break;
              }
            }
            __syncwarp();
          }
          ++tiles;
        }
      }
      // Drain: every issued fill must land before this CTA may exit.
      for (int k = fills > STAGES ? fills - STAGES : 0; loads && k < fills; ++k)
        mbar_wait_warp(&full_bar[k % STAGES], (uint32_t)(k / STAGES) & 1u, kWaitLimit);
    } else if (warp == kScoreWarp) {
      // ============================================================ score MMA issuer
      const uint32_t idesc_s = idesc_bf16_f32(128, BN, 0, 0);
      int stage = 0;
      uint32_t phase = 0, tile = 0, seg = 0;
      int u, n, t0, t1;
      bool whole;
      while (!aborted() && it.next(u, t0, t1, whole)) {
        if (!member_segment<true>(a, keys_p, u, member, n, t0, t1)) continue;
        const Sight sight = kPair ? Sight{} : sight_of(n);
        const int whole_tiles = kPair ? whole_of(n) : 0;
        if (!mbar_wait_warp(&q_full, seg & 1u, kWaitLimit)) { fail(); break; }
        for (int half = 0; half < 2; ++half) {   // the query is in TMEM: its two stages are free
          if (lane == 0) mbar_arrive(&empty_bar[stage]);
          if (++stage == STAGES) stage = 0, phase ^= 1u;
        }
        for (int t = t0; t < t1; ++t) {
          uint64_t seen0 = ~0ull, seen1 = ~0ull;
          if constexpr (kPair) {
            if (t >= whole_tiles) seen0 = seen_of(n, 0, t), seen1 = seen_of(n, 1, t);
          } else {
            seen0 = seen1 = seen_of_one(sight, t);
          }
          if (!mbar_wait_warp(&full_bar[stage], phase, kWaitLimit)) { fail(); break; }
          if ((seen0 & seen1) != ~0ull) {
            const uint64_t any = seen0 | seen1, one = seen0 ^ seen1;
            uint8_t* st = stages + stage * STAGE_BYTES;
            // Rows that nobody sees: lane l clears rows l and 32 + l, their pieces of 16 bytes in an order without bank
            // conflicts.
#pragma unroll 1
            for (int r = lane; r < BN; r += 32) {
              if (any >> r & 1) continue;
              uint8_t* lat = st + (r >> 3) * GROUP_BYTES + (r & 7) * 128;
              uint8_t* rope = st + LATENT_BYTES + r * 64;
#pragma unroll 4
              for (int v = 0; v < 32; ++v) *reinterpret_cast<uint4*>(lat + (v >> 3) * 1024 + (((v ^ r) & 7) << 4)) = make_uint4(0, 0, 0, 0);
#pragma unroll
              for (int v = 0; v < 4; ++v) *reinterpret_cast<uint4*>(rope + (((v ^ (r >> 1)) & 3) << 4)) = make_uint4(0, 0, 0, 0);
            }
            // Rows that one token sees, two at a time: lane l looks at piece l of the latents, and l % 4 of the rope dims
            // of the first (lanes 0..3) or second.
            uint64_t poison = 0;
            if constexpr (kPair) {
#pragma unroll 1
              for (uint64_t left = one; left != 0ull;) {
                const int r0 = __ffsll((long long)left) - 1;
                left &= left - 1ull;
                const int r1 = left ? __ffsll((long long)left) - 1 : r0;
                left &= left - (left != 0ull);
                const uint32_t lat = smem_u32(st) + (lane >> 3) * 1024 + (lane & 7) * 16;
                const uint32_t at0 = lat + (r0 >> 3) * GROUP_BYTES + (r0 & 7) * 128, at1 = lat + (r1 >> 3) * GROUP_BYTES + (r1 & 7) * 128;
                const int rr = lane & 4 ? r1 : r0;
                const uint32_t at2 = smem_u32(st) + LATENT_BYTES + rr * 64 + (lane & 3) * 16;
                uint4 w0 = ld_shared_16(at0), w1 = ld_shared_16(at1), w2 = ld_shared_16(at2);
                auto fix = [&](uint32_t at, uint4 w, int r) {
                  bool found = false;
                  w = make_uint4(finite_pair(w.x, found), finite_pair(w.y, found), finite_pair(w.z, found), finite_pair(w.w, found));
                  if (!found) return;
                  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
                  poison |= 1ull << r;
                };
                fix(at0, w0, r0);
                fix(at1, w1, r1);
                fix(at2, w2, rr);
              }
            }
            __syncwarp();
            fence_proxy_async_smem();
            __syncwarp();
            if (kPair && one != 0ull) {
              const uint32_t lo = __reduce_or_sync(0xffffffffu, (uint32_t)poison);
              const uint32_t hi = __reduce_or_sync(0xffffffffu, (uint32_t)(poison >> 32));
              // (tile t + kSlots gets here only once the group of tile t has read S of t + kGroups)
              if (tile > 0 && !mbar_wait_warp(&s_free[(tile - 1) % kGroups], (tile - 1) / kGroups & 1u, kWaitLimit)) { fail(); break; }
              if (lane == 0) {
                poison_s[tile % kSlots] = (uint64_t)hi << 32 | lo;
                mbar_arrive(&poison_full[tile % kSlots]);
              }
            }
          }
          if (tile > 0 && !mbar_wait_warp(&s_free[(tile - 1) % kGroups], (tile - 1) / kGroups & 1u, kWaitLimit)) { fail(); break; }
          tc_fence_after();
          // 16 latent K-steps, then this CTA's two rope K-steps
          const uint64_t d0 = smem_desc(smem_u32(stages + stage * STAGE_BYTES), 16, GROUP_BYTES, kSwizzle128B);
          const uint64_t d_rope = smem_desc(smem_u32(stages + stage * STAGE_BYTES + LATENT_BYTES), 16, 512, kSwizzle64B);
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ts(tmem + TM_S, tmem + TM_Q + c * 32 + k * 8, d0 + (uint64_t)((c * 1024 + k * 32) >> 4), idesc_s, (c | k) != 0);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
              mma_ts(tmem + TM_S, tmem + TM_Q + 128 + k * 8, d_rope + (uint64_t)((k * 32) >> 4), idesc_s, 1u);
            mma_commit(&s_full[tile % kGroups]);
          }
          __syncwarp();
          ++tile;
          if (++stage == STAGES) stage = 0, phase ^= 1u;
        }
        if (aborted()) break;
        ++seg;
      }
      // All score MMAs complete before TMEM is released.
      if (lane == 0) mma_commit(&mma_drain);
      __syncwarp();
      mbar_wait_warp(&mma_drain, 0, kWaitLimit);
    } else if (warp == kPvWarp) {
      // ============================================================ P.V MMA issuer
      const uint32_t idesc_pv = idesc_bf16_f32(128, DV, 0, 1);
      int stage = 0;
      uint32_t tile = 0, seg = 0;
      int u, n, t0, t1;
      bool whole;
      while (!aborted() && it.next(u, t0, t1, whole)) {
        if (!member_segment<true>(a, keys_p, u, member, n, t0, t1)) continue;
        stage = (stage + 2) % STAGES;   // behind the query's
        for (int t = t0; t < t1; ++t) {
          const bool first = (t == t0);
          // O is overwritten by a segment's first P.V: the previous segment's epilogue must have read it.
          if (first && seg > 0 && !mbar_wait_warp(&o_free, (seg - 1) & 1u, kWaitLimit)) { fail(); break; }
          if (!mbar_wait_warp(&p_full, tile & 1u, kWaitLimit)) { fail(); break; }
          tc_fence_after();
          const uint64_t d0 = smem_desc(smem_u32(stages + stage * STAGE_BYTES), 1024, GROUP_BYTES, kSwizzle128B);
          const uint32_t acc0 = first ? 0u : 1u;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < BN / 16; ++k)
              mma_ts(tmem + TM_O, tmem + TM_P + k * 8, d0 + (uint64_t)((k * 2 * GROUP_BYTES) >> 4), idesc_pv, k == 0 ? acc0 : 1u);
            // one commit: the stage barrier also tells the softmax warps that this P.V has completed
            mma_commit(&empty_bar[stage]);
          }
          __syncwarp();
          ++tile;
          if (++stage == STAGES) stage = 0;
        }
        if (aborted()) break;
        ++seg;
      }
      if (a.plan_in_kernel && blockIdx.x == 0) store_pieces(a, keys_p, prefix_p);   // (while the last P.V runs)
      if (lane == 0) mma_commit(&pv_drain);
      __syncwarp();
      mbar_wait_warp(&pv_drain, 0, kWaitLimit);
    }
  } else {
    // ============================================================ exchange, softmax, epilogue
    reg_alloc<regs_softmax(kPair)>();
    const int quarter = warp & 3;
    const uint32_t me = warp >> 2;                        // this group takes the tiles me, me + kGroups, ...
    const int h = 32 * quarter + lane;                    // MMA row = TMEM lane
    const int k_token = kPair ? h >> 6 : 0, head = kPair ? h & 63 : h;
    const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
    const uint32_t before = (me + kGroups - 1) % kGroups; // the group of the tile before
    const uint32_t xin_peer = mapa(smem_u32(xin), peer) + (uint32_t)h * 16u;
    const uint32_t x_full_peer = mapa(smem_u32(&x_full[me]), peer), x_free_peer = mapa(smem_u32(&x_free[me]), peer);
    uint32_t tile = 0, seg = 0, poison_phase = 0, use = 0;   // use: tiles of this group so far
    float half_max = 0.f;   // the segment's largest |half score| (checked against the fp16 exchange's range)
    // P.V(k) of the current segment has completed once its commit arrives on the barrier of its stage: fill k + 2 (seg +
    // 1), two per segment up to this one being queries.  The phase parity identifies the completion: the fill STAGES
    // before has been freed when this is called (this group has waited for a P.V at most kGroups tiles back, and read
    // scores behind this segment's query), and the fill STAGES behind cannot have been: it is a tile of this segment behind
    // the P.V that the caller is yet to allow, or lies behind the epilogue of this segment, which a later segment's
    // P.V's and the one after the next's query wait for.
    auto wait_pv = [&](uint32_t k) -> bool {
      const uint32_t f = k + 2 * (seg + 1);
      return mbar_wait_warp(&empty_bar[f % STAGES], (f / STAGES) & 1u, kWaitLimit);
    };
    // The coming segment's query from its two stages (fills f, f + 1) into TMEM.
    auto take_query = [&](uint32_t f) -> bool {
#pragma unroll 1
      for (int half = 0; half < 2; ++half, ++f) {
        if (!mbar_wait_warp(&full_bar[f % STAGES], (f / STAGES) & 1u, kWaitLimit)) return false;
        const uint8_t* st = stages + (f % STAGES) * STAGE_BYTES;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t r[32];
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            const uint4 w = *reinterpret_cast<const uint4*>(st + c * QCHUNK_BYTES + h * 128 + ((v ^ (h & 7)) << 4));
            r[4 * v] = w.x, r[4 * v + 1] = w.y, r[4 * v + 2] = w.z, r[4 * v + 3] = w.w;
          }
          tmem_st32(tmem + TM_Q + (2 * half + c) * 32 + lane_off, r);
        }
        if (h >> 6 == half) {   // (whole warps)
          uint32_t r[16];
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const uint4 w = *reinterpret_cast<const uint4*>(st + LATENT_BYTES + (h & 63) * 64 + ((v ^ ((h >> 1) & 3)) << 4));
            r[4 * v] = w.x, r[4 * v + 1] = w.y, r[4 * v + 2] = w.z, r[4 * v + 3] = w.w;
          }
          tmem_st16(tmem + TM_Q + 128 + lane_off, r);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full);
      return true;
    };
    // Whether this member has a segment behind `it`.
    auto next_row = [&]() {
      WorkIter peek = it;
      int u, n, t0, t1;
      bool whole;
      while (peek.next(u, t0, t1, whole))
        if (member_segment<true>(a, keys_p, u, member, n, t0, t1)) return true;
      return false;
    };
    int u, n = 0, t0, t1;
    bool whole, live = false;            // live: row n's segment is still in TMEM
    bool more = next_row();              // this member has a segment behind `it`
    int64_t slot = 0;
    float m = -CUDART_INF_F, l = 0.f;    // this group's sum l is relative to 2^m
    // (One place each for the query and for the epilogue: code that runs once per segment is fetched cold, and behind
    // a streamed cache from DRAM.  With a second copy of the query load for the first segment, a boundary took 14,000
    // cycles.)
    for (;;) {
      // ---- the coming segment's query, as soon as the last scores of the one before are read (by the group that will
      // read its first scores)
      if (more && tile % kGroups == me) {
        if (tile > 0 && !mbar_wait_warp(&s_free[(tile - 1) % kGroups], (tile - 1) / kGroups & 1u, kWaitLimit)) { fail(); break; }
        // (and every group has left the segment before this one: its waits on the stages' barriers are over)
        if (seg > 0 && !mbar_wait_warp(&o_free, (seg - 1) & 1u, kWaitLimit)) { fail(); break; }
        tc_fence_after();
        if (!take_query(tile + 2 * (live ? seg + 1 : 0))) { fail(); break; }
      }
      if (live) {
        // ---- the groups' sums (their slots are free once every warp has left the segment before)
        if (seg > 0 && !mbar_wait_warp(&o_free, (seg - 1) & 1u, kWaitLimit)) { fail(); break; }
        sum_s[me][h] = l;
        sum_ref_s[me][h] = m;
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_done);
        if (!mbar_wait_warp(&seg_done, seg & 1u, kWaitLimit)) { fail(); break; }
        {
          float top = m;   // the segment's last reference, which O is relative to, is the largest
  #pragma unroll
          for (uint32_t g = 0; g < kGroups; ++g) top = fmaxf(top, sum_ref_s[g][h]);
          l = 0.f;
  #pragma unroll
          for (uint32_t g = 0; g < kGroups; ++g) {
            const float lg = sum_s[g][h], mg = sum_ref_s[g][h];
            l += mg == top || mg == -CUDART_INF_F ? lg : lg * ex2_approx(mg - top);   // (without a reference: 0, or NaN)
          }
          m = top;
        }
        // ---- epilogue: the segment's last P.V, then this group's part of the context
        if (!wait_pv(tile - 1)) { fail(); break; }
        tc_fence_after();
        const bool blind = kPair && limit_of(n, k_token) == 0;
        if (blind) l = 0.f;
        // (Rows without a query score 0, a key that no token of the row sees holds zeros; the query of a token that sees
        // nothing may hold anything.)
        if (__any_sync(0xffffffffu, !blind && !(half_max <= MLA_FP16_SCORE_LIMIT)) && lane == 0 && a.status)
          atomicOr(a.status, MLA_DEVICE_SCORE_RANGE);
        half_max = 0.f;
        auto drain_o = [&](auto&& store_chunk) {   // of DV / 32 chunks of 32 columns, those of this group
  #pragma unroll 1
          for (int c = (int)me; c < DV / 32; c += kGroups) {
            uint32_t o[32];
            tmem_ld32(tmem + TM_O + c * 32 + lane_off, o);
            tmem_wait_ld_regs(o);
            if (blind) {
  #pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = 0;
            }
            store_chunk(c, o);
          }
        };
        const int i = (n % a.s_q) * kTokens + k_token;
        const int64_t token = (int64_t)(n / a.s_q) * a.tok_q + i;
        const float inv = l != 0.f ? 1.f / l : 0.f;   // 0: no entry; NaN stays NaN
        if (head >= a.heads || i >= a.tok_q) {
          // a padding row: nothing to store
        } else if (whole) {
          const int64_t off = token * a.ctx_row_stride + (int64_t)head * a.ctx_head_stride + dim_base;
          if (a.out_f32) {
            drain_o([&](int c, const uint32_t(&o)[32]) {
              float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.ctx) + off + c * 32);
  #pragma unroll
              for (int v = 0; v < 8; ++v)
                dst[v] = make_float4(__uint_as_float(o[4 * v]) * inv, __uint_as_float(o[4 * v + 1]) * inv,
                                     __uint_as_float(o[4 * v + 2]) * inv, __uint_as_float(o[4 * v + 3]) * inv);
            });
          } else {
            drain_o([&](int c, const uint32_t(&o)[32]) {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.ctx) + off + c * 32);
  #pragma unroll
              for (int v = 0; v < 4; ++v)
                dst[v] = make_uint4(pack_bf16x2(__uint_as_float(o[8 * v]) * inv, __uint_as_float(o[8 * v + 1]) * inv),
                                    pack_bf16x2(__uint_as_float(o[8 * v + 2]) * inv, __uint_as_float(o[8 * v + 3]) * inv),
                                    pack_bf16x2(__uint_as_float(o[8 * v + 4]) * inv, __uint_as_float(o[8 * v + 5]) * inv),
                                    pack_bf16x2(__uint_as_float(o[8 * v + 6]) * inv, __uint_as_float(o[8 * v + 7]) * inv));
            });
          }
          if (rank == 0 && me == 0 && a.lse)
            a.lse[token * a.heads + head] = l != 0.f ? (m + log2f(l)) * 0.69314718055994531f : -CUDART_INF_F;
        } else {
          // Partial: this piece's context normalised by its own sum in fp16, (m, l) in f32 beside it, kept in L2.
          const float m_piece = l == 0.f ? -CUDART_INF_F : m == -CUDART_INF_F ? 0.f : m;   // -inf marks an empty one
          const uint64_t keep = l2_policy_evict_last();
          uint4* dst = a.ws_o + (slot * (RANK / 8) + dim_base / 8) * HEADS + h;
          float vmax = 0.f;
          drain_o([&](int c, const uint32_t(&o)[32]) {
  #pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w[4];
  #pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float x0 = __uint_as_float(o[8 * q + 2 * j]) * inv, x1 = __uint_as_float(o[8 * q + 2 * j + 1]) * inv;
                vmax = fmaxf(vmax, fmaxf(fabsf(x0), fabsf(x1)));   // beyond 65504 the fp16 value is infinite
                const __half2 hv = __floats2half2_rn(x0, x1);
                w[j] = *reinterpret_cast<const uint32_t*>(&hv);
              }
              st_global_v4_policy(dst + (int64_t)(4 * c + q) * HEADS, make_uint4(w[0], w[1], w[2], w[3]), keep);
            }
          });
          if (!(vmax <= 65504.f) && a.status) atomicOr(a.status, MLA_DEVICE_VALUE_RANGE);
          if (rank == 0 && me == 0) {
            st_global_f32_policy(a.ws_ml + (slot * 2) * HEADS + h, m_piece, keep);
            st_global_f32_policy(a.ws_ml + (slot * 2 + 1) * HEADS + h, l, keep);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free);
        ++seg;
      }
      live = false;
      while (it.next(u, t0, t1, whole)) {
        slot = slot_of<true>(a, u, group, member, t0 == 0);
        live = member_segment<true>(a, keys_p, u, member, n, t0, t1);
        if (live) break;
        // Nothing of this row in the group's range: an empty partial (weight 0).
        if (!whole && rank == 0 && me == 0 && head < a.heads) {
          a.ws_ml[(slot * 2) * HEADS + h] = -CUDART_INF_F;
          a.ws_ml[(slot * 2 + 1) * HEADS + h] = 0.f;
        }
      }
      if (!live || aborted()) break;
      more = next_row();
      const Sight sight = kPair ? Sight{} : sight_of(n);
      const int whole_tiles = kPair ? whole_of(n) : 0;
      m = -CUDART_INF_F, l = 0.f;
      for (int t = t0; t < t1; ++t, ++tile) {
        if (tile % kGroups != me) continue;
        uint64_t valid = ~0ull;
        bool one = false;   // kPair: a key that one of the two tokens sees
        if constexpr (kPair) {
          if (t >= whole_tiles) {
            valid = seen_of(n, k_token, t);
            one = valid != seen_of(n, k_token ^ 1, t);
          }
        } else {
          valid = seen_of_one(sight, t);
        }
        // ---- this CTA's partial scores, in f32
        if (!mbar_wait_warp(&s_full[me], use & 1u, kWaitLimit)) { fail(); break; }
        tc_fence_after();
        float x[BN];
        {
          uint32_t sa[32], sb[32];
          tmem_ld32(tmem + TM_S + lane_off, sa);
          tmem_ld32(tmem + TM_S + 32 + lane_off, sb);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[me]);
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = __uint_as_float(sa[k]), x[32 + k] = __uint_as_float(sb[k]);
        }
        // Keys that the other token alone sees: no scores of this one (they would count for the exchange's range).  Keys
        // with something that is not finite in this CTA's dims, seen by one token and cleared for the other: NaN for the
        // one, here and (it crosses with the scores) in the peer.
        if (kPair && one) {
          const uint32_t k = tile % kSlots;
          if (!mbar_wait_warp(&poison_full[k], poison_phase >> k & 1u, kWaitLimit)) { fail(); break; }
          poison_phase ^= 1u << k;
          {
            const uint32_t lo = (uint32_t)valid, hi = (uint32_t)(valid >> 32);
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = lo >> j & 1u ? x[j] : 0.f, x[32 + j] = hi >> j & 1u ? x[32 + j] : 0.f;
          }
          const uint64_t poison = poison_s[k] & valid;
          if (poison != 0ull) {
            const uint32_t lo = (uint32_t)poison, hi = (uint32_t)(poison >> 32);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (lo >> j & 1u) x[j] = CUDART_NAN_F;
              if (hi >> j & 1u) x[32 + j] = CUDART_NAN_F;
            }
          }
        }
        // ---- sent to the peer in fp16, once it has read the tile two back
        const uint32_t xb = (tile & 1u) * XH_BYTES;
        if (tile >= 2 && !mbar_wait_warp(&x_free[(tile - 2) % kGroups], (tile - 2) / kGroups & 1u, kWaitLimit)) { fail(); break; }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int k = 8 * c + 2 * q;
            w[q] = pack_f16x2_sat(x[k], x[k + 1]);
          }
          st_async_v4(xin_peer + xb + (uint32_t)(c * 128 * 16), w[0], w[1], w[2], w[3], x_full_peer);
        }
        if (h == 0) mbar_arrive_expect_tx(&x_full[me], XH_BYTES);
        // While the peer's half is on its way: the largest magnitude (scores that fp16 cannot hold are rare: it decides
        // once whether ours are clamped too), and the reference that the group of the tile before has handed on.
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) top = fmax3(top, fabsf(x[k]), fabsf(x[32 + k]));
        half_max = fmaxf(half_max, top);
        if (__any_sync(0xffffffffu, !(top <= 65504.f))) {
#pragma unroll
          for (int k = 0; k < BN; ++k) x[k] = clamp_nan(x[k], 65504.f);
        }
        float m_ref = -CUDART_INF_F;
        if (t > t0) {
          if (!mbar_wait_warp(&ref_full[before][quarter], (tile - 1) / kGroups & 1u, kWaitLimit)) { fail(); break; }
          m_ref = ref_s[before][h];
        }
        // ---- the peer's half (its remote stores complete as transaction bytes on this barrier)
        if (!mbar_wait_warp(&x_full[me], use & 1u, kWaitLimit)) { fail(); break; }
        ++use;
        const uint8_t* const xi = xin + xb + h * 16;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 i4 = *reinterpret_cast<const uint4*>(xi + c * 128 * 16);
          const uint32_t iw[4] = {i4.x, i4.y, i4.z, i4.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            x[8 * c + 2 * q] = add_f16lo(iw[q], x[8 * c + 2 * q]);
            x[8 * c + 2 * q + 1] = add_f16hi(iw[q], x[8 * c + 2 * q + 1]);
          }
        }
        if (valid != ~0ull) {   // (a rolled loop over the keys that are not seen, in shared memory, took 130 cycles for each)
          const uint32_t lo = (uint32_t)valid, hi = (uint32_t)(valid >> 32);
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            x[k] = lo >> k & 1u ? x[k] : -CUDART_INF_F;
            x[32 + k] = hi >> k & 1u ? x[32 + k] : -CUDART_INF_F;
          }
        }
        // ---- tile maximum (three-input max tree)
        float mx;
        {
          float m21[22];
#pragma unroll
          for (int k = 0; k < 21; ++k) m21[k] = fmax3(x[3 * k], x[3 * k + 1], x[3 * k + 2]);
          m21[21] = x[63];
          float m7[8];
#pragma unroll
          for (int k = 0; k < 7; ++k) m7[k] = fmax3(m21[3 * k], m21[3 * k + 1], m21[3 * k + 2]);
          m7[7] = m21[21];
          mx = fmax3(fmax3(m7[0], m7[1], m7[2]), fmax3(m7[3], m7[4], m7[5]), fmaxf(m7[6], m7[7]));
        }
        // Every score above fed mx, so the warp holds all of this tile's data: the buffer is freed with a relaxed
        // arrive ordered by that dependency.
        __syncwarp();
        if (lane == 0) mbar_arrive_remote_relaxed_dep(x_free_peer, __float_as_uint(mx));
        mx *= a.scale_log2;   // (from here on in log2 units)
        // ---- the reference moves only when the tile's maximum exceeds it by more than the threshold (or on the first
        // visible entry)
        const bool moved = mx != -CUDART_INF_F && (m_ref == -CUDART_INF_F || mx > m_ref + kRescaleThreshold);
        const float m_new = moved ? mx : m_ref;
        ref_s[me][h] = m_new;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ref_full[me][quarter]);
        const bool rescale = moved && m_ref != -CUDART_INF_F;
        if (m != m_new) {
          if (m != -CUDART_INF_F) l *= ex2_approx(m - m_new);   // (a sum without a reference is 0, or NaN)
          m = m_new;
        }
        // ---- p = 2^(x - m)
        const float shift = m_new == -CUDART_INF_F ? 0.f : -m_new;
        uint32_t pk[32];
        float2 ps2[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) ps2[k] = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < BN; k += 2) {
          const float2 xs = fma_f32x2(make_float2(x[k], x[k + 1]), make_float2(a.scale_log2, a.scale_log2), make_float2(shift, shift));
          const float p0 = ex2_approx(xs.x);
          const float p1 = ex2_approx(xs.y);
          ps2[(k >> 1) & 7] = add_f32x2(ps2[(k >> 1) & 7], make_float2(p0, p1));
          const __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
          pk[k >> 1] = *reinterpret_cast<const uint32_t*>(&pb);
        }
        ps2[0] = add_f32x2(add_f32x2(ps2[0], ps2[1]), add_f32x2(ps2[2], ps2[3]));
        ps2[4] = add_f32x2(add_f32x2(ps2[4], ps2[5]), add_f32x2(ps2[6], ps2[7]));
        ps2[0] = add_f32x2(ps2[0], ps2[4]);
        l += ps2[0].x + ps2[0].y;
        // ---- P into TMEM once the previous P.V has consumed it (and O is stable; the last of a segment has been waited
        // for in its epilogue)
        if (t > t0 && !wait_pv(tile - 1)) { fail(); break; }
        tc_fence_after();
        // tcgen05.ld / st are warp-collective: the whole warp takes the
        // rescale pass when any of its rows needs it, the others with factor 1.
        if (__any_sync(0xffffffffu, rescale)) {
          const float f = rescale ? ex2_approx(m_ref - m_new) : 1.f;
#pragma unroll 1
          for (int c = 0; c < DV / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tmem + TM_O + c * 32 + lane_off, o);
            tmem_wait_ld_regs(o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st32(tmem + TM_O + c * 32 + lane_off, o);
          }
        }
        tmem_st32(tmem + TM_P + lane_off, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full);
      }
      if (aborted()) break;
    }
  }

  // ---------------------------------------------------------------- teardown
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the peer no longer writes into this CTA's shared memory
  if (warp == kScoreWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_tc_paged(const DecodeGeometry& g, int out_dtype, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
  if (workspace_bytes < tc_paged_workspace(g.batch * g.s_q)) return cudaErrorInvalidValue;
  if (g.heads != 64 && g.heads != HEADS) return cudaErrorInvalidValue;
  TcDecodeArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(g.q);
  a.q_row_stride = g.q_row_stride;
  a.q_head_stride = g.q_head_stride;
  a.kv_len = g.kv_len;
  a.tok_q = g.s_q;
  a.tokens = g.heads == 64 && g.s_q > 1 ? 2 : 1;
  a.s_q = (g.s_q + a.tokens - 1) / a.tokens;
  a.n_q = g.batch * a.s_q;
  a.n_tokens = g.batch * g.s_q;
  a.heads = g.heads;
  a.scale_log2 = g.scale_log2;
  a.ctx = g.ctx_out;
  a.ctx_row_stride = g.ctx_row_stride;
  a.ctx_head_stride = g.ctx_head_stride;
  a.out_f32 = out_dtype == MLA_DTYPE_F32;
  a.lse = g.lse_out;
  a.status = g.device_status;
  a.t_max = g.t_max;
  a.table = g.table;
  a.table_stride = g.table_stride;
  a.page_size = g.page_size;
  a.num_pages = g.num_pages;
  a.counts = g.counts;
  a.tree = g.tree;
  a.tree_words = g.tree_words;
  a.num_clusters = device_sm_count() / 2;
  a.width = a.s_q < kLockstep ? a.s_q : kLockstep;
  a.n_units = (a.n_q + a.width - 1) / a.width;
  a.min_tiles = kMinTilesPerGroup;
  a.start_charge = kStartCharge;
  a.charge_min_span = kChargeSpan;
  a.plan_in_kernel = a.n_q <= kMaxRowsInKernelPlan ? 1 : 0;
  a.box_rows = BN;   // the largest box that divides a tile and a page
  while (g.page_size % a.box_rows != 0) a.box_rows >>= 1;
  if (a.box_rows < 8) return cudaErrorInvalidValue;
  lay_out_workspace(a, workspace);

  CUtensorMap lat_map, rope_map, q_map, qrope_map;
  {
    const uint64_t row = (uint64_t)g.latent_row_stride * 2;
    const uint64_t page = g.num_pages > 1 ? (uint64_t)g.latent_page_stride * 2 : row * g.page_size;   // (one page: no stride)
    const uint64_t dims[5] = {64, 8, RANK / 64, (uint64_t)g.page_size / 8, (uint64_t)g.num_pages};
    const uint64_t strides[4] = {row, 128, 8 * row, page};
    const uint32_t box[5] = {64, 8, 4, (uint32_t)a.box_rows / 8, 1};
    if (!encode_tmap_bf16(&lat_map, g.latent, 5, dims, strides, box)) return cudaErrorInvalidValue;
  }
  {
    const uint64_t row = (uint64_t)g.rope_row_stride * 2;
    const uint64_t page = g.num_pages > 1 ? (uint64_t)g.rope_page_stride * 2 : row * g.page_size;
    const uint64_t dims[3] = {(uint64_t)g.rope_dim, (uint64_t)g.page_size, (uint64_t)g.num_pages};
    const uint64_t strides[2] = {row, page};
    const uint32_t box[3] = {32, (uint32_t)a.box_rows, 1};
    if (!encode_tmap_bf16(&rope_map, g.rope, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B)) return cudaErrorInvalidValue;
  }
  {
    const uint64_t row = a.n_tokens > 1 ? (uint64_t)g.q_row_stride * 2 : (uint64_t)g.q_head_stride * 2 * g.heads;
    const uint64_t dims[3] = {(uint64_t)(g.rank + g.rope_dim), (uint64_t)g.heads, (uint64_t)a.n_tokens};
    const uint64_t strides[2] = {(uint64_t)g.q_head_stride * 2, row};
    const uint32_t box[3] = {64, 64, 1}, rbox[3] = {32, 64, 1};
    if (!encode_tmap_bf16(&q_map, g.q, 3, dims, strides, box) ||
        !encode_tmap_bf16(&qrope_map, g.q, 3, dims, strides, rbox, CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  }
  const bool lockstep = a.width > 1;
  auto* const kernel = a.tokens == 2 ? (lockstep ? tc_paged_kernel<kPrefetchAheadGroup, true> : tc_paged_kernel<kPrefetchAheadRow, true>)
                                     : (lockstep ? tc_paged_kernel<kPrefetchAheadGroup, false> : tc_paged_kernel<kPrefetchAheadRow, false>);
  {
    // The warpgroups' register shares wait for one another: a build with other
    // registers than they add up to must not be launched.
    static const bool fits = [] {
      for (auto* k : {tc_paged_kernel<kPrefetchAheadGroup, true>, tc_paged_kernel<kPrefetchAheadRow, true>,
                      tc_paged_kernel<kPrefetchAheadGroup, false>, tc_paged_kernel<kPrefetchAheadRow, false>}) {
        cudaFuncAttributes attr;
        if (cudaFuncGetAttributes(&attr, k) != cudaSuccess || attr.numRegs < kRegsLaunch) return false;
      }
      return true;
    }();
    if (!fits) return cudaErrorInvalidConfiguration;
    const cudaError_t ea = set_max_dynamic_smem(kernel, SMEM_BYTES);
    if (ea != cudaSuccess) return ea;
  }
  cudaError_t e = a.plan_in_kernel ? cudaSuccess : launch_split_plan(a, stream);
  if (e == cudaSuccess) e = launch_pdl(kernel, dim3(2 * a.num_clusters), dim3(THREADS), SMEM_BYTES, stream, lat_map, rope_map, q_map, qrope_map, a);
  if (e == cudaSuccess) e = launch_split_combine(a, stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mla
