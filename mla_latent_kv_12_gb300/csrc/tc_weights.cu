// Accumulated attention weight of every cached key on the tensor cores:
//   W_t <- decay W_t + sum_{i, h} 2^(s_{i,h,t} scale log2(e) - lse_{i,h} log2(e)).
//
// The scores are one GEMM per query token, S[128 heads x 64 keys] =
// Q[128 x 576] . K^T, with the probabilities normalised by a given lse, so
// nothing has to be known about other keys: each tile of 64 keys is finished
// on its own.  The whole query of a token fits TMEM as the MMA's A operand (288
// columns of packed 16-bit pairs) beside two score buffers (2 x 64), so a CTA scores
// all 576 features itself and no SM pair is needed.  At one query token it is
// bound by the cache read (1152 or 641 bytes against 147 kflop per key: 0.17
// or 0.09 ns at the measured copy rate, 0.076 ns at the measured bf16 rate):
// 32 rows, 498,051 keys, take 95 to 103 us over bf16 (5.6 to 6.1 TB/s) and 85
// us over 8 bits (3.8 TB/s; the N = 64 MMAs alone, without conversion and fetch,
// 66); four tokens of 8 rows of 16384 keys 91 and 110 us.
//
//  * One persistent CTA per SM takes an equal range of the flattened tiles of
//    all rows.  With several query tokens a range is walked in chunks (of a bf16
//    cache: that stay in L2), once per token: the weights of a key are always
//    updated by the same thread, in token order (no atomics, the same bits
//    every time).
//    Two tokens of 64 heads share the MMA's 128 rows and a pass.
//  * bf16 cache: warp 0 loads [64 keys x 576] tiles by TMA into a three-stage
//    ring (nine boxes of 64 dims, 128-byte swizzle).  8-bit cache: warps
//    10..17 fetch codes and write their fp16 values into the same layout
//    (q8_tiles.cuh), warp 0 loads the rope boxes; the latent part of the query
//    is converted to fp16 too.
//  * Warp 1 issues the 36 MMAs of a tile.  Warps 2..9 load each token's query
//    into TMEM; two groups of four (one thread per head) take the tiles in
//    turn, turn scores into probabilities and sum them over a warp's 32 heads
//    with a shuffle tree that halves the keys per lane at every step; the four
//    warps' sums meet in shared memory.
#include <cuda_bf16.h>

#include "mla_internal.h"
#include "q8_tiles.cuh"
#include "tc_common.cuh"
#include "tc_host.h"

namespace mla {
namespace {

using namespace tc;

constexpr int BN = 64;                    // keys per tile
constexpr int BOX_BYTES = BN * 128;       // [64 keys][64 dims] bf16
constexpr int BOXES = 9;                  // 8 of latent dims, 1 of rope dims
constexpr int STAGE_BYTES = BOXES * BOX_BYTES;
constexpr int STAGES = 3, STAGES_Q8 = 2;   // 8-bit: the third stage's memory holds the fetch's slots
constexpr uint32_t TM_Q = 0, TM_S = 288;  // TMEM columns
constexpr int kSumWarp = 2, kSumGroups = 2;   // two groups of four warps
constexpr int kConvertWarp = kSumWarp + 4 * kSumGroups, kConvertWarps = 8, kConvertThreads = 32 * kConvertWarps;
constexpr int kThreads = 32 * kConvertWarp, kThreadsQ8 = kThreads + kConvertThreads;
using WeightFetch = Q8Fetch<32, kConvertThreads>;
constexpr int SMEM_BYTES = STAGES * STAGE_BYTES, SMEM_BYTES_Q8 = STAGES_Q8 * STAGE_BYTES + 2 * WeightFetch::kSlotBytes;
constexpr long long kWaitLimit = 1LL << 32;   // clock cycles (~2 s)
// Tiles that several query tokens walk before the next ones.  A pass begins
// with a drained pipeline, so chunks are long.  Over bf16 as long as the L2 (129
// MB) allows: 152 CTAs x 8 tiles x 72 KB = 88 MB; from 11 on full chunks are read
// from memory again (four tokens of 8 rows of 14592 keys: 77 us with 8 or 10,
// 91 with 12).  Over 8 bits a pass is slower than its reads from memory, and
// its chunks do not stay in L2 (28 tiles x 40 KB x 152 CTAs = 175 MB): with 8 / 15
// / 20 / 28 / 60 tiles four tokens of 8 rows of 65536 keys (54 tiles per CTA)
// take 369 / 323 / 306 / 296 / 280 us, of 4 such rows 210 / 179 / 181 / 166 /
// 167, three of 5 rows of 40001 132 / 120 / 113 / 112 / 112, two of 6 rows of
// 30011 89 / 83 / 75 / 75 / 75.
constexpr int kChunkTiles = 8, kChunkTilesQ8 = 28;
constexpr int kRopeAhead = 6;      // tiles ahead that an 8-bit cache's rope keys are pulled into L2
constexpr int kWeightsAhead = 8;   // tiles ahead that weights are pulled into L2

struct WeightArgs {
  DecodeGeometry g;
  const float* lse;
  float* weights;
  int64_t weights_batch_stride;
  float decay;
  int32_t n_new;
  int32_t batch_in_map, rows_in_map;   // whether the cache's batch axis and the query's row axis are mapped
};

__device__ __forceinline__ int window_tiles(const DecodeGeometry& g, int b, bool flag) {
  const int start = g.kv_start ? g.kv_start[b] : 0, len = g.kv_len[b];
  const bool fits = len >= 0 && start >= 0 && (int64_t)start + len <= g.t_max;
  const bool ok = fits && (!g.codes || (start & ((1 << g.block_shift) - 1)) == 0);
  if (!ok) {
    if (flag && g.device_status)
      atomicOr(g.device_status, fits ? MLA_DEVICE_BAD_BLOCK_START : MLA_DEVICE_INDEX_OUT_OF_RANGE);
    return 0;
  }
  return (len + BN - 1) / BN;
}

// A CTA's share of the work: passes of one query token (two of 64 heads, which
// share the MMA's 128 rows) over tiles [t0, t1) of one batch row.
struct Passes {
  int b, t, left, row_tiles;   // current row, next tile, tiles left in the CTA's range, tiles of the row
  int i, t0, t1;               // (first) token, current chunk
  static __device__ int tokens(const DecodeGeometry& g) { return g.heads == 64 ? 2 : 1; }
  __device__ void init(int b0, int first, int count, const DecodeGeometry& g) {
    b = b0;
    t = first;
    left = count;
    row_tiles = count > 0 ? window_tiles(g, b, false) : 0;
    i = g.s_q;                 // no chunk yet
    t0 = t1 = 0;
  }
  // The next pass; `fresh`: its query is not the previous pass's.
  __device__ bool next(const DecodeGeometry& g, bool& fresh) {
    fresh = true;
    if (i + tokens(g) < g.s_q) {
      i += tokens(g);
      return true;
    }
    if (left <= 0) return false;
    const int was = t1 == 0 ? -1 : b;
    while (t >= row_tiles) {
      ++b;
      t = 0;
      row_tiles = window_tiles(g, b, false);
    }
    int n = min(left, row_tiles - t);
    if (g.s_q > tokens(g)) n = min(n, g.codes ? kChunkTilesQ8 : kChunkTiles);
    i = 0;
    t0 = t;
    t1 = t + n;
    t += n;
    left -= n;
    fresh = g.s_q > tokens(g) || was != b;
    return true;
  }
};

template <bool kQ8>
__global__ void __launch_bounds__(kQ8 ? kThreadsQ8 : kThreads, 1)
    tc_key_weights_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap lat_map,
                          const __grid_constant__ CUtensorMap rope_map, const __grid_constant__ WeightArgs a) {
  constexpr int kStages = kQ8 ? STAGES_Q8 : STAGES;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if ((smem_u32(smem_raw) & 1023u) != 0) {   // the same in every CTA: nothing waits on anything yet
    if (threadIdx.x == 0 && a.g.device_status) atomicOr(a.g.device_status, MLA_DEVICE_LAYOUT);
    return;
  }
  uint8_t* stages = smem_raw;
  __shared__ __align__(8) uint64_t full_bar[kStages], empty_bar[kStages], s_full[2], s_free[2], q_full, drain;
  __shared__ uint32_t tmem_base_s;
  __shared__ volatile int abort_s;
  __shared__ int first_row_s, first_tile_s, count_s;
  __shared__ float part_s[kSumGroups][4][BN];
  const DecodeGeometry& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&q_map);
    tma_prefetch_desc(&rope_map);
    if constexpr (!kQ8) tma_prefetch_desc(&lat_map);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], kQ8 ? kConvertWarps + 1 : 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(&s_full[k], 1);
      mbar_init(&s_free[k], 4);
    }
    mbar_init(&q_full, 4 * kSumGroups);
    mbar_init(&drain, 1);
    abort_s = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_s, 512);
    tmem_relinquish();
  }
  pdl_wait();
  if (warp == 0) {
    // This CTA's tiles of the flattened sequence: the rows' tiles are counted
    // (32 rows at a time), then walked again to the range's first row.
    int total = 0;
    for (int b0 = 0; b0 < g.batch; b0 += 32)
      total += b0 + lane < g.batch ? window_tiles(g, b0 + lane, blockIdx.x == 0) : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const int per = (total + gridDim.x - 1) / (int)gridDim.x;
    const long long begin = (long long)per * blockIdx.x;
    const int count = (int)max(0LL, min((long long)per, (long long)total - begin));
    if (lane == 0) count_s = count;
    int before = 0;
    for (int b0 = 0; count > 0 && b0 < g.batch; b0 += 32) {
      const int mine = b0 + lane < g.batch ? window_tiles(g, b0 + lane, false) : 0;
      int inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      const int lo = before + inc - mine;
      const bool here = begin >= lo && begin < before + inc;
      if (here) {
        first_row_s = b0 + lane;
        first_tile_s = (int)(begin - lo);
      }
      if (__any_sync(0xffffffffu, here)) break;
      before += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  auto aborted = [&]() -> bool { return __any_sync(0xffffffffu, abort_s != 0); };
  auto fail = [&]() {
    abort_s = 1;
    if (g.device_status) atomicOr(g.device_status, MLA_DEVICE_TIMEOUT);
  };
  // One half (64 heads, of the second token where a pass has two) of a pass's
  // query into a stage: the boxes of a tile.  (A second token that is not there
  // is the first one again; its sums are dropped.)
  auto load_query = [&](int stage, int b, int i, int half) {
    const bool two = Passes::tokens(g) == 2;
    const int row = b * g.s_q + (two && i + half < g.s_q ? i + half : i);
    mbar_arrive_expect_tx(&full_bar[stage], STAGE_BYTES);
    for (int c = 0; c < BOXES; ++c)
      tma_load_3d(stages + stage * STAGE_BYTES + c * BOX_BYTES, &q_map, &full_bar[stage], 64 * c, two ? 0 : 64 * half,
                  a.rows_in_map ? row : 0);
  };
  Passes it;
  it.init(count_s > 0 ? first_row_s : 0, count_s > 0 ? first_tile_s : 0, count_s, g);
  bool fresh;

  if (warp == 0) {
    // ============================================================ TMA producer (8-bit: of queries and rope keys)
    int stage = 0, fills = 0;
    uint32_t phase = 0;
    while (!aborted() && it.next(g, fresh)) {
      const int start = g.kv_start ? g.kv_start[it.b] : 0;
      const int z = a.batch_in_map ? it.b : 0;
      bool ok = true;
      for (int half = 0; fresh && ok && half < 2; ++half) {
        if (fills >= kStages && !mbar_wait_warp(&empty_bar[stage], phase ^ 1u, kWaitLimit)) { fail(); ok = false; break; }
        ++fills;
        if (lane == 0) load_query(stage, it.b, it.i, half);
        __syncwarp();
        if (++stage == kStages) stage = 0, phase ^= 1u;
      }
      for (int t = it.t0; ok && t < it.t1; ++t) {
        if (fills >= kStages && !mbar_wait_warp(&empty_bar[stage], phase ^ 1u, kWaitLimit)) { fail(); break; }
        ++fills;   // (counts what was issued)
        if (lane == 0) {
          mbar_arrive_expect_tx(&full_bar[stage], kQ8 ? BOX_BYTES : STAGE_BYTES);
          uint8_t* st = stages + stage * STAGE_BYTES;
          if constexpr (!kQ8)
            for (int c = 0; c < 8; ++c)
              tma_load_3d(st + c * BOX_BYTES, &lat_map, &full_bar[stage], 64 * c, start + t * BN, z);
          tma_load_3d(st + 8 * BOX_BYTES, &rope_map, &full_bar[stage], 0, start + t * BN, z);
          if (kQ8 && t + kRopeAhead < it.t1) tma_prefetch_l2_3d(&rope_map, 0, start + (t + kRopeAhead) * BN, z);
        }
        __syncwarp();
        if (++stage == kStages) stage = 0, phase ^= 1u;
      }
    }
    // every issued load lands before this CTA may exit: fill k of a stage completes its phase k
    for (int k = fills > kStages ? fills - kStages : 0; k < fills; ++k)
      mbar_wait_warp(&full_bar[k % kStages], (uint32_t)(k / kStages) & 1u, kWaitLimit);
  } else if (kQ8 && warp >= kConvertWarp) {
    // ============================================================ 8-bit producers
    // A warp takes one key at a time.
    const int cw = warp - kConvertWarp;
    WeightFetch fetch;
    fetch.slot0 = smem_u32(stages + kStages * STAGE_BYTES) + (cw * 32 + lane) * 16;
    fetch.codes0 = fetch.slot0 - 16 * lane + 8 * lane;
    fetch.key0 = cw;
    fetch.peers = 0;
    fetch.mine = lane % WeightFetch::kIters;
    const uint32_t box0 = smem_u32(stages) + (lane >> 3) * BOX_BYTES + cw * 128 + (((lane & 7) ^ cw) << 4);
    int stage = 0, fills = 0;
    uint32_t phase = 0;
    while (!aborted() && it.next(g, fresh)) {
      const int b = it.b, t0 = it.t0, t1 = it.t1;
      Q8Rows rows;
      rows.codes = g.codes + b * g.codes_batch_stride + 16 * lane;
      rows.codes_stride = g.codes_row_stride;
      rows.scales = g.scales + b * g.scales_batch_stride;
      rows.shift = g.block_shift;
      rows.start = g.kv_start ? g.kv_start[b] : 0;
      rows.entries = rows.limit = g.kv_len[b];
      rows.list = nullptr;
      rows.status = lane < WeightFetch::kIters ? g.device_status : nullptr;
      // Tile t is converted while the copies of t + 1 and (from its end on) t + 2 are in flight.
      int pos = fetch.my_position(rows, t0);
      int e_now = fetch.my_exponent(rows, pos);
      fetch.issue_window(rows, t0, 0);
      cp_async_commit();
      pos = fetch.my_position(rows, t0 + 1);
      int e_next = fetch.my_exponent(rows, pos);
      if (t0 + 1 < t1) fetch.issue_window(rows, t0 + 1, 1);
      cp_async_commit();
      bool ok = true;
      for (int half = 0; fresh && ok && half < 2; ++half) {
        if (fills >= kStages && !mbar_wait_warp(&empty_bar[stage], phase ^ 1u, kWaitLimit)) { fail(); ok = false; break; }
        ++fills;
        if (lane == 0) mbar_arrive(&full_bar[stage]);   // (a half of the query, loaded by warp 0)
        __syncwarp();
        if (++stage == kStages) stage = 0, phase ^= 1u;
      }
      for (int t = t0; ok && t < t1; ++t) {
        const int slot = (t - t0) & 1;
        if (fills >= kStages && !mbar_wait_warp(&empty_bar[stage], phase ^ 1u, kWaitLimit)) { fail(); break; }
        ++fills;
        cp_async_wait<1>();   // this tile's pieces
        const uint32_t off = stage * STAGE_BYTES;
        fetch.check_exponent(rows.status, e_now);
        fetch.convert<4 * BOX_BYTES>(slot, e_now, box0 + off);
        fence_proxy_async_smem();   // generic-proxy writes, read by the MMAs
        __syncwarp();
        if (lane == 0) mbar_arrive(&full_bar[stage]);
        e_now = e_next;
        if (t + 2 < t1) {
          pos = fetch.my_position(rows, t + 2);
          e_next = fetch.my_exponent(rows, pos);
          fetch.issue_window(rows, t + 2, slot);
        }
        cp_async_commit();
        if (++stage == kStages) stage = 0, phase ^= 1u;
      }
      if (t0 == 0 && g.device_status) {
        // Once per query row: values that fp16 cannot hold.  These warps run
        // ahead of the others, whose registers are full (checked as they are
        // converted, four tokens of 8 rows of 16384 keys took 165 us, against 145 then).
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(g.q) + ((int64_t)b * g.s_q + it.i) * g.q_row_stride;
        const int rows = min(Passes::tokens(g), g.s_q - it.i) * g.heads;
        uint32_t top = 0;
#pragma unroll 4
        for (int h = cw; h < rows; h += kConvertWarps)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const __nv_bfloat16* head = q + (h >= g.heads ? g.q_row_stride + (int64_t)(h - g.heads) * g.q_head_stride : (int64_t)h * g.q_head_stride);
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(head) + 32 * v + lane);
            top = max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(top, x.x), x.y), x.z), x.w);
          }
        if (beyond_f16(top)) atomicOr(g.device_status, MLA_DEVICE_VALUE_RANGE);
      }
      cp_async_wait<0>();   // the slots are free for the next pass
    }
  } else if (warp == 1) {
    // ============================================================ MMA issuer
    const uint32_t idesc_rope = idesc_bf16_f32(128, BN, 0, 0), idesc = kQ8 ? idesc_f16_f32(128, BN, 0, 0) : idesc_rope;
    int stage = 0;
    uint32_t phase = 0, tile = 0, queries = 0;
    while (!aborted() && it.next(g, fresh)) {
      if (fresh) {
        if (!mbar_wait_warp(&q_full, queries++ & 1u, kWaitLimit)) { fail(); break; }
        for (int half = 0; half < 2; ++half) {   // the query's stages have been read
          if (lane == 0) mbar_arrive(&empty_bar[stage]);
          if (++stage == kStages) stage = 0, phase ^= 1u;
        }
        __syncwarp();
      }
      for (int t = it.t0; t < it.t1; ++t, ++tile) {
        const uint32_t buf = tile & 1u;
        if (tile >= 2 && !mbar_wait_warp(&s_free[buf], ((tile >> 1) - 1) & 1u, kWaitLimit)) { fail(); break; }
        if (!mbar_wait_warp(&full_bar[stage], phase, kWaitLimit)) { fail(); break; }
        tc_fence_after();
        const uint64_t d0 = smem_desc(smem_u32(stages + stage * STAGE_BYTES), 16, 1024, kSwizzle128B);
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < BOXES; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts(tmem + TM_S + buf * BN, tmem + TM_Q + c * 32 + k * 8,
                     d0 + (uint64_t)((c * BOX_BYTES + k * 32) >> 4), c < 8 ? idesc : idesc_rope, (c | k) != 0);
          mma_commit(&empty_bar[stage]);
          mma_commit(&s_full[buf]);
        }
        __syncwarp();
        if (++stage == kStages) stage = 0, phase ^= 1u;
      }
    }
    if (lane == 0) mma_commit(&drain);   // every MMA completes before TMEM is released
    __syncwarp();
    mbar_wait_warp(&drain, 0, kWaitLimit);
  } else if (warp >= kSumWarp && warp < kConvertWarp) {
    // ============================================================ probabilities and sums
    const int group = (warp - kSumWarp) >> 2, quarter = warp & 3;
    const int h = 32 * quarter + lane;   // MMA row
    const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
    const int token = h / g.heads;       // of the pass's tokens
    const int k_mine = threadIdx.x - 32 * (kSumWarp + 4 * group);   // key of a tile whose weight this thread updates (first two warps)
    uint32_t tile = 0, fill = 0;   // tiles and ring fills of all passes so far
    float lse2 = 0.f;
    // A group's warps meet in barriers at every pass and tile, so they leave together.
    bool stop = false, arrived = true;
    auto leave = [&]() -> bool {
      stop = named_sync_or(1 + group, 128, !arrived || abort_s != 0);
      if (stop && !arrived) fail();
      return stop;
    };
    while (!stop && it.next(g, fresh)) {
      const int b = it.b, len = g.kv_len[b];
      const int64_t start = g.kv_start ? g.kv_start[b] : 0;
      const bool real = it.i + token < g.s_q;
      const int limit = min(len, len - g.s_q + it.i + token + 1);
      if (fresh) {
        // The query into TMEM, a head per thread, every other box by either
        // group.  Every MMA of the previous passes has completed once its last
        // scores are there.
        lse2 = real ? a.lse[((int64_t)b * g.s_q + it.i) * g.heads + h] * 1.4426950408889634f : 0.f;   // (h: into the second token's)
        const uint32_t k = fill + (quarter >> 1);
        arrived = tile == 0 || mbar_wait_warp(&s_full[(tile - 1) & 1u], ((tile - 1) >> 1) & 1u, kWaitLimit);
        arrived = mbar_wait_warp(&full_bar[k % kStages], (k / kStages) & 1u, kWaitLimit) && arrived;
        if (leave()) break;
        tc_fence_after();
        const uint32_t row = smem_u32(stages) + (k % kStages) * STAGE_BYTES + (h & 63) * 128;
        for (int c = group; c < BOXES; c += kSumGroups) {
          uint32_t r[32];
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            const uint4 x = ld_shared_16(row + c * BOX_BYTES + ((v ^ (h & 7)) << 4));
            r[4 * v] = x.x, r[4 * v + 1] = x.y, r[4 * v + 2] = x.z, r[4 * v + 3] = x.w;
          }
          if (kQ8 && c < 8) {
#pragma unroll
            for (int v = 0; v < 32; ++v) r[v] = bf16x2_to_f16x2(r[v]);
          }
          tmem_st32(tmem + TM_Q + c * 32 + lane_off, r);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full);
        fill += 2;
      }
      float* w_row = a.weights + b * a.weights_batch_stride + start;
      // The weight so far of this thread's key of tile t, read a tile ahead of
      // its use, its lines pulled into L2 before that (read in the tile's own
      // iteration, the latency of a cold line bound the kernel).  The first token's pass
      // decays it, from the n_new newest keys on with 0.
      const int64_t kept_keys = it.i > 0 ? len : a.decay != 0.f ? (int64_t)len - a.n_new : 0;
      const float factor = it.i > 0 ? 1.f : a.decay;
      auto weight_of = [&](int t) -> float {
        const int key = t * BN + k_mine;
        return t < it.t1 && k_mine < BN && key < kept_keys ? w_row[key] : 0.f;
      };
      // Group t % 2 takes tile t of a row in every token's pass: a weight has one owner.
      const int first = it.t0 + ((it.t0 ^ group) & 1);
      float old_next = weight_of(first);
      const uint32_t tile0 = tile;
      tile += it.t1 - it.t0;
      fill += it.t1 - it.t0;
      for (int t = first; t < it.t1; t += kSumGroups) {
        const uint32_t my_tile = tile0 + (t - it.t0), buf = my_tile & 1u;
        const int key = t * BN + k_mine;
        const float old = old_next;
        old_next = weight_of(t + kSumGroups);
        if (k_mine < BN && (k_mine & 31) == 0 && key + kWeightsAhead * BN < len) prefetch_l2(w_row + key + kWeightsAhead * BN);
        arrived = mbar_wait_warp(&s_full[buf], (my_tile >> 1) & 1u, kWaitLimit);
        tc_fence_after();
        uint32_t s[2][32];
        tmem_ld32(tmem + TM_S + buf * BN + lane_off, s[0]);
        tmem_ld32(tmem + TM_S + buf * BN + 32 + lane_off, s[1]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[buf]);
        float sum[2];
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
          float p[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) p[k] = ex2_approx(fmaf(__uint_as_float(s[k2][k]), g.scale_log2, -lse2));
          if ((t + 1) * BN > limit) {
            // keys that this token does not see, and rows past the window (which may hold anything)
#pragma unroll
            for (int k = 0; k < 32; ++k) p[k] = t * BN + 32 * k2 + k < limit ? p[k] : 0.f;
          }
          // Sum over the warp's heads: each step halves the keys a lane holds.
          // Lane l ends with key 32 k2 + l.
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const bool upper = (lane & o) != 0;
#pragma unroll
            for (int k = 0; k < o; ++k) {
              const float keep = upper ? p[k + o] : p[k], send = upper ? p[k] : p[k + o];
              p[k] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
          }
          sum[k2] = real ? p[0] : 0.f;
        }
        named_sync(1 + kSumGroups + group, 128);   // the previous tile's sums have been read
        part_s[group][quarter][lane] = sum[0];
        part_s[group][quarter][32 + lane] = sum[1];
        if (leave()) break;
        if (k_mine < BN && key < len)
          w_row[key] = factor * old + ((part_s[group][0][k_mine] + part_s[group][1][k_mine]) +
                                       (part_s[group][2][k_mine] + part_s[group][3][k_mine]));
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_tc_key_weights(const KeyWeightParams& p, cudaStream_t stream) {
  WeightArgs a;
  a.g = p.g;
  a.lse = p.lse;
  a.weights = p.weights;
  a.weights_batch_stride = p.weights_batch_stride;
  a.decay = p.decay;
  a.n_new = p.n_new;
  const DecodeGeometry& g = p.g;
  const bool q8 = g.codes != nullptr;   // codes are copied row by row: only rope keys are mapped
  a.batch_in_map = ((g.latent_batch_stride != 0 && !q8) || g.rope_batch_stride != 0) ? 1 : 0;
  CUtensorMap q_map, lat_map = {}, rope_map;
  const uint32_t q_box[3] = {64, 64, 1};
  a.rows_in_map = g.q_row_stride != 0;
  const uint64_t q_rows = a.rows_in_map ? (uint64_t)g.batch * g.s_q : 1;
  const uint64_t qd[3] = {(uint64_t)(g.rank + g.rope_dim), (uint64_t)g.heads, q_rows};
  const uint64_t qs[2] = {(uint64_t)g.q_head_stride * 2, (uint64_t)(a.rows_in_map ? g.q_row_stride : g.heads * g.q_head_stride) * 2};
  if (!encode_tmap_bf16(&q_map, g.q, 3, qd, qs, q_box)) return cudaErrorInvalidValue;
  const uint64_t bmap = a.batch_in_map ? (uint64_t)g.batch : 1;
  const uint32_t box[3] = {64, BN, 1};
  if (!q8) {
    const uint64_t ld[3] = {(uint64_t)g.rank, (uint64_t)g.t_max, bmap};
    const uint64_t ls[2] = {(uint64_t)g.latent_row_stride * 2,
                            (a.batch_in_map ? (uint64_t)g.latent_batch_stride : (uint64_t)g.t_max * g.latent_row_stride) * 2};
    if (!encode_tmap_bf16(&lat_map, g.latent, 3, ld, ls, box)) return cudaErrorInvalidValue;
  }
  const uint64_t rd[3] = {(uint64_t)g.rope_dim, (uint64_t)g.t_max, bmap};
  const uint64_t rs[2] = {(uint64_t)g.rope_row_stride * 2,
                          (a.batch_in_map ? (uint64_t)g.rope_batch_stride : (uint64_t)g.t_max * g.rope_row_stride) * 2};
  if (!encode_tmap_bf16(&rope_map, g.rope, 3, rd, rs, box)) return cudaErrorInvalidValue;
  auto* const kernel = q8 ? tc_key_weights_kernel<true> : tc_key_weights_kernel<false>;
  const int smem = q8 ? SMEM_BYTES_Q8 : SMEM_BYTES;
  const cudaError_t ea = set_max_dynamic_smem(kernel, smem);
  if (ea != cudaSuccess) return ea;
  const cudaError_t e = launch_pdl(kernel, dim3((unsigned)device_sm_count()), dim3(q8 ? kThreadsQ8 : kThreads), smem,
                                   stream, q_map, lat_map, rope_map, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mla
