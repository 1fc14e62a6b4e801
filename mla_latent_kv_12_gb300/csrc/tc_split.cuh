// The split plan of the tensor-core decode kernels (tc_decode.cu, tc_paged.cu):
// their arguments, the tiles of each query row, the ranges of tiles that the
// clusters take, and the launches of the planner and of the combine.
#pragma once

#include "mla_internal.h"
#include "paged.cuh"
#include "pieces.cuh"
#include "tc_common.cuh"

namespace mla {
namespace tc {

constexpr int BN = 64;                    // keys per tile
constexpr int HEADS = 128, RANK = 512, DV = 256;  // DV: latent dims per CTA
constexpr long long kWaitLimit = 1LL << 32;  // clock cycles (~2 s)
constexpr float kRescaleThreshold = 8.0f;    // log2 units
// A group's tile range is at least this long: each split writes a 128 KB fp16
// partial, worth it only against a few 72 KB tiles of cache read.
constexpr int kMinTilesPerGroup = 4;
// Each work unit with tiles is charged this many tiles' worth of time for
// its start: a segment boundary drains the pair's pipeline (the next query
// enters TMEM only once the previous segment's last scores are read, then
// its first scores and exchange run before the softmax resumes), which costs
// several tiles of streaming.  The charge sits in the split plan ahead of the
// unit's tiles, so a group whose range holds more unit starts gets fewer
// tiles.  It applies when the groups stream at least kChargeMinSpan tiles
// each: with a few tiles per group (a short or selected-position batch) every
// group pays one start anyway, and a charge would only idle groups.
constexpr int kUnitStartCharge = 10;
constexpr int kChargeMinSpan = 32;
constexpr int kQueryPrefetchTiles = 4;   // the next segment's query is pulled into L2 this many tiles before
// Up to this many query rows, every CTA plans the split itself in its prologue
// (no planner launch); larger batches use the planner kernel.
constexpr int kMaxRowsInKernelPlan = 128;

struct TcDecodeArgs {
  const __nv_bfloat16* q;
  int64_t q_row_stride, q_head_stride;
  const __nv_bfloat16* latent;
  int64_t latent_row_stride, latent_batch_stride;
  const __nv_bfloat16* rope;
  int64_t rope_row_stride, rope_batch_stride;
  const int32_t* kv_start;
  const int32_t* kv_len;
  int32_t s_q, n_q;    // query rows: of a batch row, in all
  int32_t heads;       // 64 or 128; rows h >= heads of the MMA's M side are zero padding (or another token's)
  // Tokens of a query row (2: two tokens of 64 heads share the MMA's 128 rows), of a batch row and in all.
  int32_t tokens, tok_q, n_tokens;
  const int32_t* sel;
  const int32_t* sel_count;
  int32_t k_max;
  float scale_log2;
  void* ctx;
  int64_t ctx_row_stride, ctx_head_stride;
  int32_t out_f32;
  float* lse;
  int32_t* status;
  int32_t* prefix;     // [n_units + 2] the split plan: prefix over work units, then the start charge
  int32_t* keys;       // [n_q] visible entries per query row (planner)
  uint4* ws_o;         // [slots][RANK/8][H] partial context, 8 fp16 dims per entry (O / l of the piece); slots: see slot_of
  float* ws_ml;        // [slots][2][H] partial (m, l), log2 domain
  int32_t num_clusters;
  int32_t width;       // query rows per work unit = clusters per group
  int32_t n_units;     // n_q / width (over pages rounded up)
  int32_t min_tiles;   // smallest tile range given to a group
  int32_t start_charge, charge_min_span;  // kUnitStartCharge and kChargeMinSpan, or the kernel's own
  int32_t batch_in_map;  // 1: use batch coordinate b in the tensor maps
  int32_t gather_tma;    // 1: selected rows come by TMA gather4 (else cp.async)
  int32_t lat_rows_per_batch, rope_rows_per_batch;  // batch stride in rows (gather maps)
  int32_t plan_in_kernel;  // 1: n_q <= kMaxRowsInKernelPlan, each CTA plans (CTA 0 also stores the plan)
  // 1 inside a fused step: the launch before the decode kernel is the absorb
  // kernel, which writes only the query and lets its dependants start only
  // after its own wait, so every other input is complete when this grid starts.
  int32_t early_inputs;
  // 8-bit cache (null codes: `latent`); strides in bytes
  const uint8_t* codes;
  int64_t codes_row_stride, codes_batch_stride;
  const uint8_t* scales;
  int64_t scales_batch_stride;
  int32_t block_shift;
  int64_t t_max;
  // Paged cache (null table: windows): a row's keys by pages of page_size rows, read in boxes of
  // box_rows rows, or row by row (lat_rows_per_batch, rope_rows_per_batch: between pages).
  const int32_t* table;
  int64_t table_stride;
  int32_t page_size, num_pages, box_rows;
  const int32_t* counts;
  const uint64_t* tree;
  int32_t tree_words;
  bool few_units;      // no more work units than groups of clusters (set with the workspace)
};

// ------------------------------------------------------------------ helpers

// Paged caches: the ancestor mask of a token (null without a tree), the first of
// a batch row's new keys, and the keys [0, limit) that hold what its token i sees.
__device__ __forceinline__ const uint64_t* tree_of(const TcDecodeArgs& a, int token) {
  return a.tree ? a.tree + (int64_t)token * a.tree_words : nullptr;
}
__device__ __forceinline__ int paged_first(const TcDecodeArgs& a, int b) {
  return a.kv_len[b] - paged_count(a.counts, b, a.tok_q);
}
__device__ __forceinline__ int token_limit(const TcDecodeArgs& a, int b, int i) {
  const int len = a.kv_len[b], count = paged_count(a.counts, b, a.tok_q);
  if (len < 0 || len > a.t_max || count < 0) return 0;
  return paged_limit(len, count, i, i < a.tok_q ? tree_of(a, b * a.tok_q + i) : nullptr, a.tree_words);
}

// (What only paged rows need stays out of the other instances of kernels that plan.)
template <bool kPaged>
__device__ __forceinline__ int row_limit(const TcDecodeArgs& a, int n) {
  const int b = n / a.s_q, i = n % a.s_q;
  if constexpr (kPaged) {
    const int limit = token_limit(a, b, i * a.tokens);
    return a.tokens == 2 ? max(limit, token_limit(a, b, 2 * i + 1)) : limit;
  }
  const int len = a.kv_len[b];
  int lim = len - a.s_q + i + 1;
  lim = lim < 0 ? 0 : (lim > len ? len : lim);
  return lim;
}

// Work units are query rows, or -- for a dense multi-token verify -- whole
// batch rows whose `width` = s_q tokens are served by a group of `width`
// clusters in lockstep (member i takes token i), so the tokens of a batch row
// read each cache tile at the same time and three of four reads hit L2.
// The units' tiles form one flattened sequence cut into equal ranges, one per
// group (at least `min_tiles` each, so a short sequence uses fewer groups).
// In that sequence each unit with tiles occupies charge + tiles positions,
// its tiles at the end: prefix[0..n_units] holds these extents' exclusive
// prefix and prefix[n_units + 1] the charge, so unit u's tile j sits at
// position prefix[u] + charge + j.
__device__ __forceinline__ int group_span(const TcDecodeArgs& a, int total) {
  const int ngroups = a.num_clusters / a.width;
  const int per = (total + ngroups - 1) / ngroups;
  return per > a.min_tiles ? per : a.min_tiles;
}

// The start charge of a plan whose units hold `raw` tiles in all.
__device__ __forceinline__ int unit_start_charge(const TcDecodeArgs& a, int raw) {
  const int ngroups = a.num_clusters / a.width;
  return (raw + ngroups - 1) / ngroups >= a.charge_min_span ? a.start_charge : 0;
}

struct WorkIter {
  const int32_t* prefix;
  int n, t, t_begin, t_end, charge;
  __device__ void init(const TcDecodeArgs& a, const int32_t* unit_prefix, int group) {
    prefix = unit_prefix;
    charge = prefix[a.n_units + 1];
    const int total = prefix[a.n_units];
    const int per = group_span(a, total);
    const int ngroups = a.num_clusters / a.width;
    const long long b0 = group < ngroups ? (long long)group * per : total;
    t_begin = (int)min((long long)total, b0);
    t_end = (int)min((long long)total, (long long)t_begin + per);
    // first unit with prefix[n+1] > t_begin
    int lo = 0, hi = a.n_units - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid + 1] > t_begin) hi = mid; else lo = mid + 1;
    }
    n = lo;
    t = t_begin;
  }
  // Next segment: unit u, unit-local tiles [t0, t1); `whole` if all of the
  // unit's tiles lie inside this group's range.  A unit whose start charge
  // alone falls in the range is no segment.
  __device__ bool next(int& u, int& t0, int& t1, bool& whole) {
    while (t < t_end) {
      while (prefix[n + 1] <= t) ++n;
      const int rs = prefix[n] + charge, re = prefix[n + 1];   // the unit's tiles
      const int s = max(t, rs), e = min(t_end, re);
      t = e;
      if (s >= e) continue;
      u = n;
      t0 = s - rs;
      t1 = e - rs;
      whole = rs >= t_begin && re <= t_end;
      return true;
    }
    return false;
  }
};

// The groups whose ranges hold unit u's tiles: [first, last] (a unit with
// tiles; `charge` = prefix[n_units + 1]).
__device__ __forceinline__ int first_group_of(const int32_t* prefix, int u, int per, int charge) {
  return (prefix[u] + charge) / per;
}
__device__ __forceinline__ int last_group_of(const int32_t* prefix, int u, int per) {
  return (prefix[u + 1] - 1) / per;
}

// Where in the workspace the piece of unit u's row `member` lies that group g
// leaves (`begins`: g holds the unit's first tile).
template <bool kPaged>
__device__ __forceinline__ int64_t slot_of(const TcDecodeArgs& a, int u, int g, int member, bool begins) {
  const int place = kPaged ? piece_place(a.few_units, u, g, begins) : u + g;
  return (int64_t)place * a.width + member;
}

// A member's share of a unit segment: its query row n and the segment's tiles
// clipped to that row's own tiles (a verify token sees a shorter prefix than
// the last token).  False if nothing is left.
template <bool kPaged>
__device__ __forceinline__ bool member_segment(const TcDecodeArgs& a, const int32_t* keys, int u, int member,
                                               int& n, int& t0, int& t1) {
  n = u * a.width + member;
  if (kPaged && n >= a.n_q) return false;   // the last unit may have fewer rows
  const int tiles = (keys[n] + BN - 1) / BN;
  if (t1 > tiles) t1 = tiles;
  return t0 < t1;
}

// ------------------------------------------------------------------ planner
// Per query row the number of visible entries; the planner (or the decode
// prologue) turns them into tiles and the exclusive prefix of tiles over work
// units.  Bad selection counts give 0 and are flagged where `flag` is set.
template <bool kPaged>
__device__ __forceinline__ int row_keys(const TcDecodeArgs& a, int n, bool flag) {
  int keys = row_limit<kPaged>(a, n);
  if constexpr (kPaged) {
    const int b = n / a.s_q, len = a.kv_len[b];
    if (flag && a.status && (len < 0 || len > a.t_max || paged_count(a.counts, b, a.tok_q) < 0))
      atomicOr(a.status, MLA_DEVICE_INDEX_OUT_OF_RANGE);
    if (keys == 0) return 0;   // the selection of a token that sees nothing is not read
  }
  if (a.codes) {
    // the 8-bit cache is read by plain loads: a window outside the buffer, or
    // one that does not start on a whole block, is no window
    const int b = n / a.s_q, start = a.kv_start ? a.kv_start[b] : 0, len = a.kv_len[b];
    const bool fits = len >= 0 && start >= 0 && (int64_t)start + len <= a.t_max;
    if (!fits || (start & ((1 << a.block_shift) - 1)) != 0) {
      if (flag && a.status) atomicOr(a.status, fits ? MLA_DEVICE_BAD_BLOCK_START : MLA_DEVICE_INDEX_OUT_OF_RANGE);
      return 0;
    }
  }
  if (a.sel) {
    const int c = a.sel_count[n];
    if (c != -1) {
      if (c <= 0 || c > a.k_max) {
        keys = 0;
        if (flag && a.status) atomicOr(a.status, MLA_DEVICE_BAD_SELECTION_COUNT);
      } else {
        keys = c;
      }
    }
  }
  return keys;
}

// The split plan inside a kernel (n_q <= kMaxRowsInKernelPlan; called by every
// thread of the block, blockDim >= n_q): visible entries per query row, then per
// unit its tiles (the longest of its `width` rows) and their exclusive prefix,
// scanned by warp 0 (four units per lane, in unit order).
// With start_s / limit_s, also each row's first cache row (of a paged row: the
// first of its new tokens' keys) and the window limit of each of its tokens.
template <bool kPaged>
__device__ __forceinline__ void plan_rows(const TcDecodeArgs& a, int32_t* keys_s, int32_t* prefix_s, bool flag,
                                          int32_t* start_s = nullptr, int32_t* limit_s = nullptr) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x < a.n_q) {
    const int n = threadIdx.x;
    keys_s[n] = row_keys<kPaged>(a, n, flag);
    if (start_s) {
      const int b = n / a.s_q;
      start_s[n] = kPaged ? paged_first(a, b) : a.kv_start ? a.kv_start[b] : 0;
      if (kPaged && a.tokens == 2) {
        limit_s[2 * n] = token_limit(a, b, 2 * (n % a.s_q));
        limit_s[2 * n + 1] = token_limit(a, b, 2 * (n % a.s_q) + 1);
      } else {
        limit_s[n] = row_limit<kPaged>(a, n);
      }
    }
  }
  __syncthreads();
  if (warp == 0) {
    int tl[kMaxRowsInKernelPlan / 32];
    int raw = 0;
#pragma unroll
    for (int j = 0; j < kMaxRowsInKernelPlan / 32; ++j) {
      const int u = 32 * j + lane;
      int tiles = 0;
      if (u < a.n_units)
        for (int i = 0; i < a.width && (!kPaged || u * a.width + i < a.n_q); ++i)
          tiles = max(tiles, (keys_s[u * a.width + i] + BN - 1) / BN);
      tl[j] = tiles;
      raw += tiles;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) raw += __shfl_xor_sync(0xffffffffu, raw, o);
    const int charge = unit_start_charge(a, raw);
    int carry = 0;
#pragma unroll
    for (int j = 0; j < kMaxRowsInKernelPlan / 32; ++j) {
      const int u = 32 * j + lane;
      const int ext = tl[j] > 0 ? tl[j] + charge : 0;   // the unit's extent in the plan
      int v = ext;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
      }
      if (u < a.n_units) prefix_s[u] = carry + v - ext;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) {
      prefix_s[a.n_units] = carry;
      prefix_s[a.n_units + 1] = charge;
    }
  }
  __syncthreads();
}

// The groups that hold a row's pieces, for the combine of a paged call that plans in its kernel (one warp of one CTA; in
// `keys`, which only the planner launch uses otherwise): first | last << 16, or -1 for a row without keys.  With the
// plan made again in the combine, as over windows, a tree of 16 nodes behind 4050 keys took 32.1 us
// instead of 30.6, four of 20 nodes behind 20000 keys 313 instead of 300.
__device__ __forceinline__ void store_pieces(const TcDecodeArgs& a, const int32_t* keys, const int32_t* prefix) {
  const int per = group_span(a, prefix[a.n_units]);
#pragma unroll 1
  for (int n = threadIdx.x & 31; n < a.n_q; n += 32) {
    const int u = n / a.width;
    a.keys[n] = keys[n] > 0 ? first_group_of(prefix, u, per, prefix[a.n_units + 1]) | last_group_of(prefix, u, per) << 16 : -1;
  }
}

// The planner launch (more than kMaxRowsInKernelPlan rows), and the merge of
// the split rows behind a decode kernel.
cudaError_t launch_split_plan(const TcDecodeArgs& a, cudaStream_t stream);
cudaError_t launch_split_combine(const TcDecodeArgs& a, cudaStream_t stream);
// Points prefix, keys, ws_o and ws_ml (once n_units, num_clusters and width are set) into a workspace of tc_decode_workspace(n_q) or tc_paged_workspace(n_q) bytes.
void lay_out_workspace(TcDecodeArgs& a, void* workspace);

}  // namespace tc
}  // namespace mla
