// Eviction by accumulated attention weight: which tokens of a row stay, and
// their compaction to the front of the row's window, in place.
//
// Plan.  A cluster of 1..8 CTAs per row.  Between the sinks and the recent
// tokens the n_keep - n_sink - n_recent heaviest stay: their rank key is the
// order-preserving map of the f32 bits to uint32, complemented (ascending key
// = descending weight), and a radix selection (digits of 11, 11 and 10 bits)
// finds the largest kept key and how many of its equals are kept; it ends
// early when all keys with the digits so far are kept.  Each CTA
// holds its slice's keys in shared memory where they fit, so the weights
// are read once; the digit histograms are summed over the cluster through
// distributed shared memory, every CTA taking the same digit.  Bound by the
// latency of the passes, not by the 4 bytes per token: 12 us for one row of
// 8192, 17 us for 32 rows of up to 32768, 25 us for one of 131072.
//
// Compaction.  Kept positions ascend, so row j's source kept[j] >= j: rows are
// moved in chunks of consecutive j, and a chunk is written only when all
// chunks up to it have been read.  Later chunks read rows behind all of its
// own, so their loads are issued ahead (kDepth chunks, in registers) and the memory
// stays busy across the barriers.  Rows of a window are one dependent chain;
// the parallelism is over batch rows and 64-byte slices of a token's bytes, and
// over the CTAs of a cluster (which share each chunk, with a cluster barrier)
// when those are few.  8 rows of 32768 bf16 tokens halved: 59 us, 5.2 TB/s of
// the bytes moved.
#include "mla_internal.h"
#include "tc_common.cuh"
#include "tc_host.h"

namespace mla {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMaxHeldKeys = 40 * 1024;   // 160 KB of shared memory

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int2 load_peer2(const int* local, uint32_t rank) {   // 8-byte aligned
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(tc::mapa(tc::smem_u32(local), rank)) : "memory");
  return v;
}

// Heavier tokens have smaller keys.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t bits = __float_as_uint(w);
  return ~(bits ^ ((bits >> 31) ? 0xFFFFFFFFu : 0x80000000u));
}

__device__ __forceinline__ int warp_inclusive(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

__global__ void __launch_bounds__(kPlanThreads, 1) evict_plan_kernel(const __grid_constant__ EvictParams p, int held) {
  extern __shared__ uint32_t keys_s[];   // `held` keys of this CTA's slice
  __shared__ __align__(8) int hist_s[3][kBins];   // one per pass: a peer may still read the previous one
  // per pass (written once, so that no barrier keeps a reader from a later writer)
  __shared__ int total_s[3][kPlanWarps], peers_s[3][kPlanWarps];   // of each warp's bins: the cluster's, and the earlier CTAs'
  struct Found {
    int digit, rest, less, tie, last;
  };
  __shared__ Found found_s[3];
  __shared__ int less_s[kPlanWarps], tie_s[kPlanWarps];
  static_assert(kPlanWarps == 32, "one warp's sum per lane");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // (the compaction's CTAs may take their places already: they wait for this grid's end)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t crank = tc::cluster_ctarank();
  const int ncta = (int)cluster_size();
  const int b = blockIdx.x / ncta;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int len = p.kv_len[b], start = p.kv_start ? p.kv_start[b] : 0;
  const bool fits = len >= 0 && start >= 0 && (int64_t)start + len <= p.t_max;
  if (!fits || len <= p.n_keep) {   // the same in every CTA of the cluster
    if (crank == 0 && threadIdx.x == 0) {
      p.counts[b] = -1;
      if (p.kv_len_out) p.kv_len_out[b] = len;
      if (!fits && p.status) atomicOr(p.status, MLA_DEVICE_INDEX_OUT_OF_RANGE);
    }
    return;
  }
  const float* w = p.weights + b * p.weights_batch_stride + start;
  int32_t* kept = p.kept + b * p.kept_stride;
  // candidates: window positions [n_sink, len - n_recent); this CTA's slice [lo, hi)
  const int take = p.n_keep - p.n_sink - p.n_recent;
  const int first = p.n_sink, last = len - p.n_recent;
  const int span = ((last - first + ncta - 1) / ncta + 31) & ~31;
  const int lo = min(last, first + (int)crank * span), hi = min(last, lo + span);
  const bool in_smem = hi - lo <= held;
  auto key_at = [&](int i) { return in_smem ? keys_s[i - lo] : weight_key(w[i]); };

  uint32_t prefix = 0;
  int rest = take;   // the rest-th smallest key among those with the prefix is looked for
  int drop = 0;      // low key bits that need not be compared
  int peers_less = 0, peers_tie = 0;   // keys below `prefix`, and equal to it, in the earlier CTAs' slices
  if (take > 0) {
    for (int i = threadIdx.x; i < 3 * kBins; i += kPlanThreads) hist_s[0][i] = 0;
    __syncthreads();
    int known = 0;   // leading key bits fixed so far
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int width = pass < 2 ? 11 : 10, shift = 32 - known - width;
      int* hist = hist_s[pass];
      constexpr int kLoads = 8;   // independent loads in flight per thread
      for (int base = lo; base < hi; base += kPlanThreads * kLoads) {
        uint32_t key[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          const int i = base + u * kPlanThreads + threadIdx.x;
          key[u] = 0;
          if (i < hi) key[u] = pass == 0 ? weight_key(w[i]) : key_at(i);
        }
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          if (base + u * kPlanThreads >= hi) break;   // (the same in the whole block)
          const int i = base + u * kPlanThreads + threadIdx.x;
          if (pass == 0 && in_smem && i < hi) keys_s[i - lo] = key[u];
          const bool counts = i < hi && (pass == 0 || (key[u] >> (32 - known)) == prefix);
          const int digit = (int)((key[u] >> shift) & ((1u << width) - 1u));
          // Lanes with the digit of the first one that counts add once (many
          // weights share a value, zero above all, and equal addresses are
          // added one by one); the rest add for themselves.
          const uint32_t who = __ballot_sync(0xffffffffu, counts);
          if (who == 0) continue;   // (the same in the whole warp)
          const int leader = __ffs(who) - 1;
          const int common = __shfl_sync(0xffffffffu, digit, leader);   // (by every lane: not behind a condition)
          const uint32_t same = __ballot_sync(0xffffffffu, counts && digit == common);
          if (lane == leader) atomicAdd(&hist[digit], __popc(same));
          if (counts && !((same >> lane) & 1u)) atomicAdd(&hist[digit], 1);
        }
      }
      tc::cluster_sync();   // every CTA's histogram is complete
      // thread t sums bins 2t and 2t + 1 over the cluster
      const int nb = 1 << width, b0 = 2 * threadIdx.x;
      int h[2] = {0, 0}, e[2] = {0, 0};   // the cluster's, and the earlier CTAs'
      if (b0 < nb) {
        int2 part[kMaxCluster];   // all loads in flight together
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c)
          part[c] = c < ncta ? load_peer2(&hist[b0], (uint32_t)c) : make_int2(0, 0);
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
          h[0] += part[c].x, h[1] += part[c].y;
          if (c < (int)crank) e[0] += part[c].x, e[1] += part[c].y;
        }
      }
      const int hs = h[0] + h[1], es = e[0] + e[1];
      const int ht = __reduce_add_sync(0xffffffffu, hs), et = __reduce_add_sync(0xffffffffu, es);
      if (lane == 0) total_s[pass][warp] = ht, peers_s[pass][warp] = et;
      __syncthreads();
      const int total = total_s[pass][lane], upto = warp_inclusive(total, lane);
      const int holder = __ffs(__ballot_sync(0xffffffffu, upto >= rest)) - 1;   // the warp whose bins hold the rest-th key
      if (warp == holder) {
        int before = __shfl_sync(0xffffffffu, upto - total, holder) + warp_inclusive(hs, lane) - hs;
        int less = __reduce_add_sync(0xffffffffu, lane < holder ? peers_s[pass][lane] : 0) + warp_inclusive(es, lane) - es;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // (exactly one thread and bin; the last pass when all keys with this digit are kept)
          if (before < rest && rest <= before + h[k])
            found_s[pass] = Found{b0 + k, rest - before, less, e[k], rest - before == h[k]};
          before += h[k];
          less += e[k];
        }
      }
      __syncthreads();
      const Found found = found_s[pass];
      prefix = (prefix << width) | (uint32_t)found.digit;
      rest = found.rest;
      peers_less += found.less;
      peers_tie = found.tie;
      known += width;
      drop = 32 - known;
      if (found.last) break;   // (the same in the whole cluster)
    }
  }
  // The last reads of other CTAs' shared memory are done: no CTA leaves before all have arrived here.
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  // ---- kept: keys below `prefix`, and the first `rest` positions that equal it.
  // Warp w owns a contiguous part of the slice, so that ranks follow positions.
  const int wspan = ((hi - lo + kPlanWarps - 1) / kPlanWarps + 31) & ~31;
  const int wlo = min(hi, lo + warp * wspan), whi = min(hi, wlo + wspan);
  int n_less = 0, n_tie = 0;
  if (take > 0)
#pragma unroll 4
    for (int i0 = wlo; i0 < whi; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t key = i < whi ? key_at(i) >> drop : 0xFFFFFFFFu;
      n_less += __popc(__ballot_sync(0xffffffffu, i < whi && key < prefix));
      n_tie += __popc(__ballot_sync(0xffffffffu, i < whi && key == prefix));
    }
  if (lane == 0) less_s[warp] = n_less, tie_s[warp] = n_tie;
  __syncthreads();
  const int before_less = __reduce_add_sync(0xffffffffu, lane < warp ? less_s[lane] : 0) + peers_less;
  const int before_tie = __reduce_add_sync(0xffffffffu, lane < warp ? tie_s[lane] : 0) + peers_tie;
  if (take > 0) {
    int out = p.n_sink + before_less + min(before_tie, rest), ties = before_tie;
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll 4
    for (int i0 = wlo; i0 < whi; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t key = i < whi ? key_at(i) >> drop : 0xFFFFFFFFu;
      const uint32_t tie = __ballot_sync(0xffffffffu, i < whi && key == prefix);
      const bool stays = i < whi && (key < prefix || (key == prefix && ties + __popc(tie & below) < rest));
      const uint32_t who = __ballot_sync(0xffffffffu, stays);
      if (stays) kept[out + __popc(who & below)] = i;
      out += __popc(who);
      ties += __popc(tie);
    }
  }
  const int me = (int)crank * kPlanThreads + threadIdx.x;
  for (int j = me; j < p.n_sink; j += ncta * kPlanThreads) kept[j] = j;
  for (int j = me; j < p.n_recent; j += ncta * kPlanThreads) kept[p.n_keep - p.n_recent + j] = last + j;
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (crank == 0 && threadIdx.x == 0) {   // every CTA has read kv_len, which kv_len_out may alias
    p.counts[b] = p.n_keep;
    if (p.kv_len_out) p.kv_len_out[b] = p.n_keep;
  }
}

// ------------------------------------------------------------------ compaction

constexpr int kMoveThreads = 512;
// Units per thread and chunk, chunks in flight, slice width and threads: of the
// sweep (moves, depth, bytes, threads) on a bf16 batch of 8 rows halved from
// 32768 tokens (plan and compaction): (2, 3, 64, 512) 79 us, (4, 2, 64, 512) 85,
// (2, 4, 64, 512) 87, (8, 1, 64, 512) 89, (1, 8, 64, 512) 95, (4, 3, 64, 512)
// 104, (4, 2, 128, 512) 118, (2, 3, 64, 256) 83, three CTAs per SM 110: fewer
// barriers against more in flight, within 64 registers a thread.
constexpr int kMoves = 2;
constexpr int kDepth = 3;
constexpr int kSliceBytes = 64;    // of a token's bytes moved by one CTA

struct Slice {
  uint8_t* data;       // the slice's first byte of buffer row kv_start[b]
  int64_t stride;      // bytes between buffer rows
  int units;           // per row
};

// A word that depends on every byte of v (its value does not matter).
__device__ __forceinline__ uint32_t word_of(uint4 v) { return v.x ^ v.y ^ v.z ^ v.w; }
__device__ __forceinline__ uint32_t word_of(uint2 v) { return v.x ^ v.y; }
__device__ __forceinline__ uint32_t word_of(uint32_t v) { return v; }

template <typename V>
__device__ __forceinline__ void move_rows(const Slice s, const CompactParams& p, const int32_t* kept, int count,
                                          int start, int crank, int ncta, bool flags, uint32_t* arrived) {
  // Thread i of the cluster moves unit i % units of rows i / units + k * rows_per_step
  const int rows_cta = kMoveThreads / s.units;              // rows per step of this CTA
  const int row0 = threadIdx.x / s.units, part = threadIdx.x % s.units;
  const bool active = row0 < rows_cta;
  const int step = rows_cta * ncta, chunk = step * kMoves;
  const int n_chunks = (count + chunk - 1) / chunk;
  auto row_of = [&](int c, int u) { return c * chunk + u * step + crank * rows_cta + row0; };
  // The position of row j if it is one to move: above its predecessor's (so >= j), inside the buffer.
  int pos[kMoves];
  auto load_positions = [&](int c) {
    int cur[kMoves], prev[kMoves];
#pragma unroll
    for (int u = 0; u < kMoves; ++u) {
      const int j = row_of(c, u);
      const bool in = active && c < n_chunks && j < count;
      cur[u] = in ? __ldg(kept + j) : -1;
      prev[u] = in && j > 0 ? __ldg(kept + j - 1) : -1;
    }
#pragma unroll
    for (int u = 0; u < kMoves; ++u) {
      const int j = row_of(c, u);
      const bool in = active && c < n_chunks && j < count;
      const bool good = in && cur[u] >= j && cur[u] > prev[u] && (int64_t)start + cur[u] < p.t_max;
      if (in && !good && flags && p.status) atomicOr(p.status, MLA_DEVICE_INDEX_OUT_OF_RANGE);
      pos[u] = good && cur[u] != j ? cur[u] : -1;   // a row already in place stays
    }
  };
  V v[kDepth][kMoves];
  bool moved[kDepth][kMoves];
  auto load_rows = [&](V(&dst)[kMoves], bool(&m)[kMoves]) {
#pragma unroll
    for (int u = 0; u < kMoves; ++u) {
      m[u] = pos[u] >= 0;
      dst[u] = V{};
      if (m[u]) dst[u] = *(reinterpret_cast<const V*>(s.data + (int64_t)pos[u] * s.stride) + part);
    }
  };
  load_positions(0);
#pragma unroll
  for (int d = 0; d < kDepth; ++d) {
    load_rows(v[d], moved[d]);
    load_positions(d + 1);
  }
  for (int c0 = 0; c0 < n_chunks; c0 += kDepth) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int c = c0 + d;
      if (c >= n_chunks) break;   // the same in the whole cluster
      // Every thread of the cluster holds its rows of chunk c: the store of a
      // word made of them waits for them before the barrier.
      uint32_t word = 0;
#pragma unroll
      for (int u = 0; u < kMoves; ++u) word ^= word_of(v[d][u]);
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(tc::smem_u32(arrived)), "r"(word) : "memory");
      if (ncta > 1) {
        // No memory is handed over: the loads have their values, and nothing
        // written is read again.  (A releasing arrival waits for the stores of
        // the chunk before: 59 against 51 us for one row of 131072.)
        asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
      } else {
        __syncthreads();
      }
#pragma unroll
      for (int u = 0; u < kMoves; ++u)
        if (moved[d][u]) *(reinterpret_cast<V*>(s.data + (int64_t)row_of(c, u) * s.stride) + part) = v[d][u];
      load_rows(v[d], moved[d]);   // chunk c + kDepth
      load_positions(c + kDepth + 1);
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads, 2) compact_kernel(const __grid_constant__ CompactParams p) {
  __shared__ uint32_t arrived_s[kMoveThreads];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int ncta = (int)cluster_size();
  const int crank = (int)tc::cluster_ctarank();
  const int b = blockIdx.y;
  int slice = blockIdx.x / ncta;
  const bool flags = slice == 0;
  const int count = p.counts[b], start = p.kv_start ? p.kv_start[b] : 0;
  const bool good = count >= -1 && count <= p.n_keep;
  const bool fits = start >= 0 && (int64_t)start + count <= p.t_max;
  if (!good || !fits || count <= 0) {   // the same in the whole cluster
    if (flags && crank == 0 && threadIdx.x == 0 && p.status) {
      if (!good) atomicOr(p.status, MLA_DEVICE_BAD_SELECTION_COUNT);
      else if (!fits) atomicOr(p.status, MLA_DEVICE_INDEX_OUT_OF_RANGE);
    }
  } else {
    // this CTA's array and slice
    int k = 0;
    auto slices_of = [&](int i) { return (p.a[i].row_bytes + kSliceBytes - 1) / kSliceBytes; };
    while (slice >= slices_of(k)) slice -= slices_of(k++);
    const CompactArray& a = p.a[k];
    const int bytes = min(kSliceBytes, a.row_bytes - slice * kSliceBytes);
    const Slice s{a.data + b * a.batch_bytes_stride + (int64_t)start * a.row_bytes_stride + slice * kSliceBytes,
                  a.row_bytes_stride, bytes / a.unit};
    const int32_t* kept = p.kept + b * p.kept_stride;
    switch (a.unit) {
      case 16: move_rows<uint4>(s, p, kept, count, start, crank, ncta, flags, arrived_s + threadIdx.x); break;
      case 8: move_rows<uint2>(s, p, kept, count, start, crank, ncta, flags, arrived_s + threadIdx.x); break;
      case 4: move_rows<uint32_t>(s, p, kept, count, start, crank, ncta, flags, arrived_s + threadIdx.x); break;
      case 2: move_rows<uint16_t>(s, p, kept, count, start, crank, ncta, flags, arrived_s + threadIdx.x); break;
      default: move_rows<uint8_t>(s, p, kept, count, start, crank, ncta, flags, arrived_s + threadIdx.x); break;
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, int threads, int smem, int ncta, cudaStream_t stream,
                           Args... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ncta;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_evict_plan(const EvictParams& p, cudaStream_t stream) {
  // CTAs per row: one per 2048 candidates of the longest possible row, at most
  // 8, and few enough that all rows run at once.
  const int64_t most = p.t_max < 2048 ? 1 : p.t_max / 2048;
  int ncta = 1;
  while (ncta * 2 <= kMaxCluster && ncta * 2 <= most && (int64_t)ncta * 2 * p.batch <= device_sm_count()) ncta *= 2;
  // a row's slice is at most ceil(t_max / ncta), rounded up to 32
  const int64_t slice = (((p.t_max + ncta - 1) / ncta) + 31) & ~31LL;
  const int held = (int)(slice < kMaxHeldKeys ? slice : 0);
  if (held * 4 > 0) {
    const cudaError_t ea = set_max_dynamic_smem(evict_plan_kernel, kMaxHeldKeys * 4);
    if (ea != cudaSuccess) return ea;
  }
  return launch_cluster(evict_plan_kernel, dim3((unsigned)(p.batch * ncta)), kPlanThreads, held * 4, ncta, stream, p,
                        held);
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream) {
  int64_t slices = 0;
  for (int i = 0; i < p.n_arrays; ++i) slices += (p.a[i].row_bytes + kSliceBytes - 1) / kSliceBytes;
  // CTAs per slice: enough to fill the GPU twice, while each still has a chunk of rows
  const int64_t chunk = kMoveThreads * kMoves / (kSliceBytes / 16);
  const int64_t chunks = (p.n_keep + chunk - 1) / chunk;
  int ncta = 1;
  while (ncta * 2 <= kMaxCluster && ncta * 2 <= chunks && slices * p.batch * ncta * 2 <= 2 * device_sm_count()) ncta *= 2;
  if (slices * ncta > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_cluster(compact_kernel, dim3((unsigned)(slices * ncta), (unsigned)p.batch), kMoveThreads, 0, ncta,
                        stream, p);
}

}  // namespace mla
