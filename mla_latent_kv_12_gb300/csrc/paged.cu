// Writing a paged latent cache: append of new tokens (RMSNorm, RoPE), the plan
// of a tree of drafted tokens, and the commit of its accepted path.
#include <cuda_bf16.h>

#include "mla_internal.h"
#include "paged.cuh"
#include "rope_math.cuh"
#include "tc_host.h"

namespace mla {
namespace {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void flag(int32_t* status, int bit) {
  if (status) atomicOr(status, bit);
}

// ------------------------------------------------------------------ append

constexpr int kAppendWarps = 8;

// Eight consecutive values, 16-byte aligned.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) v[2 * j] = __uint_as_float(w[j] << 16), v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// grid (ceil(s_new / warps), batch rows): one warp per new token, which holds
// its values in registers between the sum of squares and the store.  Bound by
// memory for prompt chunks (2 (rank + rope) elements per token), by the chain
// of dependent loads (length, page, store) for single tokens: what does not
// depend on them is loaded first.  Measured: one token 2.6 us, 8 rows of 0 to
// 2048 tokens 6.9 us (2.7 TB/s of 18.9 MB; the copy's rate would take 2.8).  kGroups: groups of eight values per lane
// (rank a multiple of 8 up to 256 kGroups, aligned rows), or 0: one by one.
template <typename TI, typename TC, int kGroups>
__global__ void __launch_bounds__(kAppendWarps * 32) append_paged_kernel(const __grid_constant__ AppendPagedParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = p.rope_dim >> 1;
  const int t = blockIdx.x * (blockDim.x >> 5) + warp;
  const int64_t capacity = (int64_t)p.table_width * p.page_size;
  const TI* w = static_cast<const TI*>(p.weight);
  for (int b = blockIdx.y; b < p.batch; b += gridDim.y) {
    const int len = p.kv_len[b], count = paged_count(p.counts, b, p.s_new);
    const TI* x = static_cast<const TI*>(p.latent_raw) + b * p.lr_row_stride + t * p.lr_tok_stride;
    const TI* rr = static_cast<const TI*>(p.rope_raw) + b * p.rr_row_stride + t * p.rr_tok_stride;
    float v[kGroups ? kGroups : 1][8], re0 = 0.f, im0 = 0.f;
    auto load = [&] {
      if constexpr (kGroups > 0) {
#pragma unroll
        for (int c = 0; c < kGroups; ++c)
          if (256 * c + 8 * lane < p.rank) load8(x + 256 * c + 8 * lane, v[c]);
      }
      if (lane < half) re0 = to_f(rr[2 * lane]), im0 = to_f(rr[2 * lane + 1]);
    };
    const bool early = !p.counts && t < p.s_new;   // before the length is known: every token is there
    if (early) load();
    const bool fits = len >= 0 && count >= 0 && (int64_t)len + count <= capacity;
    if (blockIdx.x == 0) {
      if (p.lengths_here == 2) __syncthreads();   // (one CTA per row: its warps have read the length that is overwritten)
      if (threadIdx.x == 0) {
        if (!fits) flag(p.status, MLA_DEVICE_INDEX_OUT_OF_RANGE);
        if (p.lengths_here) p.kv_len_out[b] = fits ? len + count : len;
      }
    }
    if (!fits || t >= count) continue;
    const int row = len + t, at = row / p.page_size;
    const int page = p.table[b * p.table_stride + at];
    const int64_t pos = p.positions ? (int64_t)p.positions[(int64_t)b * p.s_new + t] : (int64_t)row;
    if (!early) load();
    float inv;
    {
      float sq = 0.f;
      if constexpr (kGroups > 0) {
#pragma unroll
        for (int c = 0; c < kGroups; ++c)
          if (256 * c + 8 * lane < p.rank) {
#pragma unroll
            for (int j = 0; j < 8; ++j) sq = fmaf(v[c][j], v[c][j], sq);
          }
      } else {
        for (int i = lane; i < p.rank; i += 32) {
          const float u = to_f(x[i]);
          sq = fmaf(u, u, sq);
        }
      }
      inv = rsqrtf(warp_sum(sq) / (float)p.rank + p.eps);
    }
    if (page < 0 || page >= p.num_pages || pos < 0) {   // (the same in the whole warp)
      if (lane == 0) flag(p.status, MLA_DEVICE_INDEX_OUT_OF_RANGE);
      continue;
    }
    const int in_page = row - at * p.page_size;
    TC* dl = static_cast<TC*>(p.latent) + page * p.l_page_stride + in_page * p.l_row_stride;
    TC* dr = static_cast<TC*>(p.rope) + page * p.r_page_stride + in_page * p.r_row_stride;
    if constexpr (kGroups > 0) {
#pragma unroll
      for (int c = 0; c < kGroups; ++c)
        if (256 * c + 8 * lane < p.rank) {
          float g[8];
          load8(w + 256 * c + 8 * lane, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] = v[c][j] * inv * g[j];
          store8(dl + 256 * c + 8 * lane, g);
        }
    } else {
      for (int i = lane; i < p.rank; i += 32) put(dl + i, to_f(x[i]) * inv * to_f(w[i]));
    }
    for (int j = lane; j < half; j += 32) {
      if (j != lane) re0 = to_f(rr[2 * j]), im0 = to_f(rr[2 * j + 1]);
      const float angle = rope_angle(pos, p.inv_freq[j]);
      float s, c;
      if (angle <= kSmallAngle) sincos_small(angle, s, c); else sincosf(angle, &s, &c);
      put(dr + j, re0 * c - im0 * s);
      put(dr + half + j, im0 * c + re0 * s);
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// kv_len_out = kv_len + count where that fits: a launch of its own where CTAs
// of the launch before read lengths that another would overwrite.
__global__ void __launch_bounds__(256) paged_lengths_kernel(const int32_t* kv_len, const int32_t* counts, int32_t most,
                                                            int64_t capacity, int32_t batch, int32_t* kv_len_out) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.x * 256 + threadIdx.x;
  if (b < batch) {
    const int len = kv_len[b], count = paged_count(counts, b, most);
    kv_len_out[b] = len >= 0 && count >= 0 && (int64_t)len + count <= capacity ? len + count : len;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ------------------------------------------------------------------ trees

// One CTA per tree, one thread per node.  Each node holds the mask of itself
// and the ancestors found so far, and the ancestor behind them; in a round it
// takes over both from that ancestor, so paths double in length (walking up
// node by node took 8.9 us for 64 trees of 256 nodes and depths around 45,
// launches included; this takes 4.0).  A launch and a few barriers: one tree of
// 16 nodes 2.2 us.
__global__ void __launch_bounds__(kMaxTreeNodes) tree_plan_kernel(const __grid_constant__ TreePlanParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  extern __shared__ uint64_t mask_s[];   // [n_nodes][words]
  __shared__ int32_t up_s[kMaxTreeNodes];
  const int b = blockIdx.x, j = threadIdx.x, n = p.n_nodes, words = (n + 63) >> 6;
  int up = j < n ? p.parents[b * p.parents_stride + j] : -1;
  int count = paged_count(p.counts, b, n);
  const int len = p.kv_len ? p.kv_len[b] : 0;
  if (count < 0 || len < 0) {
    if (j == 0) flag(p.status, MLA_DEVICE_INDEX_OUT_OF_RANGE);
    count = 0;
  }
  if (j >= count) {
    up = -1;
  } else if (up < -1 || up >= j) {   // not below an earlier node: a root
    flag(p.status, MLA_DEVICE_INDEX_OUT_OF_RANGE);
    up = -1;
  }
  uint64_t* mine = mask_s + j * words;
  const int own = j >> 6;   // ancestors have smaller numbers: the words behind a node's own stay empty
  if (j < n) {
    for (int k = 0; k < words; ++k) mine[k] = k == own && j < count ? 1ull << (j & 63) : 0ull;
    up_s[j] = up;
  }
  while (__syncthreads_or(up >= 0)) {
    uint64_t w[kMaxTreeNodes / 64];
    int next = -1;
    if (up >= 0) {
      next = up_s[up];
#pragma unroll
      for (int k = 0; k < kMaxTreeNodes / 64; ++k)
        if (k <= own) w[k] = mask_s[up * words + k];
    }
    __syncthreads();
    if (up >= 0) {
#pragma unroll
      for (int k = 0; k < kMaxTreeNodes / 64; ++k)
        if (k <= own) mine[k] |= w[k];
      up_s[j] = up = next;
    }
  }
  uint64_t* mask = p.mask + (int64_t)b * n * words;
  for (int i = j; i < n * words; i += blockDim.x) mask[i] = mask_s[i];
  if (j < n) {
    int nodes = 0;
    for (int k = 0; k <= own; ++k) nodes += __popcll(mine[k]);
    p.positions[(int64_t)b * n + j] = len + (nodes > 0 ? nodes - 1 : 0);
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ------------------------------------------------------------------ commit

constexpr int kCommitThreads = 128;
constexpr int kCommitBatch = 8;   // rows of a column in flight

// A thread owns one column of units of an array's rows and moves them in
// order, a batch of loads before its stores: row j comes from path[j] >= j,
// so no later row's source is overwritten and no thread waits for another.
// Bound by launch and the chain length, path, page, row: one row and layer 2.2
// us, 32 rows of up to 10 tokens in 24 layers 4.0 us (1.3 at the copy rate).
template <typename V>
__device__ __forceinline__ void commit_rows(const CommitArray& a, int count, const int64_t* from, const int64_t* to) {
  const int units = a.row_bytes / (int)sizeof(V);
  for (int u = threadIdx.x; u < units; u += kCommitThreads) {
    for (int j0 = 0; j0 < count; j0 += kCommitBatch) {
      V v[kCommitBatch];
#pragma unroll
      for (int k = 0; k < kCommitBatch; ++k)
        if (j0 + k < count && from[j0 + k] >= 0) {
          const int64_t f = from[j0 + k];
          v[k] = *(reinterpret_cast<const V*>(a.data + (f >> 32) * a.page_bytes_stride + (f & 0xffffffff) * a.row_bytes_stride) + u);
        }
#pragma unroll
      for (int k = 0; k < kCommitBatch; ++k)
        if (j0 + k < count && from[j0 + k] >= 0) {
          const int64_t t = to[j0 + k];
          *(reinterpret_cast<V*>(a.data + (t >> 32) * a.page_bytes_stride + (t & 0xffffffff) * a.row_bytes_stride) + u) = v[k];
        }
    }
  }
}

// grid (arrays, batch)
__global__ void __launch_bounds__(kCommitThreads) commit_paged_kernel(const __grid_constant__ CommitParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ int64_t from_s[kMaxTreeNodes], to_s[kMaxTreeNodes];   // page << 32 | row in it; from < 0: not moved
  const int b = blockIdx.y;
  const bool first = blockIdx.x == 0;
  const int64_t capacity = (int64_t)p.table_width * p.page_size;
  const int len = p.kv_len[b], count = paged_count(p.counts, b, p.path_width);
  const bool fits = len >= 0 && count >= 0 && (int64_t)len + count <= capacity;
  if (first && threadIdx.x == 0) {
    if (!fits) flag(p.status, MLA_DEVICE_INDEX_OUT_OF_RANGE);
    if (p.lengths_here) p.kv_len_out[b] = fits ? len + count : len;
  }
  const int moved = fits ? count : 0;
  const int32_t* path = p.path + b * p.path_stride;
  const int32_t* table = p.table + b * p.table_stride;
  for (int j = threadIdx.x; j < moved; j += kCommitThreads) {
    const int node = path[j], before = j > 0 ? path[j - 1] : -1;
    bool good = node >= j && node > before && (int64_t)len + node < capacity;
    int64_t from = -1, to = 0;
    if (good && node != j) {
      const int f = (len + node) / p.page_size, t = (len + j) / p.page_size;
      const int fp = table[f], tp = table[t];
      good = fp >= 0 && fp < p.num_pages && tp >= 0 && tp < p.num_pages;
      if (good) {
        from = (int64_t)fp << 32 | (len + node - f * p.page_size);
        to = (int64_t)tp << 32 | (len + j - t * p.page_size);
      }
    }
    if (!good && first) flag(p.status, MLA_DEVICE_INDEX_OUT_OF_RANGE);
    from_s[j] = from;
    to_s[j] = to;
  }
  __syncthreads();
  const CommitArray& a = p.a[blockIdx.x];
  switch (a.unit) {
    case 16: commit_rows<uint4>(a, moved, from_s, to_s); break;
    case 8: commit_rows<uint2>(a, moved, from_s, to_s); break;
    case 4: commit_rows<uint32_t>(a, moved, from_s, to_s); break;
    case 2: commit_rows<uint16_t>(a, moved, from_s, to_s); break;
    default: commit_rows<uint8_t>(a, moved, from_s, to_s); break;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

cudaError_t launch_lengths(const int32_t* kv_len, const int32_t* counts, int32_t most, int64_t capacity, int32_t batch,
                           int32_t* kv_len_out, cudaStream_t stream) {
  return launch_pdl(paged_lengths_kernel, dim3((unsigned)((batch + 255) / 256)), dim3(256), 0, stream, kv_len, counts,
                    most, capacity, batch, kv_len_out);
}

}  // namespace

cudaError_t launch_append_paged(AppendPagedParams p, int in_dtype, int cache_dtype, bool vec, cudaStream_t stream) {
  const int warps = p.s_new < kAppendWarps ? p.s_new : kAppendWarps;
  const dim3 grid((unsigned)((p.s_new + warps - 1) / warps), (unsigned)(p.batch < 65535 ? p.batch : 65535)), block(warps * 32);
  // Lengths written in place: by the kernel where one CTA has a row's tokens, else by a launch of their own.
  const bool in_place = p.kv_len_out == p.kv_len, after = in_place && grid.x > 1;
  p.lengths_here = !p.kv_len_out || after ? 0 : in_place ? 2 : 1;
  auto launch = [&](auto in, auto out) {
    using TI = decltype(in);
    using TC = decltype(out);
    return !vec             ? launch_pdl(append_paged_kernel<TI, TC, 0>, grid, block, 0, stream, p)
           : p.rank <= 512 ? launch_pdl(append_paged_kernel<TI, TC, 2>, grid, block, 0, stream, p)
                           : launch_pdl(append_paged_kernel<TI, TC, kMaxAppendRank / 256>, grid, block, 0, stream, p);
  };
  cudaError_t e;
  if (in_dtype == MLA_DTYPE_F32 && cache_dtype == MLA_DTYPE_F32)
    e = launch(0.f, 0.f);
  else if (in_dtype == MLA_DTYPE_F32)
    e = launch(0.f, __nv_bfloat16());
  else if (cache_dtype == MLA_DTYPE_F32)
    e = launch(__nv_bfloat16(), 0.f);
  else
    e = launch(__nv_bfloat16(), __nv_bfloat16());
  if (e == cudaSuccess && after)
    e = launch_lengths(p.kv_len, p.counts, p.s_new, (int64_t)p.table_width * p.page_size, p.batch, p.kv_len_out, stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_tree_plan(const TreePlanParams& p, cudaStream_t stream) {
  constexpr int most = kMaxTreeNodes * (kMaxTreeNodes / 64) * 8;
  const size_t smem = (size_t)p.n_nodes * ((p.n_nodes + 63) / 64) * 8;
  if (smem > 40 * 1024) {   // (48 KB a kernel has without asking, less its static part)
    const cudaError_t ea = set_max_dynamic_smem(tree_plan_kernel, most);
    if (ea != cudaSuccess) return ea;
  }
  const cudaError_t e = launch_pdl(tree_plan_kernel, dim3((unsigned)p.batch), dim3((unsigned)((p.n_nodes + 31) & ~31)), smem,
                                   stream, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_commit_paged(CommitParams& p, cudaStream_t stream) {
  const bool after = p.kv_len_out == p.kv_len;
  p.lengths_here = p.kv_len_out && !after;
  cudaError_t e = launch_pdl(commit_paged_kernel, dim3((unsigned)p.n_arrays, (unsigned)p.batch), dim3(kCommitThreads), 0,
                             stream, p);
  if (e == cudaSuccess && after)
    e = launch_lengths(p.kv_len, p.counts, p.path_width, (int64_t)p.table_width * p.page_size, p.batch, p.kv_len_out, stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mla
