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

// One warp per new token.
template <typename TI, typename TC>
__global__ void __launch_bounds__(kAppendWarps * 32) append_paged_kernel(const __grid_constant__ AppendPagedParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float freq_s[kMaxRotaryDims / 2];
  const int half = p.rope_dim >> 1;
  if ((int)threadIdx.x < half) freq_s[threadIdx.x] = p.inv_freq[threadIdx.x];
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tokens = (int64_t)p.batch * p.s_new, capacity = (int64_t)p.table_width * p.page_size;
  for (int64_t k = (int64_t)blockIdx.x * kAppendWarps + warp; k < tokens; k += (int64_t)gridDim.x * kAppendWarps) {
    const int b = (int)(k / p.s_new), t = (int)(k % p.s_new);
    const int len = p.kv_len[b], count = paged_count(p.counts, b, p.s_new);
    const bool fits = len >= 0 && count >= 0 && (int64_t)len + count <= capacity;
    if (lane == 0 && t == 0) {
      if (!fits) flag(p.status, MLA_DEVICE_INDEX_OUT_OF_RANGE);
      if (p.lengths_here) p.kv_len_out[b] = fits ? len + count : len;
    }
    if (!fits || t >= count) continue;
    const int row = len + t, at = row / p.page_size;
    const int page = p.table[b * p.table_stride + at];
    const int64_t pos = p.positions ? (int64_t)p.positions[k] : (int64_t)row;
    if (page < 0 || page >= p.num_pages || pos < 0) {
      if (lane == 0) flag(p.status, MLA_DEVICE_INDEX_OUT_OF_RANGE);
      continue;
    }
    const int in_page = row - at * p.page_size;
    const TI* x = static_cast<const TI*>(p.latent_raw) + b * p.lr_row_stride + t * p.lr_tok_stride;
    const TI* w = static_cast<const TI*>(p.weight);
    TC* dl = static_cast<TC*>(p.latent) + page * p.l_page_stride + in_page * p.l_row_stride;
    float sq = 0.f;
    for (int i = lane; i < p.rank; i += 32) {
      const float v = to_f(x[i]);
      sq = fmaf(v, v, sq);
    }
    const float inv = rsqrtf(warp_sum(sq) / (float)p.rank + p.eps);
    for (int i = lane; i < p.rank; i += 32) put(dl + i, to_f(x[i]) * inv * to_f(w[i]));
    const TI* rr = static_cast<const TI*>(p.rope_raw) + b * p.rr_row_stride + t * p.rr_tok_stride;
    TC* dr = static_cast<TC*>(p.rope) + page * p.r_page_stride + in_page * p.r_row_stride;
    for (int j = lane; j < half; j += 32) {
      float re, im;
      rope_rotate_pair(to_f(rr[2 * j]), to_f(rr[2 * j + 1]), pos, freq_s[j], re, im);
      put(dr + j, re);
      put(dr + half + j, im);
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

// One CTA per tree, one thread per node.  A node's ancestors have smaller
// numbers, so walking up from it fills its mask's words from the last to the
// first.
__global__ void __launch_bounds__(kMaxTreeNodes) tree_plan_kernel(const __grid_constant__ TreePlanParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ int32_t parent_s[kMaxTreeNodes];
  const int b = blockIdx.x, j = threadIdx.x;
  int count = paged_count(p.counts, b, p.n_nodes);
  const int len = p.kv_len ? p.kv_len[b] : 0;
  if (count < 0 || len < 0) {
    if (j == 0) flag(p.status, MLA_DEVICE_INDEX_OUT_OF_RANGE);
    count = 0;
  }
  if (j < p.n_nodes) {
    int up = -1;
    if (j < count) {
      up = p.parents[b * p.parents_stride + j];
      if (up < -1 || up >= j) {   // not below an earlier node: a root
        flag(p.status, MLA_DEVICE_INDEX_OUT_OF_RANGE);
        up = -1;
      }
    }
    parent_s[j] = up;
  }
  __syncthreads();
  if (j < p.n_nodes) {
    const int words = (p.n_nodes + 63) >> 6;
    uint64_t* mask = p.mask + ((int64_t)b * p.n_nodes + j) * words;
    int at = words - 1, depth = -1;
    uint64_t word = 0;
    for (int node = j < count ? j : -1; node >= 0; node = parent_s[node]) {
      for (; at > node >> 6; --at) mask[at] = word, word = 0;
      word |= 1ull << (node & 63);
      ++depth;
    }
    for (; at >= 0; --at) mask[at] = word, word = 0;
    p.positions[(int64_t)b * p.n_nodes + j] = len + (depth > 0 ? depth : 0);
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ------------------------------------------------------------------ commit

constexpr int kCommitThreads = 128;
constexpr int kCommitBatch = 8;   // rows of a column in flight

// A thread owns one column of units of an array's rows and moves them in
// order, a batch of loads before its stores: row j comes from path[j] >= j,
// so no later row's source is overwritten and no thread waits for another.
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

cudaError_t launch_append_paged(AppendPagedParams p, int in_dtype, int cache_dtype, cudaStream_t stream) {
  const int64_t tokens = (int64_t)p.batch * p.s_new;
  const int64_t ctas = (tokens + kAppendWarps - 1) / kAppendWarps, most = 8LL * device_sm_count();
  const dim3 grid((unsigned)(ctas < most ? ctas : most)), block(kAppendWarps * 32);
  // lengths that other CTAs still read are written by a launch of their own
  const bool after = p.kv_len_out == p.kv_len;
  p.lengths_here = p.kv_len_out && !after;
  cudaError_t e;
  if (in_dtype == MLA_DTYPE_F32 && cache_dtype == MLA_DTYPE_F32)
    e = launch_pdl(append_paged_kernel<float, float>, grid, block, 0, stream, p);
  else if (in_dtype == MLA_DTYPE_F32)
    e = launch_pdl(append_paged_kernel<float, __nv_bfloat16>, grid, block, 0, stream, p);
  else if (cache_dtype == MLA_DTYPE_F32)
    e = launch_pdl(append_paged_kernel<__nv_bfloat16, float>, grid, block, 0, stream, p);
  else
    e = launch_pdl(append_paged_kernel<__nv_bfloat16, __nv_bfloat16>, grid, block, 0, stream, p);
  if (e == cudaSuccess && after)
    e = launch_lengths(p.kv_len, p.counts, p.s_new, (int64_t)p.table_width * p.page_size, p.batch, p.kv_len_out, stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_tree_plan(const TreePlanParams& p, cudaStream_t stream) {
  const cudaError_t e = launch_pdl(tree_plan_kernel, dim3((unsigned)p.batch), dim3((unsigned)((p.n_nodes + 31) & ~31)), 0,
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
