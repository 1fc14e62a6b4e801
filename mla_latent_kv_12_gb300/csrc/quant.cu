// Writing and reading an 8-bit latent cache: append of new tokens (RMSNorm,
// RoPE, 8-bit codes), and conversion of cache windows between bf16 / f32 and
// 8 bits.
//
// Rows are taken in tiles of max(block, 16) buffer rows that start on whole
// blocks, one CTA per tile, one warp per token at a time.  The unit of a block is
// known only once the largest magnitude of all its tokens is, so a tile is
// walked twice: the first walk reduces each token (sum of squares, largest
// magnitude), the second, after a barrier, encodes; it reads the tokens again
// from L1 / L2, which costs no memory traffic.  Bound by memory: 2 * rank +
// 2 * rope bytes in and rank + 2 * rope bytes out per bf16 token.
#include <cuda_bf16.h>

#include "e4m3.cuh"
#include "mla_internal.h"
#include "rope_math.cuh"
#include "tc_host.h"

namespace mla {
namespace {

constexpr int kWarps = 8;
constexpr int kMinTileRows = 16;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Eight consecutive values, 16-byte aligned.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}

// Calls f(i, v, n) for this lane's groups of a row's elements: eight at a time
// from 16-byte loads (kVec: rank a multiple of 8, aligned rows), else one.
template <bool kVec, typename T, typename F>
__device__ __forceinline__ void for_row(const T* row, int rank, int lane, F&& f) {
  if constexpr (kVec) {
#pragma unroll 2
    for (int i = 8 * lane; i < rank; i += 256) {
      float v[8];
      load8(row + i, v);
      f(i, v, 8);
    }
  } else {
    for (int i = lane; i < rank; i += 32) {
      float v[8];
      v[0] = to_f(row[i]);
      f(i, v, 1);
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// NaN is passed over (it has a code of its own), so it does not set a unit.
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// kNorm: new tokens of an append (normalised, weighted, with their rope key);
// otherwise the tokens of each row's window of a latent buffer.
template <bool kNorm, bool kVec, typename TI, typename TR>
__global__ void __launch_bounds__(kWarps * 32) encode_kernel(const __grid_constant__ EncodeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ uint32_t amax_s[kMaxScaleBlock];   // per block of the tile, f32 bits (non-negative: ordered as integers)
  __shared__ int exp_s[kMaxScaleBlock], old_exp_s[kMaxScaleBlock];
  __shared__ float inv_s[kMaxScaleBlock];       // per row of the tile
  const int b = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = p.kv_len[b];
  const int start = p.kv_start ? p.kv_start[b] : 0;
  const int64_t pos0 = !kNorm ? 0 : (p.row_offsets ? (int64_t)p.row_offsets[b] : (int64_t)len);
  const int block = 1 << p.block_shift;
  const bool aligned = (start & (block - 1)) == 0;
  const bool fits = len >= 0 && start >= 0 && pos0 >= 0 &&
                    (int64_t)start + len + (kNorm ? p.s_new : 0) <= p.t_max;
  const bool ok = fits && aligned;
  if (!ok && blockIdx.x == 0 && threadIdx.x == 0 && p.status)
    atomicOr(p.status, fits ? MLA_DEVICE_BAD_BLOCK_START : MLA_DEVICE_INDEX_OUT_OF_RANGE);
  // the rows written: [lo, hi)
  const int64_t lo = kNorm ? (int64_t)start + len : start;
  const int64_t hi = kNorm ? lo + p.s_new : (int64_t)start + len;
  const int tile_rows = p.tile_rows;
  const int64_t tile0 = lo / tile_rows;
  const int64_t n_tiles = ok && hi > lo ? (hi - 1) / tile_rows - tile0 + 1 : 0;
  uint8_t* codes = p.codes + b * p.codes_batch_stride;
  uint8_t* scales = p.scales + b * p.scales_batch_stride;
  const TI* src = static_cast<const TI*>(p.latent_raw) + b * p.lr_row_stride;
  const TI* gain = static_cast<const TI*>(p.weight);
  // token row r of the buffer: token r - lo of the new ones, or row r of the source buffer
  auto source = [&](int64_t r) { return src + (kNorm ? r - lo : r) * p.lr_tok_stride; };

  for (int64_t tile = blockIdx.x; tile < n_tiles; tile += gridDim.x) {
    const int64_t base = (tile0 + tile) * tile_rows;
    const int r_lo = (int)max((int64_t)0, lo - base), r_hi = (int)min((int64_t)tile_rows, hi - base);
    const int n_blocks = tile_rows >> p.block_shift;
    for (int k = threadIdx.x; k < n_blocks; k += kWarps * 32) amax_s[k] = 0;
    __syncthreads();
    for (int r = r_lo + warp; r < r_hi; r += kWarps) {
      const TI* row = source(base + r);
      float inv = 1.f;
      if constexpr (kNorm) {
        float sq = 0.f;
        for_row<kVec>(row, p.rank, lane, [&](int, const float(&v)[8], int n) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < n) sq = fmaf(v[j], v[j], sq);
        });
        inv = rsqrtf(warp_sum(sq) / (float)p.rank + p.eps);
      }
      float amax = 0.f;
      for_row<kVec>(row, p.rank, lane, [&](int i, const float(&v)[8], int n) {
        if constexpr (kNorm) {
          float g[8];
          if constexpr (kVec) load8(gain + i, g); else g[0] = to_f(gain[i]);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < n) amax = fmaxf(amax, fabsf(v[j] * inv * g[j]));
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < n) amax = fmaxf(amax, fabsf(v[j]));
        }
      });
      amax = warp_max(amax);
      if (lane == 0) {
        atomicMax(&amax_s[r >> p.block_shift], __float_as_uint(amax));
        inv_s[r] = inv;
      }
    }
    __syncthreads();
    // one thread per block with rows to write: its exponent, never below that of the tokens it holds already
    for (int k = threadIdx.x; k < n_blocks; k += kWarps * 32) {
      const int k_lo = k << p.block_shift, k_hi = k_lo + block;
      if (k_hi <= r_lo || k_lo >= r_hi) continue;
      const float amax = __uint_as_float(amax_s[k]);
      int e = exponent_for(amax), old = -1;
      uint8_t* at = scales + (base >> p.block_shift) + k;
      if (kNorm && base + k_lo < lo && start < lo) {   // rows [max(block start, start), lo) hold tokens
        old = *at;
        e = max(e, clamp_exponent(old));
      }
      if (!(amax <= 448.f * 128.f) && p.status) atomicOr(p.status, MLA_DEVICE_VALUE_RANGE);
      exp_s[k] = e;
      old_exp_s[k] = old;
      *at = (uint8_t)e;
    }
    __syncthreads();
    for (int r = r_lo + warp; r < r_hi; r += kWarps) {
      const TI* row = source(base + r);
      const float inv = inv_s[r], to_units = inverse_unit_of(exp_s[r >> p.block_shift]);
      uint8_t* dst = codes + (base + r) * p.codes_row_stride;
      for_row<kVec>(row, p.rank, lane, [&](int i, const float(&v)[8], int n) {
        float x[8], g[8];
        if constexpr (kNorm) {
          if constexpr (kVec) load8(gain + i, g); else g[0] = to_f(gain[i]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) x[j] = (kNorm ? v[j] * inv * g[j] : v[j]) * to_units;   // a power of two: exact
        if constexpr (kVec) {
          const uint32_t w0 = encode_e4m3x2(x[0], x[1]) | (uint32_t)encode_e4m3x2(x[2], x[3]) << 16;
          const uint32_t w1 = encode_e4m3x2(x[4], x[5]) | (uint32_t)encode_e4m3x2(x[6], x[7]) << 16;
          *reinterpret_cast<uint2*>(dst + i) = make_uint2(w0, w1);
        } else {
          dst[i] = encode_e4m3(x[0]);
        }
      });
      if constexpr (kNorm) {
        const int64_t t = base + r - lo;
        const TI* rr = static_cast<const TI*>(p.rope_raw) + b * p.rr_row_stride + t * p.rr_tok_stride;
        TR* dr = static_cast<TR*>(p.rope) + b * p.rope_batch_stride + (base + r) * p.rope_row_stride;
        const int half = p.rope_dim >> 1;
        for (int j = lane; j < half; j += 32) {
          float re, im;
          rope_rotate_pair(to_f(rr[2 * j]), to_f(rr[2 * j + 1]), pos0 + t, p.inv_freq[j], re, im);
          put(dr + j, re);
          put(dr + half + j, im);
        }
      }
    }
    if constexpr (kNorm) {
      // tokens that the first block held before: their codes move to the larger unit
      const int k0 = r_lo >> p.block_shift;
      const int old = old_exp_s[k0], e = exp_s[k0];
      if (old >= 0 && clamp_exponent(old) != e) {
        const float unit = unit_of(clamp_exponent(old)), to_units = inverse_unit_of(e);
        const int64_t first = max(base + ((int64_t)k0 << p.block_shift), (int64_t)start);
        for (int64_t r = first + warp; r < lo; r += kWarps) {
          uint8_t* dst = codes + r * p.codes_row_stride;
          for (int i = lane; i < p.rank; i += 32) dst[i] = encode_e4m3(decode_e4m3(dst[i], unit) * to_units);
        }
      }
    }
    __syncthreads();   // the tile's shared state is read before the next one overwrites it
  }
  if constexpr (kNorm) {
    // one CTA per row: every thread has read the length before it may be overwritten
    if (p.lengths_here) {
      __syncthreads();
      if (threadIdx.x == 0) p.kv_len_out[b] = ok ? len + p.s_new : len;
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The new lengths of an append whose rows take several CTAs each (they read
// kv_len, which kv_len_out may alias): the same conditions, after the append.
__global__ void lengths_kernel(const __grid_constant__ EncodeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b < p.batch) {
    const int len = p.kv_len[b], start = p.kv_start ? p.kv_start[b] : 0;
    const int64_t pos0 = p.row_offsets ? (int64_t)p.row_offsets[b] : (int64_t)len;
    const bool ok = len >= 0 && start >= 0 && pos0 >= 0 && (int64_t)start + len + p.s_new <= p.t_max &&
                    (start & ((1 << p.block_shift) - 1)) == 0;
    p.kv_len_out[b] = ok ? len + p.s_new : len;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// One warp per window row: 16 codes a lane (kVec) or one.
template <bool kVec, typename TO>
__global__ void __launch_bounds__(kWarps * 32) decode_rows_kernel(const __grid_constant__ EncodeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = p.kv_len[b];
  const int start = p.kv_start ? p.kv_start[b] : 0;
  const bool aligned = (start & ((1 << p.block_shift) - 1)) == 0;
  const bool fits = len >= 0 && start >= 0 && (int64_t)start + len <= p.t_max;
  if (!(fits && aligned)) {
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.status)
      atomicOr(p.status, fits ? MLA_DEVICE_BAD_BLOCK_START : MLA_DEVICE_INDEX_OUT_OF_RANGE);
  } else {
    const uint8_t* codes = p.codes + b * p.codes_batch_stride;
    const uint8_t* scales = p.scales + b * p.scales_batch_stride;
    TO* out = static_cast<TO*>(p.latent_out) + b * p.lo_batch_stride;
    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < len; t += (int64_t)gridDim.x * kWarps) {
      const int64_t r = start + t;
      const int e = clamp_exponent(scales[r >> p.block_shift]);
      const uint8_t* row = codes + r * p.codes_row_stride;
      TO* dst = out + r * p.lo_row_stride;
      if constexpr (kVec) {
        for (int i = 16 * lane; i < p.rank; i += 512) {
          uint32_t v[8];
          const uint4 c = *reinterpret_cast<const uint4*>(row + i);
          if (decode_e4m3x16(c, bf16_unit(e), v)) mend_nan_e4m3x16(c, v);
          uint4* d = reinterpret_cast<uint4*>(dst + i);
          if constexpr (sizeof(TO) == 2) {
            d[0] = make_uint4(v[0], v[1], v[2], v[3]);
            d[1] = make_uint4(v[4], v[5], v[6], v[7]);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              d[k] = make_uint4(v[2 * k] << 16, v[2 * k] & 0xFFFF0000u, v[2 * k + 1] << 16, v[2 * k + 1] & 0xFFFF0000u);
          }
        }
      } else {
        const float unit = unit_of(e);
        for (int i = lane; i < p.rank; i += 32) put(dst + i, decode_e4m3(row[i], unit));
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <bool kNorm, typename TI, typename TR>
cudaError_t launch_encode_t(const EncodeParams& p, bool vec, dim3 grid, cudaStream_t stream) {
  const dim3 block(kWarps * 32);
  return vec ? launch_pdl(encode_kernel<kNorm, true, TI, TR>, grid, block, 0, stream, p)
             : launch_pdl(encode_kernel<kNorm, false, TI, TR>, grid, block, 0, stream, p);
}

}  // namespace

cudaError_t launch_append_q8(const EncodeParams& p_in, int in_dtype, int rope_dtype, bool vec, cudaStream_t stream) {
  EncodeParams p = p_in;
  p.tile_rows = (1 << p.block_shift) > kMinTileRows ? (1 << p.block_shift) : kMinTileRows;
  // Tiles that s_new rows can touch.  Up to two are walked by one CTA per row,
  // which then writes the row's new length itself (a decode step's append is
  // one launch); more are spread over CTAs and the lengths take a launch of
  // their own.
  const int64_t tiles = ((int64_t)p.s_new + p.tile_rows - 2) / p.tile_rows + 1;
  const unsigned gx = tiles <= 2 ? 1u : (unsigned)(tiles < 65535 ? tiles : 65535);
  p.lengths_here = gx == 1 && p.kv_len_out != nullptr;
  const dim3 grid(gx, (unsigned)p.batch);
  cudaError_t e;
  if (in_dtype == MLA_DTYPE_F32)
    e = rope_dtype == MLA_DTYPE_F32 ? launch_encode_t<true, float, float>(p, vec, grid, stream)
                                    : launch_encode_t<true, float, __nv_bfloat16>(p, vec, grid, stream);
  else
    e = rope_dtype == MLA_DTYPE_F32 ? launch_encode_t<true, __nv_bfloat16, float>(p, vec, grid, stream)
                                    : launch_encode_t<true, __nv_bfloat16, __nv_bfloat16>(p, vec, grid, stream);
  if (e != cudaSuccess) return e;
  if (p.kv_len_out && !p.lengths_here)
    e = launch_pdl(lengths_kernel, dim3((p.batch + 127) / 128), dim3(128), 0, stream, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_quantize(const EncodeParams& p_in, int dtype, bool vec, cudaStream_t stream) {
  EncodeParams p = p_in;
  p.tile_rows = (1 << p.block_shift) > kMinTileRows ? (1 << p.block_shift) : kMinTileRows;
  const int64_t tiles = (p.t_max + p.tile_rows - 1) / p.tile_rows;
  const dim3 grid((unsigned)(tiles < 65535 ? tiles : 65535), (unsigned)p.batch);
  const cudaError_t e = dtype == MLA_DTYPE_F32
                            ? launch_encode_t<false, float, float>(p, vec, grid, stream)
                            : launch_encode_t<false, __nv_bfloat16, __nv_bfloat16>(p, vec, grid, stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_dequantize(const EncodeParams& p, int dtype, bool vec, cudaStream_t stream) {
  const int64_t per_cta = 4 * kWarps;   // a few rows per warp
  const int64_t gx = (p.t_max + per_cta - 1) / per_cta;
  const dim3 grid((unsigned)(gx < 65535 ? gx : 65535), (unsigned)p.batch), block(kWarps * 32);
  cudaError_t e;
  if (dtype == MLA_DTYPE_F32)
    e = vec ? launch_pdl(decode_rows_kernel<true, float>, grid, block, 0, stream, p)
            : launch_pdl(decode_rows_kernel<false, float>, grid, block, 0, stream, p);
  else
    e = vec ? launch_pdl(decode_rows_kernel<true, __nv_bfloat16>, grid, block, 0, stream, p)
            : launch_pdl(decode_rows_kernel<false, __nv_bfloat16>, grid, block, 0, stream, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mla
