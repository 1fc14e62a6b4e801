// Writing and reading an 8-bit latent cache: append of new tokens (RMSNorm,
// RoPE, 8-bit codes), and conversion of cache windows between bf16 / f32 and
// 8 bits.
//
// The unit of a block is known only once the largest magnitude of all its tokens
// is.  Rows are taken in tiles that start on whole blocks, one CTA per tile.
// encode_kernel (ranks up to 512 of aligned rows) takes 64 rows, four
// neighbouring ones per warp, and holds them in registers: a warp's loads are
// all in flight together, its tokens are reduced, and then encoded -- after a
// barrier where a block spans warps, at once where it does not (blocks of up
// to four tokens).  encode_walk_kernel serves every other shape: it walks a
// tile of max(block, 16) rows twice, the second time from L1 / L2.  Bound by
// memory: 2 * rank + 2 * rope bytes in and rank + 2 * rope bytes out per bf16
// token.  Measured: 16 x 16384 tokens quantised in 68 us (5.9 TB/s), 8 x 2048
// appended in 14.7 us (2.0 TB/s: one wave of CTAs), 16 x 16384 dequantised in
// 67 us (6.0 TB/s).
#include <cuda_bf16.h>
#include <float.h>

#include "e4m3.cuh"
#include "mla_internal.h"
#include "rope_math.cuh"
#include "tc_common.cuh"
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
// Four sums over the warp at once, every lane receiving all of them: the first
// two steps halve the sums a lane carries.
__device__ __forceinline__ void warp_sum4(float (&v)[4]) {
  const int lane = threadIdx.x & 31;
  const bool b4 = lane & 16, b3 = lane & 8;
  float x = (b4 ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, b4 ? v[0] : v[2], 16);
  const float y = (b4 ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, b4 ? v[1] : v[3], 16);
  x = (b3 ? y : x) + __shfl_xor_sync(0xffffffffu, b3 ? x : y, 8);   // lanes 0-7: v[0], 8-15: v[1], 16-23: v[2], 24-31: v[3]
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = __shfl_sync(0xffffffffu, x, 8 * k);
}
// NaN is passed over (it has a code of its own), so it does not set a unit.
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The rows that a batch row's call writes, and the state of its tile walk.
template <bool kNorm>
struct EncodeRow {
  int len, start;
  int64_t pos0;        // position of the first new token
  bool ok;
  int64_t lo, hi;      // rows written: [lo, hi)
  __device__ EncodeRow(const EncodeParams& p, int b, bool flag) {
    len = p.kv_len[b];
    start = p.kv_start ? p.kv_start[b] : 0;
    pos0 = !kNorm ? 0 : (p.row_offsets ? (int64_t)p.row_offsets[b] : (int64_t)len);
    const bool aligned = (start & ((1 << p.block_shift) - 1)) == 0;
    const bool fits = len >= 0 && start >= 0 && pos0 >= 0 && (int64_t)start + len + (kNorm ? p.s_new : 0) <= p.t_max;
    ok = fits && aligned;
    if (!ok && flag && p.status) atomicOr(p.status, fits ? MLA_DEVICE_BAD_BLOCK_START : MLA_DEVICE_INDEX_OUT_OF_RANGE);
    lo = kNorm ? (int64_t)start + len : start;
    hi = kNorm ? lo + p.s_new : (int64_t)start + len;
  }
  __device__ int64_t tiles(int tile_rows) const { return ok && hi > lo ? (hi - 1) / tile_rows - lo / tile_rows + 1 : 0; }
};

// The exponent of block k of a tile at buffer row `base`, from the largest
// magnitude of its new tokens: never below that of tokens the block holds
// already (rows [max(block start, start), lo); `old` receives their exponent
// byte, else -1).  Written to the cache.
template <bool kNorm>
__device__ __forceinline__ int block_exponent(const EncodeParams& p, const EncodeRow<kNorm>& row, uint8_t* scales,
                                              int64_t base, int k, float amax, int& old) {
  uint8_t* at = scales + (base >> p.block_shift) + k;
  int e = exponent_for(amax);
  old = -1;
  if (kNorm && base + ((int64_t)k << p.block_shift) < row.lo && row.start < row.lo) {
    old = *at;
    e = max(e, clamp_exponent(old));
  }
  if (!(amax <= 448.f * 128.f) && p.status) atomicOr(p.status, MLA_DEVICE_VALUE_RANGE);
  *at = (uint8_t)e;
  return e;
}

// The rope key of new token t, pairs from `lane` on (every 32nd): rotated at its position, into buffer row `row`.
// (`freq`: the inverse frequencies in shared memory; lanes that index the
// parameters' constant bank apart are served one by one.)
template <typename TI, typename TR>
__device__ __forceinline__ void append_rope(const EncodeParams& p, const float* freq, int b, int64_t t, int64_t row,
                                            int64_t pos, int lane) {
  const TI* rr = static_cast<const TI*>(p.rope_raw) + b * p.rr_row_stride + t * p.rr_tok_stride;
  TR* dr = static_cast<TR*>(p.rope) + b * p.rope_batch_stride + row * p.rope_row_stride;
  const int half = p.rope_dim >> 1;
  for (int j = lane; j < half; j += 32) {
    float re, im;
    rope_rotate_pair(to_f(rr[2 * j]), to_f(rr[2 * j + 1]), pos, freq[j], re, im);
    put(dr + j, re);
    put(dr + half + j, im);
  }
}

// Sine and cosine of |x| <= kSmallAngle without branches: x less the nearest
// multiple of pi / 2, which is subtracted in three f32 parts with fused
// multiply-adds (Cody and Waite; the first is exact: x and the multiple are both
// multiples of 2^-24, their difference is below 1), then the Taylor sums, whose
// remainders on [-pi/4, pi/4] are below 2^-28.  Absolute error below 1.2 * 2^-24
// (against 64 bits over the range and next to the multiples of pi / 2).
constexpr float kSmallAngle = 65536.f;
__device__ __forceinline__ void sincos_small(float x, float& sine, float& cosine) {
  const float shifted = fmaf(x, 0.6366197723675814f, 12582912.f);   // 1.5 * 2^23: the low bits are the nearest integer
  const uint32_t quadrant = __float_as_uint(shifted);
  const float k = shifted - 12582912.f;
  float r = fmaf(-k, 0x1.921fb6p+0f, x);
  r = fmaf(-k, -0x1.777a5cp-25f, r);
  r = fmaf(-k, -0x1.ee59dap-50f, r);
  const float z = r * r;
  float s = fmaf(fmaf(fmaf(1.f / 362880, z, -1.f / 5040), z, 1.f / 120), z, -1.f / 6);
  s = fmaf(r * z, s, r);
  float c = fmaf(fmaf(fmaf(-1.f / 3628800, z, 1.f / 40320), z, -1.f / 720), z, 1.f / 24);
  c = fmaf(fmaf(c, z, -0.5f), z, 1.f);
  const bool swap = quadrant & 1u;
  sine = __uint_as_float(__float_as_uint(swap ? c : s) ^ ((quadrant & 2u) << 30));
  cosine = __uint_as_float(__float_as_uint(swap ? s : c) ^ (((quadrant + 1u) & 2u) << 30));
}

// The codes of rows [first, lo), which a block held before, move from unit `old` to unit `e`.
template <int kThreads>
__device__ __forceinline__ void move_codes(const EncodeParams& p, uint8_t* codes, int64_t first, int64_t lo, int old,
                                           int e) {
  const float unit = unit_of(clamp_exponent(old)), to_units = inverse_unit_of(e);
  for (int64_t r = first + (threadIdx.x >> 5); r < lo; r += kThreads / 32) {
    uint8_t* dst = codes + r * p.codes_row_stride;
    for (int i = threadIdx.x & 31; i < p.rank; i += 32) dst[i] = encode_e4m3(decode_e4m3(dst[i], unit) * to_units);
  }
}

__device__ __forceinline__ uint2 encode8(const float (&x)[8]) {
  return make_uint2(encode_e4m3x2(x[0], x[1]) | (uint32_t)encode_e4m3x2(x[2], x[3]) << 16,
                    encode_e4m3x2(x[4], x[5]) | (uint32_t)encode_e4m3x2(x[6], x[7]) << 16);
}

// Eight consecutive raw values as loaded, and as four pairs.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ void get(float2 (&v)[4]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ void load(const float* p) { a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1]; }
  __device__ void get(float2 (&v)[4]) const {
    v[0] = make_float2(a.x, a.y), v[1] = make_float2(a.z, a.w), v[2] = make_float2(b.x, b.y), v[3] = make_float2(b.z, b.w);
  }
};
// (a0 b0 + c0, a1 b1 + c1) as one packed f32x2 operation.
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

// Tiles of 64 rows, four neighbouring ones per warp; lane l holds elements
// 8l .. 8l + 7 and 256 + those of each.
constexpr int kHeldWarps = 16, kHeldRows = 4, kHeldTile = kHeldWarps * kHeldRows, kHeldRank = 512;
static_assert(kHeldTile >= kMaxScaleBlock, "a tile holds whole blocks");

template <bool kNorm, typename TI, typename TR>
__global__ void __launch_bounds__(kHeldWarps * 32, sizeof(TI) == 2 ? 2 : 1) encode_kernel(const __grid_constant__ EncodeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ uint32_t amax_s[kHeldTile];   // per block of the tile, f32 bits (non-negative: ordered as integers)
  __shared__ int exp_s[kHeldTile], old_s;
  __shared__ float freq_s[kNorm ? kMaxRotaryDims / 2 : 1];
  const int b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const EncodeRow<kNorm> row(p, b, blockIdx.x == 0 && threadIdx.x == 0);
  uint8_t* codes = p.codes + b * p.codes_batch_stride;
  uint8_t* scales = p.scales + b * p.scales_batch_stride;
  const TI* src = static_cast<const TI*>(p.latent_raw) + b * p.lr_row_stride;
  const TI* gain = static_cast<const TI*>(p.weight);
  const int block = 1 << p.block_shift, n_blocks = kHeldTile >> p.block_shift;
  const bool warp_blocks = block <= kHeldRows;   // no block spans warps
  const int64_t n_tiles = row.tiles(kHeldTile);
  const int half = p.rope_dim >> 1;
  if constexpr (kNorm) {
    if ((int)threadIdx.x < half) freq_s[threadIdx.x] = p.inv_freq[threadIdx.x];   // (read behind the tile's barriers)
  }
  bool live[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) live[c] = 256 * c + 8 * lane < p.rank;

  for (int64_t tile = blockIdx.x; tile < n_tiles; tile += gridDim.x) {
    const int64_t base = (row.lo / kHeldTile + tile) * kHeldTile;
    const int r_lo = (int)max((int64_t)0, row.lo - base), r_hi = (int)min((int64_t)kHeldTile, row.hi - base);
    const int r0 = kHeldRows * warp;   // this warp's first row
    auto mine = [&](int k) { return r0 + k >= r_lo && r0 + k < r_hi; };
    Raw8<TI> raw[kHeldRows][2];
    float ra[kHeldRows], rb[kHeldRows];   // this lane's rope pair (j = lane)
#pragma unroll
    for (int k = 0; k < kHeldRows; ++k) {
      if (!mine(k)) continue;
      const int64_t t = kNorm ? base + r0 + k - row.lo : base + r0 + k;
      const TI* x = src + t * p.lr_tok_stride + 8 * lane;
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (live[c]) raw[k][c].load(x + 256 * c);
      if (kNorm && lane < half) {
        const TI* rr = static_cast<const TI*>(p.rope_raw) + b * p.rr_row_stride + t * p.rr_tok_stride;
        ra[k] = to_f(rr[2 * lane]);
        rb[k] = to_f(rr[2 * lane + 1]);
      }
    }
    Raw8<TI> g[2];
    if constexpr (kNorm) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (live[c]) g[c].load(gain + 256 * c + 8 * lane);
    }
    if (!warp_blocks)
      for (int k = threadIdx.x; k < n_blocks; k += kHeldWarps * 32) amax_s[k] = 0;
    if (kNorm || !warp_blocks) __syncthreads();
    // The rope keys first: their sines and cosines while the latents arrive.
    if constexpr (kNorm) {
      if (lane < half) {
        const int64_t pos = row.pos0 + (base + r0 - row.lo);   // of the warp's first row
        const float freq = freq_s[lane];
        float sine[kHeldRows], cosine[kHeldRows], top = 0.f;
#pragma unroll
        for (int k = 0; k < kHeldRows; ++k) {
          // (the angle of rope_angle; sine holds it first)
          sine[k] = row.pos0 + p.s_new <= (1 << 24) ? __fmul_rn((float)(int)(pos + k), freq) : rope_angle(pos + k, freq);
          top = fmaxf(top, fabsf(sine[k]));
        }
        if (top <= kSmallAngle) {
#pragma unroll
          for (int k = 0; k < kHeldRows; ++k) sincos_small(sine[k], sine[k], cosine[k]);
        } else {
#pragma unroll
          for (int k = 0; k < kHeldRows; ++k) sincosf(sine[k], &sine[k], &cosine[k]);
        }
        TR* dr = static_cast<TR*>(p.rope) + b * p.rope_batch_stride + (base + r0) * p.rope_row_stride + lane;
#pragma unroll
        for (int k = 0; k < kHeldRows; ++k, dr += p.rope_row_stride) {
          if (!mine(k)) continue;
          put(dr, ra[k] * cosine[k] - rb[k] * sine[k]);
          put(dr + half, rb[k] * cosine[k] + ra[k] * sine[k]);
        }
      }
      if (half > 32) {   // wider rope keys
        for (int k = 0; k < kHeldRows; ++k) {
          const int64_t t = base + r0 + k - row.lo;
          if (mine(k)) append_rope<TI, TR>(p, freq_s, b, t, base + r0 + k, row.pos0 + t, lane + 32);
        }
      }
    }
    // A token's value is x inv g.  Its largest magnitude is taken as inv
    // max |x g| (half a unit in the last place of the exact one either way, as
    // the values themselves), in one walk with the sum of squares.
    float inv[kHeldRows], amax[kHeldRows], sum[kHeldRows];
#pragma unroll
    for (int k = 0; k < kHeldRows; ++k) inv[k] = 1.f, amax[k] = 0.f, sum[k] = 0.f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (!live[c]) continue;
      float2 w[4];
      if constexpr (kNorm) g[c].get(w);
#pragma unroll
      for (int k = 0; k < kHeldRows; ++k) {
        if (!mine(k)) continue;
        float2 v[4], sq = make_float2(0.f, 0.f);
        raw[k][c].get(v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 x = v[j];
          if constexpr (kNorm) {
            sq = fma_f32x2(x, x, sq);
            x = tc::mul_f32x2(x, w[j]);
          }
          amax[k] = tc::fmax3(amax[k], fabsf(x.x), fabsf(x.y));
        }
        sum[k] += sq.x + sq.y;
      }
    }
    if constexpr (kNorm) {
      warp_sum4(sum);
#pragma unroll
      for (int k = 0; k < kHeldRows; ++k) inv[k] = rsqrtf(sum[k] / (float)p.rank + p.eps);
    }
#pragma unroll
    for (int k = 0; k < kHeldRows; ++k) {
      // (non-negative: ordered as integers)
      amax[k] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax[k])));
      // NaN sets no unit: a token with a NaN or infinite element, or of zeros at eps = 0, has no finite inv.
      if constexpr (kNorm) amax[k] = fmaxf(amax[k] * inv[k], 0.f);
      if (!warp_blocks && lane == 0 && mine(k)) atomicMax(&amax_s[(r0 + k) >> p.block_shift], __float_as_uint(amax[k]));
    }
    if (warp_blocks) {
      // lane k: block k of the warp's rows
      if (lane < kHeldRows >> p.block_shift) {
        const int k_lo = lane << p.block_shift;
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < kHeldRows; ++k)
          if (k >= k_lo && k < k_lo + block) m = fmaxf(m, amax[k]);
        const int bk = (r0 + k_lo) >> p.block_shift;
        if (r0 + k_lo + block > r_lo && r0 + k_lo < r_hi) {
          int old;
          exp_s[bk] = block_exponent<kNorm>(p, row, scales, base, bk, m, old);
          if (bk == (r_lo >> p.block_shift)) old_s = old;
        }
      }
      __syncwarp();
    } else {
      __syncthreads();
      for (int k = threadIdx.x; k < n_blocks; k += kHeldWarps * 32) {
        const int k_lo = k << p.block_shift;
        if (k_lo + block <= r_lo || k_lo >= r_hi) continue;
        int old;
        exp_s[k] = block_exponent<kNorm>(p, row, scales, base, k, __uint_as_float(amax_s[k]), old);
        if (k == (r_lo >> p.block_shift)) old_s = old;
      }
      __syncthreads();
    }
    // in units: (x inv) g 2^(127 - e), the power of two taken with inv: exact, but
    // that the product of a finite inv stays finite.  (It passes f32's range for
    // tokens below 2^-65 at eps = 0 whose weights are so small, or 0, that the
    // block takes one of the smallest units: a weight of 0 must give 0, and
    // values of at most 2^-45 may be coded smaller than they are.)
#pragma unroll
    for (int k = 0; k < kHeldRows; ++k) {
      if (!mine(k)) continue;
      const float units = inv[k] * inverse_unit_of(exp_s[(r0 + k) >> p.block_shift]);
      inv[k] = kNorm && fabsf(inv[k]) <= FLT_MAX ? fminf(units, FLT_MAX) : units;
    }
    uint8_t* dst = codes + (base + r0) * p.codes_row_stride + 8 * lane;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (!live[c]) continue;
      float2 w[4];
      if constexpr (kNorm) g[c].get(w);
#pragma unroll
      for (int k = 0; k < kHeldRows; ++k) {
        if (!mine(k)) continue;
        float2 v[4];
        raw[k][c].get(v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = tc::mul_f32x2(v[j], make_float2(inv[k], inv[k]));
          if constexpr (kNorm) v[j] = tc::mul_f32x2(v[j], w[j]);
        }
        const float x[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
        *reinterpret_cast<uint2*>(dst + k * p.codes_row_stride + 256 * c) = encode8(x);
      }
    }
    if constexpr (kNorm) {
      // tokens that the first block held before: their codes move to the larger unit
      __syncthreads();
      const int k0 = r_lo >> p.block_shift, old = old_s, e = exp_s[k0];
      if (old >= 0 && clamp_exponent(old) != e)
        move_codes<kHeldWarps * 32>(p, codes, max(base + ((int64_t)k0 << p.block_shift), (int64_t)row.start), row.lo, old, e);
    }
    __syncthreads();   // the tile's shared state is read before the next one overwrites it
  }
  if constexpr (kNorm) {
    // one CTA per row: every thread has read the length before it may be overwritten
    if (p.lengths_here && blockIdx.x == 0) {
      __syncthreads();
      if (threadIdx.x == 0) p.kv_len_out[b] = row.ok ? row.len + p.s_new : row.len;
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// kNorm: new tokens of an append (normalised, weighted, with their rope key);
// otherwise the tokens of each row's window of a latent buffer.
template <bool kNorm, bool kVec, typename TI, typename TR>
__global__ void __launch_bounds__(kWarps * 32) encode_walk_kernel(const __grid_constant__ EncodeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ uint32_t amax_s[kMaxScaleBlock];   // per block of the tile, f32 bits (non-negative: ordered as integers)
  __shared__ int exp_s[kMaxScaleBlock], old_exp_s[kMaxScaleBlock];
  __shared__ float inv_s[kMaxScaleBlock];       // per row of the tile
  __shared__ float freq_s[kNorm ? kMaxRotaryDims / 2 : 1];
  const int b = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const EncodeRow<kNorm> row_of(p, b, blockIdx.x == 0 && threadIdx.x == 0);
  if constexpr (kNorm) {
    if ((int)threadIdx.x < p.rope_dim >> 1) freq_s[threadIdx.x] = p.inv_freq[threadIdx.x];   // (read behind the tile's barriers)
  }
  const int64_t lo = row_of.lo, hi = row_of.hi;
  const int block = 1 << p.block_shift;
  const int tile_rows = p.tile_rows;
  const int64_t tile0 = lo / tile_rows;
  const int64_t n_tiles = row_of.tiles(tile_rows);
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
      exp_s[k] = block_exponent<kNorm>(p, row_of, scales, base, k, __uint_as_float(amax_s[k]), old_exp_s[k]);
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
          *reinterpret_cast<uint2*>(dst + i) = encode8(x);
        } else {
          dst[i] = encode_e4m3(x[0]);
        }
      });
      if constexpr (kNorm) {
        append_rope<TI, TR>(p, freq_s, b, base + r - lo, base + r, row_of.pos0 + (base + r - lo), lane);
      }
    }
    if constexpr (kNorm) {
      // tokens that the first block held before: their codes move to the larger unit
      const int k0 = r_lo >> p.block_shift, old = old_exp_s[k0], e = exp_s[k0];
      if (old >= 0 && clamp_exponent(old) != e)
        move_codes<kWarps * 32>(p, codes, max(base + ((int64_t)k0 << p.block_shift), (int64_t)row_of.start), lo, old, e);
    }
    __syncthreads();   // the tile's shared state is read before the next one overwrites it
  }
  if constexpr (kNorm) {
    // one CTA per row: every thread has read the length before it may be overwritten
    if (p.lengths_here && blockIdx.x == 0) {
      __syncthreads();
      if (threadIdx.x == 0) p.kv_len_out[b] = row_of.ok ? row_of.len + p.s_new : row_of.len;
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

bool held_shape(const EncodeParams& p, bool vec) { return vec && p.rank <= kHeldRank; }
int tile_rows_of(const EncodeParams& p, bool vec) {
  if (held_shape(p, vec)) return kHeldTile;
  return (1 << p.block_shift) > kMinTileRows ? (1 << p.block_shift) : kMinTileRows;
}

template <bool kNorm, typename TI, typename TR>
cudaError_t launch_encode_t(const EncodeParams& p, bool vec, dim3 grid, cudaStream_t stream) {
  const dim3 held(kHeldWarps * 32), walk(kWarps * 32);
  if (held_shape(p, vec)) return launch_pdl(encode_kernel<kNorm, TI, TR>, grid, held, 0, stream, p);
  return vec ? launch_pdl(encode_walk_kernel<kNorm, true, TI, TR>, grid, walk, 0, stream, p)
             : launch_pdl(encode_walk_kernel<kNorm, false, TI, TR>, grid, walk, 0, stream, p);
}

}  // namespace

cudaError_t launch_append_q8(const EncodeParams& p_in, int in_dtype, int rope_dtype, bool vec, cudaStream_t stream) {
  EncodeParams p = p_in;
  p.tile_rows = tile_rows_of(p, vec);
  // Tiles that s_new rows can touch.  Up to two are walked by one CTA per row (a
  // decode step's append); more are spread over CTAs.  The new lengths are
  // written by the row's first CTA unless they may overwrite the lengths or
  // offsets that other CTAs of the row still have to read: then by a launch of
  // their own.
  const int64_t tiles = ((int64_t)p.s_new + p.tile_rows - 2) / p.tile_rows + 1;
  const unsigned gx = tiles <= 2 ? 1u : (unsigned)(tiles < 65535 ? tiles : 65535);
  auto apart = [&](const int32_t* x) { return !x || p.kv_len_out + p.batch <= x || x + p.batch <= p.kv_len_out; };
  p.lengths_here = p.kv_len_out != nullptr && (gx == 1 || (apart(p.kv_len) && apart(p.row_offsets)));
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
  p.tile_rows = tile_rows_of(p, vec);
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
