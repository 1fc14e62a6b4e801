// Tiles of an 8-bit cache as the bf16 operand tiles of tcgen05 MMAs: fetch of
// the codes, exponents and rope keys of 64 keys, and their bf16 values in the
// swizzled shared-memory layout that a TMA load of a bf16 cache would leave.
//
// The fetch runs two tiles ahead: every thread copies its own 16-byte pieces
// with cp.async into one of two private slots (10 pieces: eight of codes, two
// of rope keys), so nothing but its own wait_group lies between the copy and
// the conversion, and a window and a selection are the same work.  The loops
// are rolled: with eight pieces unrolled beside the softmax's code the
// instruction cache missed on most of them (a ragged decode of 32 rows took
// 398 us that way).
//
// kLanes lanes (16 or 32) take one key, 16 dims each; a group of warps takes
// eight keys at once: piece i of a thread belongs to key 8i + key0.  Keys of
// one thread differ by multiples of 8, so its place in the 128-byte swizzle
// (piece ^ (row % 8)) is fixed.
#pragma once

#include "e4m3.cuh"
#include "tc_common.cuh"

namespace mla {

constexpr int kTileKeys = 64;
constexpr int kPieces = 10;   // 16-byte pieces per thread and slot

// The cache row range of a pass, with the pointers moved to this thread's pieces.
struct Q8Rows {
  const uint8_t* codes;          // + 16 * (lane % kLanes), first dim of the CTA
  int64_t codes_stride;
  const uint8_t* scales;
  int shift;
  const __nv_bfloat16* rope;     // + 8 * rope piece
  int64_t rope_stride;
  int start;                     // buffer row of window position 0
  int entries, limit;            // entries of the pass's key list; visible window length
  const int32_t* list;           // selected positions, or NULL: entry e is position e
  int32_t* status;               // non-NULL: flag positions outside the window
};

template <int kLanes>
struct Q8Fetch {
  uint32_t slot0;                // shared address of this thread's first piece
  uint32_t slot_bytes, piece_bytes;
  int key0;                      // key of piece i is 8i + key0
  int rope_group;                // rope pieces belong to this thread's keys rope_group and rope_group + 4
  int peers;                     // first lane of the lanes that share this lane's keys
  int mine;                      // piece whose position and exponent this lane looks up (lane % 8)

  // Window position of entry e, -1 for none (past the entries, or outside the window: skipped and flagged).
  __device__ __forceinline__ int position(const Q8Rows& r, int e) const {
    if (e >= r.entries) return -1;
    if (!r.list) return e;
    const int p = __ldg(r.list + e);
    if (p >= 0 && p < r.limit) return p;
    if (r.status) atomicOr(r.status, MLA_DEVICE_INDEX_OUT_OF_RANGE);
    return -1;
  }
  __device__ __forceinline__ int my_position(const Q8Rows& r, int tile) const {
    return position(r, tile * kTileKeys + 8 * mine + key0);
  }
  // Exponent byte of the key at `pos` (any value for no key).
  __device__ __forceinline__ int my_exponent(const Q8Rows& r, int pos) const {
    return pos >= 0 ? __ldg(r.scales + (((int64_t)r.start + pos) >> r.shift)) : kMinExponent;
  }
  // Copies of one tile into slot s; `pos` from my_position.
  __device__ __forceinline__ void issue(const Q8Rows& r, int s, int pos) const {
    const uint32_t dst = slot0 + s * slot_bytes;
#pragma unroll 2
    for (int i = 0; i < 8; ++i) {
      const int p = __shfl_sync(0xffffffffu, pos, peers + i);
      tc::cp_async_16(dst + i * piece_bytes, r.codes + (int64_t)(r.start + max(p, 0)) * r.codes_stride, p >= 0 ? 16u : 0u);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int p = __shfl_sync(0xffffffffu, pos, peers + 4 * j + rope_group);
      tc::cp_async_16(dst + (8 + j) * piece_bytes, r.rope + (int64_t)(r.start + max(p, 0)) * r.rope_stride,
                      p >= 0 ? 16u : 0u);
    }
  }
  // Slot s as bf16 values: box `box0` / `box1` receive dims 0..7 and 8..15 of
  // the thread's 16 (shared addresses for key0; keys 8 apart lie 1024 bytes
  // apart), `rope0` / `rope1` the rope pieces.  `exponent` from my_exponent.
  __device__ __forceinline__ void convert(int s, int exponent, uint32_t box0, uint32_t box1, uint32_t rope0,
                                          uint32_t rope1, bool swap) const {
    const uint32_t src = slot0 + s * slot_bytes;
    const uint32_t unit = bf16_unit(clamp_exponent(exponent));
#pragma unroll 2
    for (int i = 0; i < 8; ++i) {
      const uint32_t mul2 = __shfl_sync(0xffffffffu, unit, peers + i);
      const uint4 c = ld_shared_16(src + i * piece_bytes);
      uint32_t v[8];
      const uint32_t nan = decode_e4m3x16(c, mul2, v);
      // half of the lanes store their second piece first (eight lanes, eight bank groups)
      st_shared_16(swap ? box1 : box0, swap ? make_uint4(v[4], v[5], v[6], v[7]) : make_uint4(v[0], v[1], v[2], v[3]));
      st_shared_16(swap ? box0 : box1, swap ? make_uint4(v[0], v[1], v[2], v[3]) : make_uint4(v[4], v[5], v[6], v[7]));
      if (nan) {
#pragma unroll 1
        for (int k = 0; k < 16; ++k) {
          uint32_t code;
          asm volatile("ld.shared.u8 %0, [%1];" : "=r"(code) : "r"(src + i * piece_bytes + k) : "memory");
          if ((code & 0x7Fu) == 0x7Fu) tc::st_shared_u16((k < 8 ? box0 : box1) + 2 * (k & 7), 0x7FC0u);
        }
      }
      box0 += 1024;
      box1 += 1024;
    }
    st_shared_16(rope0, ld_shared_16(src + 8 * piece_bytes));
    st_shared_16(rope1, ld_shared_16(src + 9 * piece_bytes));
  }

  static __device__ __forceinline__ uint4 ld_shared_16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
  }
  static __device__ __forceinline__ void st_shared_16(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
  }
};

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest `n` groups of this thread's copies have landed.
template <int n>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

}  // namespace mla
