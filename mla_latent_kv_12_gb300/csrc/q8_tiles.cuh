// Tiles of an 8-bit cache as the fp16 operand tiles of tcgen05 MMAs: fetch of
// the codes and exponents of 64 keys, and their fp16 values in the swizzled
// shared-memory layout that a TMA load of a bf16 cache would leave.  (Rope keys
// need no conversion: the kernels load those of whole tiles by TMA.)
//
// The fetch runs two tiles ahead: every warp copies its own 16-byte pieces
// with cp.async into one of two slots of its own, so nothing but its own
// wait_group lies between the copy and the conversion, and a window and a
// selection are the same work.  (Codes fetched into registers a tile ahead took
// 220 us on a ragged decode of 32 rows, 498,051 keys, against 165 then: the
// fence that publishes a tile also waits for the loads in flight.)
//
// kLanes lanes (16 or 32) take one key and kThreads threads take 64 / kIters
// keys at once: piece i of a thread belongs to key i * kStep + key0.  Lane c
// copies the key's codes 16c .. 16c + 15, and decodes the eight codes from 8c
// on and the eight from 8 (kLanes + c) on: two 16-byte pieces of fp16, c % 8
// of boxes c / 8 and (kLanes + c) / 8, so that every eight lanes of a load or a
// store cover all banks.  (Sixteen neighbouring codes per lane cost 128 more
// shared-memory wavefronts per tile.)
// kStep is a multiple of 8, so a thread's place in the 128-byte swizzle (piece
// ^ (row % 8)) is fixed.
#pragma once

#include "e4m3.cuh"
#include "tc_common.cuh"

namespace mla {

constexpr int kTileKeys = 64;

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

template <int kLanes, int kThreads>
struct Q8Fetch {
  static constexpr int kStep = kThreads / kLanes;         // keys taken at once
  static constexpr int kIters = kTileKeys / kStep;        // pieces of codes per thread and tile
  static constexpr int kPieceBytes = 16 * kThreads;
  static constexpr int kSlotBytes = kIters * kPieceBytes;
  static_assert(kStep % 8 == 0 && kIters >= 4 && kIters <= 8, "fixed swizzle; lanes to look the keys up");
  uint32_t slot0;                // shared address of this thread's first piece
  uint32_t codes0;               // and of the codes that it decodes
  int key0;                      // key of piece i is i * kStep + key0
  int rope_group;                // this thread's rope piece belongs to its key rope_group
  int peers;                     // first lane of the lanes that share this lane's keys
  int mine;                      // piece whose position and exponent this lane looks up (lane % kIters)

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
    return position(r, tile * kTileKeys + kStep * mine + key0);
  }
  // Exponent byte of the key at `pos` (any value for no key).
  __device__ __forceinline__ int my_exponent(const Q8Rows& r, int pos) const {
    return pos >= 0 ? __ldg(r.scales + (((int64_t)r.start + pos) >> r.shift)) : kMinExponent;
  }
  // Flags a unit in which fp16 loses bits (the smallest one is that of zeros).
  __device__ __forceinline__ void check_exponent(int32_t* status, int e) const {
    if (e < kMinExponentF16 && e > kMinExponent && status) atomicOr(status, MLA_DEVICE_VALUE_RANGE);
  }
  // Copies of a window tile's codes into slot s: rows at one distance, zeros past the entries.
  __device__ __forceinline__ void issue_window(const Q8Rows& r, int tile, int s) const {
    const int e0 = tile * kTileKeys + key0;
    const uint8_t* c = r.codes + ((int64_t)r.start + e0) * r.codes_stride;
    const uint32_t dst = slot0 + s * kSlotBytes;
#pragma unroll
    for (int i = 0; i < kIters; ++i, c += kStep * r.codes_stride) {
      const bool in = e0 + i * kStep < r.entries;
      tc::cp_async_16(dst + i * kPieceBytes, in ? c : r.codes, in ? 16u : 0u);
    }
  }
  // Copies of one tile's codes into slot s; `pos` from my_position.
  __device__ __forceinline__ void issue_codes(const Q8Rows& r, int s, int pos) const {
    const uint32_t dst = slot0 + s * kSlotBytes;
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const int p = __shfl_sync(0xffffffffu, pos, peers + i);
      tc::cp_async_16(dst + i * kPieceBytes, r.codes + (int64_t)(r.start + max(p, 0)) * r.codes_stride, p >= 0 ? 16u : 0u);
    }
  }
  // This thread's rope piece of one tile (one per thread), zeros for no key.
  __device__ __forceinline__ uint4 load_rope(const Q8Rows& r, int pos) const {
    static_assert(kIters == 4, "one piece per thread");
    const int p = __shfl_sync(0xffffffffu, pos, peers + rope_group);
    return p >= 0 ? __ldg(reinterpret_cast<const uint4*>(r.rope + (int64_t)(r.start + p) * r.rope_stride)) : make_uint4(0, 0, 0, 0);
  }
  // Slot s as fp16 values: this lane's first eight dims at shared address `box`,
  // the others kBox bytes behind, rows 128 bytes apart.  `exponent` from
  // my_exponent.
  template <int kBox>
  __device__ __forceinline__ void convert(int s, int exponent, uint32_t box) const {
    const uint32_t src0 = codes0 + s * kSlotBytes, src1 = src0 + 8 * kLanes;
    const uint32_t unit = f16_unit(clamp_exponent(exponent));
    __syncwarp();   // the warp's copies have landed (each lane has waited for its own)
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const uint32_t mul2 = __shfl_sync(0xffffffffu, unit, peers + i);
      const uint2 c0 = ld_shared_8(src0 + i * kPieceBytes), c1 = ld_shared_8(src1 + i * kPieceBytes);
      uint32_t v[4];
      decode_e4m3x8_f16(c0, mul2, v);
      st_shared_16(box + i * kStep * 128, make_uint4(v[0], v[1], v[2], v[3]));
      decode_e4m3x8_f16(c1, mul2, v);
      st_shared_16(box + kBox + i * kStep * 128, make_uint4(v[0], v[1], v[2], v[3]));
    }
  }

  static __device__ __forceinline__ uint2 ld_shared_8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
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
