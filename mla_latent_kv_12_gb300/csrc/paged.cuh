// What the kernels of the paged cache share: where a key of a sequence lies,
// and which keys a new token sees.
//
// Key t of batch row b is row t % page_size of page table[b, t / page_size].
// The row's last `count` keys are its new tokens (count = s_q, or counts[b]).
// In a row of drafted tokens, token i sees the keys up to its own; in a tree,
// the keys before the new tokens and the nodes j whose bit is set in its mask
// (64-bit words, node 0 the lowest bit of the first).
#pragma once

#include <stdint.h>

namespace mla {

// New tokens of row b, or -1 for a count that is not one.
__device__ __forceinline__ int paged_count(const int32_t* counts, int b, int s_q) {
  if (!counts) return s_q;
  const int c = counts[b];
  return c >= 0 && c <= s_q ? c : -1;
}

// One past the highest node below `count` in a token's mask (0: none).
__device__ __forceinline__ int tree_top(const uint64_t* mask, int words, int count) {
  for (int w = min(words, (count + 63) >> 6) - 1; w >= 0; --w) {
    uint64_t m = mask[w];
    if (count - 64 * w < 64) m &= (1ull << (count - 64 * w)) - 1ull;
    if (m) return 64 * w + 64 - __clzll((long long)m);
  }
  return 0;
}

// Keys [0, limit) hold all that token i sees of a row of `len` keys (in a tree some of them are not seen).
__device__ __forceinline__ int paged_limit(int len, int count, int i, const uint64_t* mask, int words) {
  if (i >= count) return 0;
  const int first = len - count;
  const int limit = first + (mask ? tree_top(mask, words, count) : i + 1);
  return limit > 0 ? limit : 0;
}

// Which of keys base .. base + 63 a token sees: those below `limit`, and in a
// tree (mask not null) from key `first` on those whose bit is set.
__device__ __forceinline__ uint64_t paged_seen(int base, int limit, int first, const uint64_t* mask, int words) {
  const int n = limit - base;
  uint64_t seen = n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1ull;
  if (mask && base + 64 > first) {
    const int off = base - first;   // node of key `base`
    uint64_t bits;
    if (off < 0) {
      bits = (mask[0] << -off) | ((1ull << -off) - 1ull);
    } else {
      const int w = off >> 6, s = off & 63;
      bits = w < words ? mask[w] >> s : 0ull;
      if (s && w + 1 < words) bits |= mask[w + 1] << (64 - s);
    }
    seen &= bits;
  }
  return seen;
}

}  // namespace mla
