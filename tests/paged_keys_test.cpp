// Host test of csrc/paged.cuh: the keys that new tokens see, against brute force.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <vector>

#define __device__
#define __forceinline__ inline
#define __clzll(x) __builtin_clzll((unsigned long long)(x))
using std::min;
#include "paged.cuh"

using namespace mla;

static bool node_seen(const std::vector<uint64_t>& m, int j) { return j >= 0 && j < 64 * (int)m.size() && (m[j >> 6] >> (j & 63) & 1); }

int main() {
  srand(1);
  for (int trial = 0; trial < 200000; ++trial) {
    const int s_q = 1 + rand() % (trial % 3 ? 200 : 4), words = (s_q + 63) / 64;
    const int count = trial % 5 ? s_q : rand() % (s_q + 1), len = rand() % 500, i = rand() % s_q;
    const bool tree = trial & 1;
    std::vector<uint64_t> m(words);
    for (auto& w : m)
      for (int k = 0; k < 64; ++k) w |= (uint64_t)(rand() % (trial % 7 ? 3 : 40) == 0) << k;   // bits behind count too
    if (trial % 11 == 0) std::fill(m.begin(), m.end(), 0);
    const int first = len - count;
    auto sees = [&](int t) {   // the definition
      if (i >= count || t < 0 || t >= len) return false;
      if (!tree) return t <= first + i;
      return t < first || (t - first < count && node_seen(m, t - first));
    };
    const uint64_t* mask = tree ? m.data() : nullptr;
    const int limit = paged_limit(len, count, i, mask, words);
    int top = 0;
    for (int t = 0; t < len; ++t)
      if (sees(t)) top = t + 1;
    // a token whose mask is empty may keep the whole prefix: limit is the smallest bound of that form
    if (limit != top) return printf("limit %d != %d (tree %d len %d count %d i %d)\n", limit, top, tree, len, count, i), 1;
    if (tree && tree_top(mask, words, count) > count) return puts("top"), 1;
    for (int base = 0; base < len + 64; base += 64) {
      const uint64_t seen = paged_seen(base, limit, first, mask, words);
      for (int k = 0; k < 64; ++k)
        if ((bool)(seen >> k & 1) != sees(base + k))
          return printf("key %d of tree %d len %d count %d i %d\n", base + k, tree, len, count, i), 1;
    }
  }
  const int32_t counts[] = {0, 3, 4, 5, -1};
  const int want[] = {0, 3, 4, -1, -1};
  for (int b = 0; b < 5; ++b)
    if (paged_count(counts, b, 4) != want[b]) return puts("count"), 1;
  if (paged_count(nullptr, 7, 9) != 9) return puts("count"), 1;
  puts("ok");
}
