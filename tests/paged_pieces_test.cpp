// Host test of csrc/pieces.cuh: where the pieces of split rows lie in the workspace, over random plans.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <set>
#include <vector>

#define __device__
#define __host__
#define __forceinline__ inline
#include "pieces.cuh"

using namespace mla;

int main() {
  srand(2);
  long cut = 0, most = 0;
  for (int trial = 0; trial < 20000; ++trial) {
    const int groups = 1 + rand() % (trial % 2 ? 76 : 9), units = 1 + rand() % (trial % 3 ? 200 : 2 * groups);
    const int charge = trial % 4 ? 0 : 7, min_tiles = trial % 5 ? 1 : 4;
    // units in a row, each a charge and its tiles (some without any), cut into equal ranges
    std::vector<int> tiles(units), begin(units), end(units);
    int total = 0;
    for (int u = 0; u < units; ++u) {
      tiles[u] = rand() % 4 ? rand() % (trial % 7 ? 40 : 400) : 0;
      begin[u] = total + (tiles[u] ? charge : 0);
      total = end[u] = begin[u] + tiles[u];
    }
    const int per = std::max(min_tiles, (total + groups - 1) / groups);
    std::set<int> places;
    for (int u = 0; u < units; ++u) {
      if (!tiles[u]) continue;
      const int first = begin[u] / per, last = (end[u] - 1) / per;
      if (last >= groups) return puts("more ranges than groups"), 1;
      if (first == last) continue;   // whole: no pieces
      for (int g = first; g <= last; ++g) {
        const int t0 = std::max(begin[u], g * per) - begin[u];   // the group's first tile of the unit
        const bool begins = t0 == 0;
        if (begins != (g == first)) return puts("the first piece"), 1;
        const int place = piece_place(few_units(units, groups), u, g, begins);
        if (place < 0 || place >= piece_places(units, groups)) return printf("place %d of %d\n", place, piece_places(units, groups)), 1;
        if (!places.insert(place).second) return printf("place %d twice (units %d groups %d)\n", place, units, groups), 1;
        ++cut;
      }
    }
    most = std::max(most, (long)places.size());
  }
  // what the workspace holds for rows in units of `width`: clusters and as many more, at most one a row
  for (int clusters : {74, 76})
    for (int width = 1; width <= 4; ++width)
      for (int rows = 1; rows < 400; ++rows)
        if (piece_places((rows + width - 1) / width, clusters / width) * width > piece_slots(rows, clusters))
          return printf("rows %d width %d\n", rows, width), 1;
  if (cut < 100000 || most < 76) return puts("too few pieces"), 1;
  puts("ok");
}
