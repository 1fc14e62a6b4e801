// Where the attention over pages keeps the pieces of split rows.
#pragma once

namespace mla {

// The attention's work units (query rows, or a few in lockstep) are laid out one
// behind the other and cut into equal ranges, one per group of clusters.  A unit
// that a cut divides leaves a piece of each of its rows with every group it
// meets, at the group's place for it: of such units a group's range holds at
// most one that an earlier group begins (its first), and one that it begins
// itself (its last).  With no more units than groups fewer places do, counted
// along both: from a piece to the next the group or the unit goes up.
__host__ __device__ __forceinline__ bool few_units(int units, int groups) { return units <= groups; }
__host__ __device__ __forceinline__ int piece_place(bool few, int u, int g, bool begins) {
  return few ? u + g : 2 * g + (begins ? 1 : 0);
}
__host__ __device__ __forceinline__ int piece_places(int units, int groups) {
  return few_units(units, groups) ? units + groups - 1 : 2 * groups;
}
// Enough for the rows' pieces whatever the number of rows in a unit, which is
// that of the clusters in a group.
__host__ __device__ __forceinline__ int piece_slots(int rows, int clusters) {
  return clusters + (rows < clusters ? rows : clusters);
}

}  // namespace mla
