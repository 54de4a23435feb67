// The loop of a workgroup over its tiles, without anything of the GPU's, so that a
// program on the host can run it too.
#pragma once

#include <type_traits>

namespace moe {

// Calls body(height, it, nx) for tile after tile from `first` on, by the height of each
// in blocks of 64 rows, as a constant up to HIGH (1, 2 or 4).  body asks for the tile
// after it in its own time, and returns whether there is one; then it has set nx.
// Where there is none, nx is not looked at.
template <int HIGH, class ITEM, class BODY>
constexpr void walk_tiles(const ITEM &first, BODY body) {
  ITEM it = first;
  for (;;) {
    ITEM nx{};
    if (it.blocks == 1) {
      if (!body(std::integral_constant<int, 1>{}, it, nx)) return;
      it = nx;
    }
    if constexpr (HIGH >= 2) {
      if (it.blocks == 2) {
        if (!body(std::integral_constant<int, 2>{}, it, nx)) return;
        it = nx;
      }
    }
    if constexpr (HIGH >= 4) {
      if (it.blocks == 3) {
        if (!body(std::integral_constant<int, 3>{}, it, nx)) return;
        it = nx;
      }
      if (it.blocks == 4) {
        if (!body(std::integral_constant<int, 4>{}, it, nx)) return;
        it = nx;
      }
    }
    if (it.blocks < 1 || it.blocks > HIGH) return;
  }
}

}  // namespace moe
