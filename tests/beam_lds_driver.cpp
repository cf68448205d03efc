// CPU driver for the layout of a selecting wave's LDS: prints, for each number of beams,
// the sizes and places (bytes) of its lists.
#include <cstdio>

#include "beam_lds.h"

int main() {
  for (int K = 1; K <= ckhip::kBeamMaxK; ++K) {
    const ckhip::BeamLds l(K);
    std::printf("%d %d %d %zu %zu %zu %zu\n", K, l.packs, l.above, l.above_at, l.level_at,
                l.places_at, l.bytes);
  }
  return 0;
}
