// beam_lds.h -- what a wave of beam search's selection keeps in LDS (no GPU code: the
// tests look at it on the CPU).
#pragma once

#include <cstddef>
#include <cstdint>

namespace ckhip {

constexpr int kBeamMaxK = 32;
constexpr int kBeamV = 8;        // logits a lane and access
constexpr int kBeamPacks = 8;    // accesses of a wave
constexpr size_t kBeamLdsAlign = 16;  // of a wave's share: candidates are written by 16 bytes

// For K beams, in this order: candidates' logits, the keys above the limit, those at it,
// and the candidates' places.
struct BeamLds {
  int packs;       // lanes' accesses with a logit at the limit or above
  int above;       // keys above it
  size_t above_at, level_at, places_at;  // bytes (the logits come first)
  size_t bytes;    // a multiple of kBeamLdsAlign, so that every wave's share begins aligned
  constexpr explicit BeamLds(int K)
      : packs((K - 1) * kBeamPacks + K), above((K - 1) * kBeamPacks * kBeamV),
        above_at((size_t)packs * kBeamV * sizeof(float)),
        level_at(above_at + (size_t)above * sizeof(uint64_t)),
        places_at(level_at + (size_t)K * sizeof(uint64_t)),
        bytes((places_at + (size_t)packs * sizeof(int) + kBeamLdsAlign - 1) &
              ~(kBeamLdsAlign - 1)) {}
};

constexpr bool beam_lds_aligned() {
  for (int K = 1; K <= kBeamMaxK; ++K) {
    const BeamLds l(K);
    if (l.bytes % kBeamLdsAlign || l.above_at % sizeof(uint64_t) || l.level_at % sizeof(uint64_t) ||
        l.places_at % sizeof(int))
      return false;
  }
  return true;
}
static_assert(beam_lds_aligned());

}  // namespace ckhip
