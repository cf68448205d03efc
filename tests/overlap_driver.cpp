// CPU driver for csrc/overlap.h: reads two tensors a line (address, n0, s0, n1, s1, bytes
// of each) and prints whether they are found to share memory (bit 0), and to lie side by
// side (bit 1).
#include <cstdio>

#include "overlap.h"

int main() {
  long long v[12];
  for (;;) {
    for (int k = 0; k < 12; ++k)
      if (std::scanf("%lld", &v[k]) != 1) return k ? 2 : 0;
    ckhip::Pieces p[2];
    for (int k = 0; k < 2; ++k) {
      p[k].at = (uintptr_t)v[6 * k];
      p[k].n0 = v[6 * k + 1], p[k].s0 = v[6 * k + 2];
      p[k].n1 = v[6 * k + 3], p[k].s1 = v[6 * k + 4];
      p[k].bytes = v[6 * k + 5];
    }
    const auto a = ckhip::slice_of(p[0]), b = ckhip::slice_of(p[1]);
    const bool beside = a.at <= b.at ? ckhip::side_by_side(a, b) : ckhip::side_by_side(b, a);
    std::printf("%d\n", (ckhip::pieces_meet(p[0], p[1]) ? 1 : 0) | (beside ? 2 : 0));
  }
}
