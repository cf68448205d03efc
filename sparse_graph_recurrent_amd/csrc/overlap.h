// overlap.h -- whether two strided tensors share memory, by their addresses, sizes and
// strides (no GPU code: the tests look at it on the CPU).
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <utility>

namespace ckhip {

// n0 x n1 pieces of `bytes` adjacent bytes, s0 and s1 bytes apart.
struct Pieces {
  uintptr_t at = 0;
  int64_t n0 = 1, s0 = 0, n1 = 1, s1 = 0, bytes = 0;

  bool empty() const { return !at || n0 <= 0 || n1 <= 0 || bytes <= 0; }
  // One behind the last byte.  (Strides may be any: 64 bits would overflow.)
  __int128 end() const {
    return (__int128)at + (__int128)(n0 - 1) * s0 + (__int128)(n1 - 1) * s1 + bytes;
  }
};
inline Pieces range_of(const void* p, size_t bytes) {
  Pieces r;
  r.at = reinterpret_cast<uintptr_t>(p);
  r.bytes = (int64_t)bytes;
  return r;
}

namespace overlap {

typedef __int128 Wide;
inline Wide floor_div(Wide a, Wide b) { return a >= 0 ? a / b : -((b - 1 - a) / b); }

// Whether lo < at + i s0 + j s1 < hi for some i < n0, j < n1.
inline bool any_between(Wide at, Wide n0, Wide s0, Wide n1, Wide s1, Wide lo, Wide hi) {
  const auto row = [&](Wide from) {  // the first j past lo
    const Wide j = s1 ? std::max<Wide>(0, floor_div(lo - from, s1) + 1) : 0;
    return j < n1 && from + j * s1 > lo && from + j * s1 < hi;
  };
  if (!s0) return row(at);
  const Wide reach = (n1 - 1) * s1;
  const Wide first = std::max<Wide>(0, floor_div(lo - at - reach, s0) + 1);
  const Wide last = std::min<Wide>(n0 - 1, floor_div(hi - 1 - at, s0));
  const Wide past = std::max<Wide>(first, floor_div(lo - at, s0) + 1);  // begins past lo
  if (past <= last) return true;
  // (rows that begin before lo: one or two, but where rows lie within one another)
  constexpr int kMost = 4096;
  int looked = 0;
  for (Wide i = std::min(past - 1, last); i >= first && looked < kMost; --i, ++looked)
    if (row(at + i * s0)) return true;
  return false;
}

// The same bytes in as few levels as it takes, the longer stride first.
inline Pieces plain(Pieces p) {
  if (p.n0 == 1) p.s0 = 0;
  if (p.n1 == 1) p.s1 = 0;
  if (!p.s0) p.n0 = 1;
  if (!p.s1) p.n1 = 1;
  if (p.s0 < p.s1) std::swap(p.s0, p.s1), std::swap(p.n0, p.n1);
  const auto join = [&](int64_t& n, int64_t& s) {
    if (!s || s > p.bytes) return;
    p.bytes += (n - 1) * s;
    n = 1, s = 0;
  };
  join(p.n1, p.s1);
  if (!p.s1) join(p.n0, p.s0);
  return p;
}

inline bool solid_meets(const Pieces& a, const Pieces& solid) {
  return any_between(a.at, a.n0, a.s0, a.n1, a.s1, (Wide)solid.at - a.bytes,
                     (Wide)solid.at + solid.bytes);
}

}  // namespace overlap

// A tensor as a slice of a wider one's rows, for many comparisons: all its pieces begin at
// `at` and a multiple of `step` (0: no such step).
struct Slice {
  uintptr_t at, end;
  int64_t step, bytes;
};
inline Slice slice_of(const Pieces& whole) {
  const Pieces p = overlap::plain(whole);
  const __int128 end = p.end();
  return Slice{p.at, end > (__int128)UINTPTR_MAX ? UINTPTR_MAX : (uintptr_t)end,
               !p.s1 ? p.s0 : p.s0 % p.s1 ? 0 : p.s1, p.bytes};
}
// Whether two of them, b not before a, lie beside one another in the same rows.  (Quick;
// no other answer than yes says anything.)
inline bool side_by_side(const Slice& a, const Slice& b) {
  if (a.step != b.step || !a.step) return false;
  uintptr_t by = b.at - a.at;
  if (by >= (uintptr_t)a.step) by %= (uintptr_t)a.step;
  return by >= (uintptr_t)a.bytes && by + (uintptr_t)b.bytes <= (uintptr_t)a.step;
}

// Whether a byte lies in both.  Exact where one has no gaps, where both have the same
// strides (slices of one tensor) or where one has few pieces; of others with gaps only
// such are found as begin at the same address.
inline bool pieces_meet(const Pieces& x, const Pieces& y) {
  using namespace overlap;
  if (x.empty() || y.empty() || x.end() <= (Wide)y.at || y.end() <= (Wide)x.at) return false;
  Pieces a = plain(x), b = plain(y);
  if (a.at == b.at) return true;
  if (!b.s0) return solid_meets(a, b);
  if (!a.s0) return solid_meets(b, a);
  // a single level of one is the level of the other that has its stride
  const auto settle = [](Pieces& p, const Pieces& q) {
    if (p.s1) return;
    if (p.s0 == q.s1) p.n1 = p.n0, p.s1 = p.s0, p.n0 = 1, p.s0 = q.s0;
    else if (p.s0 == q.s0) p.s1 = q.s1;
  };
  settle(a, b);
  settle(b, a);
  if (a.s0 == b.s0 && a.s1 == b.s1)  // places of a's pieces as seen from b's
    return any_between((Wide)a.at - b.at - (Wide)(b.n0 - 1) * b.s0 - (Wide)(b.n1 - 1) * b.s1,
                       (Wide)a.n0 + b.n0 - 1, a.s0, (Wide)a.n1 + b.n1 - 1, a.s1,
                       -(Wide)a.bytes, b.bytes);
  constexpr int64_t kFew = 1024;
  if ((Wide)a.n0 * a.n1 < (Wide)b.n0 * b.n1) std::swap(a, b);
  if ((Wide)b.n0 * b.n1 > kFew) return false;
  for (int64_t i = 0; i < b.n0; ++i)
    for (int64_t j = 0; j < b.n1; ++j) {
      Pieces one;
      one.at = b.at + (uintptr_t)i * (uintptr_t)b.s0 + (uintptr_t)j * (uintptr_t)b.s1;
      one.bytes = b.bytes;
      if (solid_meets(a, one)) return true;
    }
  return false;
}

}  // namespace ckhip
