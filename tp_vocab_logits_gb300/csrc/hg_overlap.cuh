// Whether arrays of a call share memory (host side of the norm and the beam search).
#pragma once

#include <cstddef>
#include <cstdint>

namespace hg {

// Rows of `width` bytes, `distance` apart; rows of one block do not overlap.
struct Block {
  const void* p = nullptr;  // null: no memory
  size_t rows = 0, distance = 0, width = 0;
  Block() = default;
  Block(const void* p, size_t rows, size_t distance, size_t width)
      : p(rows && width ? p : nullptr), rows(rows), distance(distance), width(width) {}
  Block(const void* p, size_t bytes) : Block(p, 1, bytes, bytes) {}
};

// Blocks side by side in one buffer (columns of wider rows) do not overlap. All sizes together
// are below 2^62 bytes.
inline bool overlap(const Block& a, const Block& b) {
  if (!a.p || !b.p) return false;
  typedef long long ll;
  const ll wa = (ll)a.width, wb = (ll)b.width, da = (ll)a.distance, db = (ll)b.distance;
  const ll ra = (ll)a.rows, rb = (ll)b.rows;
  const ll apart = (ll)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
  if (apart >= (ra - 1) * da + wa || -apart >= (rb - 1) * db + wb) return false;
  if (da == db && da > 0) {
    // Row j of b lies apart + (j - i) * da bytes behind row i of a: the least j - i at which it
    // does not end before that begins.
    const ll reach = -wb - apart;
    ll m = reach >= 0 ? reach / da + 1 : -((-reach - 1) / da);
    if (m < 1 - ra) m = 1 - ra;
    return m < rb && apart + m * da < wa;
  }
  for (ll i = 0, j = 0;;) {
    const ll gap = apart + j * db - i * da;  // from row i of a to row j of b
    if (gap >= wa) {
      if (ra == 1 || (i += (gap - wa) / da + 1) >= ra) return false;
    } else if (-gap >= wb) {
      if (rb == 1 || (j += (-gap - wb) / db + 1) >= rb) return false;
    } else {
      return true;
    }
  }
}

// What a call writes, the first `outs`, overlaps neither each other nor the rest.
template <int N>
bool apart(const Block (&a)[N], int outs) {
  for (int i = 0; i < outs; ++i)
    for (int j = i + 1; j < N; ++j)
      if (overlap(a[i], a[j])) return false;
  return true;
}

}  // namespace hg
