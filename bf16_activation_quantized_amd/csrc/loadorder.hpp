// Counts of loads in flight in a ring of LDS stages (plain C++, checked at compile
// time). A wave's loads land in the order of their requests, so waiting until at
// most n of them are in flight leaves the youngest n.
#pragma once

namespace w4a16 {

// A ring of NS stages. Ahead of the loop stages 0 .. NS - 2 are requested, one after
// the other, each with at least `parts` loads of a wave and, from stage `worded` on,
// one more (the scale word of a later stage); then stages 0 and 1 have to be there.
// Step j requests stage j + NS - 1 with such a word, and at its end stage j + 2 has to
// be there. Whether waits for at most `start` and `step` loads in flight see to that,
// at every step, wherever among its stage's loads a word stands.
constexpr bool ring_waits_hold(int NS, int parts, int worded, int start, int step) {
  // loads requested behind those of stage s, once stage `last` was
  const auto younger = [&](int s, int last) {
    int n = 0;
    for (int i = s + 1; i <= last; ++i) n += parts + (i >= worded || i >= NS - 1 ? 1 : 0);
    return n;
  };
  if (start > younger(1, NS - 2)) return false;
  for (int j = 0; j <= 2 * NS; ++j)
    if (step > younger(j + 2, j + NS - 1)) return false;
  return true;
}

}  // namespace w4a16
