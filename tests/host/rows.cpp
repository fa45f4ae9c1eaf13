// The gated delta rule's rows and slots for any offsets (delta.h): every sequence
// lies in the packed rows, its chunks in the plan's slots, and in order and disjoint
// where the offsets rise; for the two ways in which a call splits its sequences between
// the token by token and the chunked form.
#include <algorithm>
#include <climits>
#include <cstdio>
#include <random>
#include <vector>

#include "delta.h"

#define CHECK(c)                                                        \
  do {                                                                  \
    if (!(c)) {                                                         \
      std::fprintf(stderr, "check failed line %d: %s\n", __LINE__, #c); \
      return 1;                                                         \
    }                                                                   \
  } while (0)

static int check(long tokens, const std::vector<int>& offsets, unsigned flags) {
  const int S = (int)offsets.size() - 1;
  s4dplr_delta_plan* p = nullptr;
  CHECK(s4dplr_delta_plan_create(&p, S, tokens, 1, 1, 8, 8, S4DPLR_BF16, flags) == S4DPLR_OK);
  const int least = !flags && s4::packed_steps(p) ? s4::step_limit(p) + 1 : 1;
  bool rises = offsets[0] >= 0 && offsets[S] <= tokens;
  for (int s = 0; s < S; ++s) rises = rises && offsets[s] <= offsets[s + 1];
  long next = 0;
  for (int s = 0; s < S; ++s) {
    const s4::Rows r = s4::clamp_rows((int)tokens, offsets[s], offsets[s + 1]);
    CHECK(r.start >= 0 && r.len >= 0 && r.start + r.len <= tokens);
    if (rises) CHECK(r.start == offsets[s] && r.len == offsets[s + 1] - offsets[s]);
    if (r.len < least) continue;
    const long first = r.first(s, least);
    CHECK(first >= 0 && first + r.chunks() <= p->slots);
    if (rises) {
      CHECK(first >= next);
      // the search for a slot's sequence: the last that begins at or before it
      for (int t = s + 1; t < S; ++t)
        CHECK(s4::clamp_rows((int)tokens, offsets[t], offsets[t + 1]).first(t, least) >=
              first + r.chunks());
    }
    next = first + r.chunks();
  }
  s4dplr_delta_plan_destroy(p);
  return 0;
}

static int check(long tokens, const std::vector<int>& offsets) {
  return check(tokens, offsets, 0) || check(tokens, offsets, S4DPLR_DELTA_TRAINING);
}

int main() {
  const int bad[] = {INT_MIN, INT_MIN + 1, INT_MIN + 200, -5, -1, 0,
                     1,       63,          64,            199, 200, 201, INT_MAX - 1, INT_MAX};
  for (int a : bad)
    for (int b : bad)
      for (int c : bad)
        if (check(200, {a, b, c, b, 200})) return 1;
  std::mt19937 gen(1);
  for (int i = 0; i < 20000; ++i) {
    const long tokens = gen() % 700;
    const int S = 1 + (int)(gen() % 40), top = gen() % 3 ? 4 : 150;
    std::vector<int> o{(int)(gen() % 3)};
    for (int s = 0; s < S; ++s)   // some longer ones among many short
      o.push_back(o.back() + (int)(gen() % (gen() % 8 ? top : 4 * top + 20)));
    if (check(std::max<long>(tokens, o.back()), o)) return 1;
    if (check(tokens, o)) return 1;   // some end behind the last row
    o[gen() % o.size()] = (int)gen();
    if (check(tokens, o)) return 1;
  }
  std::puts("ok");
  return 0;
}
