// Linear attention's segments and slots for any offsets (linear.h): every segment of a sequence
// that has several lies in the plan's slots, in order and disjoint where the offsets rise.
#include <algorithm>
#include <climits>
#include <cstdio>
#include <random>
#include <vector>

#include "delta.h"
#include "linear.h"

#define CHECK(c)                                                        \
  do {                                                                  \
    if (!(c)) {                                                         \
      std::fprintf(stderr, "check failed line %d: %s\n", __LINE__, #c); \
      return 1;                                                         \
    }                                                                   \
  } while (0)

namespace s4 {
s4dplr_status hip_failure(hipError_t) { return S4DPLR_ERR_HIP; }
hipError_t launch_linear_steps(const LinStep&, int, hipStream_t) { return hipSuccess; }
hipError_t launch_linear_sums(const LinPass&, int, hipStream_t) { return hipSuccess; }
hipError_t launch_linear_pass(const LinPass&, int, hipStream_t) { return hipSuccess; }
hipError_t launch_linear_gates(const LinGates&, hipStream_t) { return hipSuccess; }
hipError_t launch_linear_groups(const LinGroups&, int, hipStream_t) { return hipSuccess; }
int linear_parts(int, int, int) { return 4; }
}  // namespace s4

static int check(long tokens, const std::vector<int>& offsets, int Hv) {
  const int S = (int)offsets.size() - 1;
  s4dplr_linear_attention_plan* p = nullptr;
  CHECK(s4dplr_linear_attention_plan_create(&p, S, tokens, 1, Hv, 8, 8, S4DPLR_BF16, 1) == S4DPLR_OK);
  CHECK(p->segment > 0 && p->segment % s4::kLinChunk == 0);
  bool rises = offsets[0] >= 0 && offsets[S] <= tokens;
  for (int s = 0; s < S; ++s) rises = rises && offsets[s] <= offsets[s + 1];
  long next = 0;
  for (int s = 0; s < S; ++s) {
    const s4::Rows c = s4::clamp_rows((int)tokens, offsets[s], offsets[s + 1]);
    const s4::LinRows r{c.start, c.len};
    if (r.len <= p->segment) continue;
    const long first = r.slot(s, p->segment), n = r.segments(p->segment);
    CHECK(first >= 0 && first + n <= p->slots);
    CHECK((n - 1) * p->segment < r.len && n * p->segment >= r.len);
    if (rises) {
      CHECK(first >= next);
      // the search for a slot's sequence: the last whose first slot is at most it
      for (int t = s + 1; t < S; ++t) {
        const s4::Rows d = s4::clamp_rows((int)tokens, offsets[t], offsets[t + 1]);
        CHECK((s4::LinRows{d.start, d.len}.slot(t, p->segment) >= first + n));
      }
    }
    next = first + n;
  }
  s4dplr_linear_attention_plan_destroy(p);
  return 0;
}

int main() {
  const int bad[] = {INT_MIN, INT_MIN + 1, INT_MIN + 200, -5, -1, 0, 1, 255, 256, 257, 2000, 2001, INT_MAX - 1, INT_MAX};
  for (int a : bad)
    for (int b : bad)
      for (int c : bad)
        if (check(2000, {a, b, c, b, 2000}, 1)) return 1;
  std::mt19937 gen(1);
  for (int i = 0; i < 20000; ++i) {
    const long tokens = gen() % 9000;
    const int S = 1 + (int)(gen() % 40), top = gen() % 3 ? 4 : 900, Hv = gen() % 4 ? 1 : 600;
    std::vector<int> o{(int)(gen() % 3)};
    for (int s = 0; s < S; ++s)
      o.push_back(o.back() + (int)(gen() % 5 == 0 ? 256 * (gen() % 4) + gen() % 3 : gen() % (gen() % 8 ? top : 4 * top + 20)));
    if (check(std::max<long>(tokens, o.back()), o, Hv)) return 1;
    if (check(tokens, o, Hv)) return 1;   // some end behind the last row
    o[gen() % o.size()] = (int)gen();
    if (check(tokens, o, Hv)) return 1;
  }
  std::puts("ok");
  return 0;
}
