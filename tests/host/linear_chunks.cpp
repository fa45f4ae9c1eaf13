// Where the decays' gradient keeps the states before the chunks inside segments (linear.h): chunk
// boundaries of a plan's segments have places of their own within what the plan reserves, and the chunks as
// items of their own lie in the plan's slots.
#include <algorithm>
#include <cstdio>
#include <random>
#include <set>
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

static int check(long tokens, const std::vector<int>& offsets, int Hv, int dv, int dtype) {
  const int S = (int)offsets.size() - 1, chunk = s4::linear_chunk(dv, s4::linear_type_parts(dtype));
  s4dplr_linear_attention_plan* p = nullptr;
  CHECK(s4dplr_linear_attention_plan_create(&p, S, tokens, 1, Hv, 8, dv, dtype, 1) == S4DPLR_OK);
  CHECK(p->segment % chunk == 0);
  const size_t place = sizeof(float) * Hv * 4 * 16 * s4::linear_rows(dv), room = p->off_dgsum - p->off_inner;
  std::set<long> places;
  long next = 0;
  for (int s = 0; s < S; ++s) {
    const s4::Rows c = s4::clamp_rows((int)tokens, offsets[s], offsets[s + 1]);
    const s4::LinRows r{c.start, c.len};
    for (long m = 0; m < r.len; m += p->segment)
      for (long t = m + chunk; t < std::min(r.len, m + p->segment); t += chunk) {
        const long at = (r.start + t) / chunk;
        CHECK((at + 1) * place <= room);
        CHECK(places.insert(at).second);
      }
    if (r.len <= chunk) continue;
    const long first = r.slot(s, chunk);
    CHECK(first >= next && first + r.segments(chunk) <= p->chunk_slots);
    next = first + r.segments(chunk);
  }
  s4dplr_linear_attention_plan_destroy(p);
  return 0;
}

int main() {
  std::mt19937 gen(1);
  for (int i = 0; i < 20000; ++i) {
    const int S = 1 + (int)(gen() % 40), top = gen() % 3 ? 4 : 900, Hv = gen() % 4 ? 1 : 600;
    std::vector<int> o{(int)(gen() % 70)};
    for (int s = 0; s < S; ++s)
      o.push_back(o.back() + (int)(gen() % 5 == 0 ? 32 * (gen() % 40) + gen() % 3 : gen() % (gen() % 8 ? top : 4 * top + 20)));
    const long tokens = o.back() + (gen() % 2 ? 0 : (long)(gen() % 100));
    if (check(tokens, o, Hv, gen() % 2 ? 8 : 200, (int)(gen() % 3))) return 1;
  }
  std::puts("ok");
  return 0;
}
