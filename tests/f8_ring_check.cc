// Runs the 8-bit product's load producer (f8_ring.h) against a model of its
// barriers: every fill's loads land at once, a consumer frees stages in order,
// and the n-th wait for a free stage runs out.  Prints the first thing that is
// wrong, or "ok".
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "f8_ring.h"

namespace {

struct Model {
  int stages, k_blocks, kbs, k_split, fail_at;   // fail_at: this wait_empty runs out (-1: none)
  std::vector<int> fills, waited;
  int waits = 0, cur_tile = -1;
  bool stop = false;
  std::vector<std::pair<int, int>> loaded;   // (tile, K block) of the real fills

  void bad(const char* what, int a, int b) {
    std::printf("%s (%d, %d): stages %d, K blocks %d, slices %d, wait %d runs out\n", what, a, b, stages, k_blocks,
                k_split, fail_at);
    std::exit(0);
  }
  bool aborted() const { return stop; }
  void abort() { stop = true; }
  void tile(int t) { cur_tile = t; }
  bool wait_empty(int stage, uint32_t parity) {
    if (stop) bad("waits for a free stage after a wait ran out", stage, (int)parity);
    // completes when the consumer has freed the stage once per earlier fill: `fills` phases, of parity fills - 1;
    // the first pass waits for the phase before the first one
    if (parity != (uint32_t)((fills[stage] - 1) & 1)) bad("wrong phase of a free stage", stage, (int)parity);
    return waits++ != fail_at;
  }
  void fill(int stage, int kb, bool real) {
    int sum = 0;
    for (int f : fills) sum += f;
    if (stage != sum % stages) bad("fills out of order", stage, sum);
    ++fills[stage];
    if (real) loaded.push_back({cur_tile, kb});
  }
  void wait_full(int stage, uint32_t parity) {
    // a barrier that has completed f phases lets a wait for parity (f - 1) & 1 through; for the other one it waits on
    if (fills[stage] == 0 || parity != (uint32_t)((fills[stage] - 1) & 1))
      bad("waits for a phase that does not complete", stage, (int)parity);
    ++waited[stage];
  }
};

template <int kGroups>
void check(int total, int first, int step, int k_split, int k_blocks, int fail_at) {
  Model m;
  m.stages = 4 * kGroups;
  m.k_blocks = k_blocks;
  m.k_split = k_split;
  m.kbs = (k_blocks + k_split - 1) / k_split;
  m.fail_at = fail_at;
  m.fills.assign(m.stages, 0);
  m.waited.assign(m.stages, 0);
  csa::f8_fill_ring<kGroups>(m, first, total, step, k_split, m.kbs, k_blocks);
  if (m.stop) {
    for (int s = 0; s < m.stages; ++s)
      if (m.waited[s] != (m.fills[s] > 0)) m.bad("a load is not waited for, or twice", s, m.waited[s]);
    return;
  }
  std::vector<std::pair<int, int>> want;
  for (int u = first; u < total; u += step)
    for (int kb = u % k_split * m.kbs; kb < k_blocks && kb < u % k_split * m.kbs + m.kbs; ++kb)
      want.push_back({u / k_split, kb});
  if (m.loaded != want) m.bad("wrong blocks loaded", (int)m.loaded.size(), (int)want.size());
}

}  // namespace

int main() {
  for (int fail_at = -1; fail_at < 70; ++fail_at)
    for (int k_blocks : {1, 3, 4, 5, 8, 12, 13, 16, 17, 32})
      for (int total : {1, 2, 5}) {
        check<1>(total, 0, 1, 1, k_blocks, fail_at);
        check<2>(total, 0, 1, 1, k_blocks, fail_at);
        check<2>(total + 3, 1, 2, 1, k_blocks, fail_at);
        for (int k_split : {2, 4, 8})
          if (k_blocks % (4 * k_split) == 0) check<2>(total * k_split, 1, 3, k_split, k_blocks, fail_at);
      }
  std::puts("ok");
  return 0;
}
