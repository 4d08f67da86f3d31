// A warp's ring of steps on the host: barriers that count their phases, copies that land when they are waited
// for, and a step whose copies are late. Whatever the number of steps and the one that is late, what is still
// on its way is waited for, and nothing that was never issued. Prints the cases that fail.
#include <cstdio>

#include "step_ring.cuh"

namespace {

constexpr int kStages = 2;

struct Model {
  int issued[kStages] = {}, landed[kStages] = {};
  bool done(int stage, uint32_t parity) const { return (landed[stage] & 1u) != parity; }
};

// `steps` steps, of which number `late` (from 0; past the end: none) does not land in time.
bool run(int steps, int late) {
  Model m;
  quail::StepRing<kStages> due;
  int next = 0;
  bool more = steps > 0, is_late = false, ok = true;
  auto issue = [&](int stage) {
    if (!more) return;
    ok = ok && m.issued[stage] == m.landed[stage];  // the stage is free
    ++m.issued[stage];
    more = ++next < steps;
  };
  for (int s = 0; s < kStages - 1; ++s) issue(s);
  for (int step = 0; step < steps; ++step) {
    const bool next_too = more;
    issue(due.ahead());
    const int stage = due.stage;
    if (!is_late) {
      ok = ok && m.issued[stage] == m.landed[stage] + 1 && !m.done(stage, due.parity);
      if (step == late) {
        is_late = true;
        more = false;
        due.drain(next_too ? 2 : 1, [&](int s, uint32_t parity) {
          ok = ok && m.issued[s] == m.landed[s] + 1 && !m.done(s, parity);
          ++m.landed[s];
          ok = ok && m.done(s, parity);
        });
      } else {
        ++m.landed[stage];
        ok = ok && m.done(stage, due.parity);
      }
    }
    due.next();
  }
  for (int s = 0; s < kStages; ++s) ok = ok && m.issued[s] == m.landed[s];
  return ok;
}

}  // namespace

int main() {
  int failed = 0;
  for (int steps = 0; steps < 20; ++steps)
    for (int late = 0; late <= steps; ++late)
      if (!run(steps, late)) {
        printf("FAILED: %d steps, number %d late\n", steps, late);
        ++failed;
      }
  return failed != 0;
}
