// step_ring.cuh - where a ring of steps stands: which stage and which phase of the stage's mbarrier a step
// uses. Plain arithmetic, for the GPU and for programs on the host.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define QUAIL_RING_FN __host__ __device__ __forceinline__
#else
#define QUAIL_RING_FN inline
#endif

namespace quail {

// A reader's place: the step that it waits for next. The step that uses stage i for the n-th time (from 0)
// is phase n of the stage's barrier, and a wait takes n's lowest bit.
template <int STAGES>
struct StepRing {
  int stage = 0;
  uint32_t parity = 0;

  // The stage that the last step of a full ring goes into: the one read before this.
  QUAIL_RING_FN int ahead() const { return stage == 0 ? STAGES - 1 : stage - 1; }
  QUAIL_RING_FN void next() {
    if (++stage == STAGES) {
      stage = 0;
      parity ^= 1;
    }
  }
  // wait(stage, parity) for `steps` steps from this one on, which have been issued.
  template <class Wait>
  QUAIL_RING_FN void drain(int steps, Wait&& wait) const {
    StepRing at = *this;
    for (int i = 0; i < steps; ++i, at.next()) wait(at.stage, at.parity);
  }
};

}  // namespace quail
