// code_ring.cuh -- how the sets of converting warps of the small-batch kernel walk over its
// ring of code stages.  Plain C++ without CUDA headers, so that a model of the ring on the
// host runs the code that the kernel runs.
//
// Groups (128 channels of a tile) are numbered tile by tile; set j converts groups j, j + 4,
// ...  A stage holds up to four neighbouring groups, and every tile starts a new one: where
// a tile's groups are not a multiple of four, its last stage is short, and a set finds
// stages without a group of its own.
//
// Invariant: every set visits every stage, in order: it waits until the stage is full,
// converts its group if it has one there (one at most), and gives the stage back.  A stage
// is loaded anew once all four sets have given it back.  So a set that waits for phase p of
// a slot has seen phase p - 1 complete (its own visit), and phase p + 1 cannot complete
// before it has passed p: the two phases that one bit of parity tells apart.  Neither half
// can go.  A set that jumps over stages waits for a phase whose predecessor may not be
// complete, and passes at once; a set that waits for all stages without giving them back
// can be overtaken by a phase, and then waits for ever.
//
// A set may end behind its last group without visiting the stages left: those are three at
// most (each with a group of another set), and with three slots or more nothing is loaded
// into the places of stages that it has not visited.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define W4_RING_FN __host__ __device__ __forceinline__
#else
#define W4_RING_FN inline
#endif

namespace w4 {
namespace fsk {

constexpr int kSets = 4;        // sets of converting warps
constexpr int kCodeGroups = 4;  // groups of a stage
constexpr int kMinCodeStages = 3;
static_assert(kCodeGroups <= kSets, "a set has one group of a stage at most");
static_assert(kMinCodeStages >= kSets - 1, "stages behind a set's last group find room without its visit");

struct CodeWalk {
  int groups, slots;        // groups of a tile, slots of the ring
  int tile = 0, group = 0;  // the set's next group: its tile, its number there
  int slot = 0;             // the stage to visit next: its slot, its phase's parity
  uint32_t phase = 0;
  int skip = 0;             // stages without a group of this set in front of the next one's

  W4_RING_FN CodeWalk(int set, int ng, int nc) : groups(ng), slots(nc), group(set) { settle(0, 0); }

  // On to the set's next group (after leave()).
  W4_RING_FN void next() {
    const int from = group / kCodeGroups;
    group += kSets;
    settle(from, 1);
  }
  // Waits for the stages up to the one of the next group and gives those in front of it back;
  // false where a wait ran out.
  template <class Wait, class Give>
  W4_RING_FN bool reach(Wait wait, Give give) {
    for (; skip > 0; --skip) {
      if (!wait(slot, phase)) return false;
      give(slot);
      leave();
    }
    return wait(slot, phase);
  }
  // Behind a visit: the next stage in order.
  W4_RING_FN void leave() {
    if (++slot == slots) slot = 0, phase ^= 1u;
  }

 private:
  // `group` counts from the start of `tile`, and may lie behind its end; stages [0, from +
  // done) of that tile were visited.
  W4_RING_FN void settle(int from, int done) {
    int stages = -from - done;
    while (group >= groups) {
      group -= groups;
      stages += (groups + kCodeGroups - 1) / kCodeGroups;
      ++tile;
    }
    skip = stages + group / kCodeGroups;
  }
};

}  // namespace fsk
}  // namespace w4
