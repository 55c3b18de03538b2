"""A model of the small-batch kernel's ring of code stages, driven on the CPU by the walk that
the kernel's converting sets run (csrc/code_ring.cuh, compiled here for the host).

The ring: a producer loads stages of up to four groups into `slots` slots, in order, each once
the slot's stage before has been given back by all sets; loads take random times and may land
out of order.  Four sets convert the groups in turn, and the products of a group, in order,
free the buffer that its set needs again four groups later.  In front of a tile's first group
a set takes a random time (it reads the tile's scales from memory there).  Barriers are modelled as the
hardware has them: a wait names a parity, and passes when the phase that is under way has the
other one.  So a wait can pass too early (the phase before the wanted one is not complete
either) or miss its phase (the one behind it is complete too): the model says which.

Row factors of a tile are kept in one of 16 places, read when its results go out.

The model is checked with two faulty rules, planted here: sets that jump over stages without
a group of theirs, and sets that wait for those but do not give them back."""
import ctypes
import heapq
import os
import random
import subprocess

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_int4_w4_b200", "csrc")
SETS, STAGE = 4, 4
ROW_FACTORS = 16  # tiles whose row factors are kept (kRowFactors of csrc/fused_skinny.cu)

HARNESS = r"""
#include "code_ring.cuh"
// The steps of one set: 3 ints each, (kind, slot, parity or group); kind 0 waits, 1 gives
// back, 2 converts, 3 starts a tile.  Returns their number.
extern "C" int steps(int set, int groups, int tiles, int slots, int *out, int room) {
  using namespace w4::fsk;
  int n = 0;
  auto put = [&](int kind, int a, int b) {
    if (n < room) out[3 * n] = kind, out[3 * n + 1] = a, out[3 * n + 2] = b;
    ++n;
  };
  CodeWalk walk(set, groups, slots);
  int tile = -1;
  for (int i = set; i < groups * tiles; i += kSets, walk.next()) {
    if (walk.tile * groups + walk.group != i) return -1;
    if (walk.tile != tile) put(3, 0, tile = walk.tile);
    walk.reach([&](int c, uint32_t ph) { put(0, c, (int)ph); return true; }, [&](int c) { put(1, c, 0); });
    put(2, walk.slot, i);
    put(1, walk.slot, 0);
    walk.leave();
  }
  return n;
}
extern "C" int min_slots() { return w4::fsk::kMinCodeStages; }
extern "C" int sets_and_groups() { return w4::fsk::kSets * 100 + w4::fsk::kCodeGroups; }
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    (d / "h.cpp").write_text(HARNESS)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I" + SRC, "-o", str(d / "h.so"), str(d / "h.cpp")])
    lib = ctypes.CDLL(str(d / "h.so"))
    lib.steps.argtypes = [ctypes.c_int] * 4 + [ctypes.POINTER(ctypes.c_int), ctypes.c_int]
    assert lib.sets_and_groups() == SETS * 100 + STAGE and lib.min_slots() == 3
    return lib


def kernel_steps(lib, j, ng, tiles, slots):
    room = 8 * ng * tiles + 8
    buf = (ctypes.c_int * (3 * room))()
    n = lib.steps(j, ng, tiles, slots, buf, room)
    assert 0 <= n <= room
    return [tuple(buf[3 * k:3 * k + 3]) for k in range(n)]


def stage_of(i, ng):
    return i // ng * -(-ng // STAGE) + i % ng // STAGE


def jumping_steps(j, ng, tiles, slots):
    """Planted: waits for the stages with a group of its own only; a tile's last group gives back
    for the groups that its stage lacks."""
    out = []
    for i in range(j, ng * tiles, SETS):
        c = stage_of(i, ng)
        out += [(3, 0, i // ng)] if i % ng < SETS else []
        out += [(0, c % slots, c // slots & 1), (2, c % slots, i)]
        out += [(1, c % slots, 0)] * (STAGE - i % ng % STAGE if i % ng == ng - 1 else 1)
    return out


def waiting_steps(j, ng, tiles, slots):
    """Planted: waits for every stage in order, but gives back as above."""
    out, c = [], 0
    for i in range(j, ng * tiles, SETS):
        out += [(3, 0, i // ng)] if i % ng < SETS else []
        while c <= stage_of(i, ng):
            out.append((0, c % slots, c // slots & 1))
            c += 1
        k = (c - 1) % slots
        out += [(2, k, i)] + [(1, k, 0)] * (STAGE - i % ng % STAGE if i % ng == ng - 1 else 1)
    return out


def simulate(programs, ng, tiles, slots, seed, latency=(800, 2500), pause=(0, 4000)):
    """Runs the ring once; the list of what went wrong (empty: every group was converted from its
    own stage, whole, and everything came to an end)."""
    rng = random.Random(seed)
    total = ng * tiles
    stages = tiles * -(-ng // STAGE)
    full = [0] * slots                      # completed phases
    given, empty = [0] * slots, [0] * slots  # give-backs of the phase under way, completed phases
    holds = [None] * slots                  # stage that has landed, None while a load is under way
    reading = [0] * slots
    converted, done = set(), 0              # groups; products done, in order
    wrong, queue, tick = [], [], 0

    def at(t, what, *a):
        nonlocal tick
        tick += 1
        heapq.heappush(queue, (t, tick, what, a))

    summed, out_busy = 0, False             # tiles whose results are out, which frees one of two accumulators
    issued, pc, busy = 0, [0] * SETS, [False] * SETS
    mma_busy = False

    def settle(t):
        """Everything that can go on at time t does."""
        nonlocal issued, mma_busy, out_busy
        moved = True
        while moved and not wrong:
            moved = False
            if issued < stages:
                s, want = issued % slots, issued // slots & 1 ^ 1
                if empty[s] & 1 != want:
                    if reading[s]:
                        wrong.append(f"stage {issued} is loaded over one that is read")
                    holds[s] = None
                    at(t + rng.randint(*latency), "landed", s, issued)
                    issued += 1
                    moved = True
            for j in range(SETS):
                while not busy[j] and pc[j] < len(programs[j]):
                    kind, s, x = programs[j][pc[j]]
                    if kind == 0:
                        if full[s] & 1 == x:
                            break
                    elif kind == 1:
                        given[s] += 1
                        if given[s] == SETS:
                            given[s], empty[s] = 0, empty[s] + 1
                    elif kind == 3:
                        if x - ROW_FACTORS >= summed:
                            wrong.append(f"row factors of tile {x} written over tile {x - ROW_FACTORS}'s")
                        busy[j] = True
                        at(t + rng.randint(*pause), "ready", j)
                    else:
                        if x >= SETS and done <= x - SETS:
                            break  # the buffer is still multiplied (the codes are read by then: later is stricter)
                        if holds[s] != stage_of(x, ng):
                            wrong.append(f"group {x} is read from a slot that holds {holds[s]}")
                        reading[s] += 1
                        busy[j] = True
                        at(t + rng.randint(150, 400), "converted", j, s, x)
                    pc[j] += 1
                    moved = True
            if not mma_busy and done < total and done in converted and done // ng < summed + 2:
                mma_busy = True
                at(t + rng.randint(180, 230), "multiplied")
                moved = True
            if not out_busy and summed < done // ng:
                out_busy = True
                at(t + rng.randint(100, 3000), "summed")
                moved = True

    t = 0
    settle(0)
    while queue and not wrong:
        t, _, what, a = heapq.heappop(queue)
        if what == "landed":
            holds[a[0]] = a[1]
            full[a[0]] += 1
        elif what == "ready":
            busy[a[0]] = False
        elif what == "converted":
            j, s, x = a
            if holds[s] != stage_of(x, ng):
                wrong.append(f"group {x}: its stage was overwritten")
            reading[s] -= 1
            busy[j] = False
            converted.add(x)
        elif what == "summed":
            out_busy = False
            summed += 1
        else:
            mma_busy = False
            done += 1
        settle(t)
    if not wrong and (summed < tiles or any(p < len(q) for p, q in zip(pc, programs))):
        wrong.append(f"stands still after {done} of {total} groups")
    return wrong


@pytest.mark.parametrize("slots", [3, 4, 5])
@pytest.mark.parametrize("ng", list(range(1, 10)) + [14, 28, 32])
def test_every_group_is_read_from_its_own_stage(walk, ng, slots):
    for tiles in (1, 2, 3, 4, 7, 23):
        programs = [kernel_steps(walk, j, ng, tiles, slots) for j in range(SETS)]
        for seed in range(6 if ng * tiles < 200 else 2):
            assert simulate(programs, ng, tiles, slots, seed) == [], (ng, slots, tiles, seed)


def test_a_set_visits_every_stage_in_order(walk):
    for slots in (3, 4, 5):
        for ng in range(1, 10):
            for j in range(SETS):
                p = kernel_steps(walk, j, ng, 9, slots)
                waits = [(s, x) for k, s, x in p if k == 0]
                assert waits == [(c % slots, c // slots & 1) for c in range(len(waits))]
                assert [s for k, s, _ in p if k == 1] == [s for s, _ in waits]  # each given back once
                left = 9 * -(-ng // STAGE) - len(waits)
                assert 0 <= left <= SETS - 1  # what it may leave at the end


@pytest.mark.parametrize("plant,says", [(jumping_steps, "is read from a slot"), (waiting_steps, "stands still")])
def test_the_model_sees_planted_faults(plant, says):
    seen = [w for seed in range(40) for w in simulate([plant(j, 1, 12, 3) for j in range(SETS)], 1, 12, 3, seed)]
    assert any(says in w for w in seen), seen[:3]
    # neither shows where a tile's groups fill its stages
    for seed in range(5):
        assert simulate([plant(j, 8, 5, 3) for j in range(SETS)], 8, 5, 3, seed) == []
