"""The order of waits and arrivals of the 4-bit product on tcgen05 (csrc/llm/w4_tiles.cuh), in a model
of its roles on the CPU.

Every barrier wait of that kernel is by parity, which tells two uses of a slot apart only for a
waiter that has seen each of them complete.  The model walks the loops of the kernel's roles in
random orders and checks that no wait passes on another use than its own, that no barrier gets more
arrivals than a phase takes, and that everything comes to an end."""
import random

import pytest

GROUPS = STAGES = 4   # decoding warpgroups, a TMEM stage for each


class Barrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.phase = self.tx = 0

    def arrive(self, tx=0):
        assert self.pending > 0, "an arrival more than the phase takes"
        self.pending -= 1
        self.tx += tx
        self.settle()

    def land(self):
        self.tx -= 1
        self.settle()

    def settle(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def passes(self, use):
        """wait.parity for the end of use `use` (-1: of none)."""
        if (self.phase & 1) == (use & 1):
            return False
        assert self.phase == use + 1, "the wait passed on another use"
        return True


def run(blocks, KB, codes, rng):
    atoms, steps = (blocks + 3) // 4, (blocks + KB - 1) // KB
    full = [Barrier(5) for _ in range(STAGES)]                 # a group's warps, and the bytes of A
    empty = [Barrier(1) for _ in range(STAGES)]
    c_full = [Barrier(1) for _ in range(codes)]
    c_empty = [Barrier(16 // KB) for _ in range(codes)]
    copies, commits = [], []                                   # in flight

    def load_a():
        for t in range(steps):
            s, use = t % STAGES, t // STAGES
            yield empty[s], use - 1
            n = min(KB, blocks - KB * t)
            full[s].arrive(n)
            copies.extend([full[s]] * n)

    def load_codes():
        for at in range(atoms):
            c, use = at % codes, at // codes
            yield c_empty[c], use - 1
            c_full[c].arrive(3)                                # codes, scales, zero points
            copies.extend([c_full[c]] * 3)

    def multiply():
        for t in range(steps):
            s, use = t % STAGES, t // STAGES
            yield full[s], use
            commits.append(empty[s])

    def decode(group):
        for t in range(group, steps, GROUPS):
            at, use = t // (4 // KB), t // STAGES
            yield c_full[at % codes], at // codes
            c_empty[at % codes].arrive()
            if use > 0:
                yield empty[group], use - 1
            full[group].arrive()

    roles = [load_a(), load_codes(), multiply()] + [decode(w // 4) for w in range(4 * GROUPS)]
    waits = {}
    for role in roles:
        step = next(role, None)
        if step is not None:
            waits[role] = step
    while waits or copies or commits:
        choices = [("role", r) for r, (bar, use) in waits.items() if bar.passes(use)]
        if copies:
            choices.append(("copy", None))
        if commits:
            choices.append(("commit", None))
        assert choices, "nothing can go on"
        what, role = rng.choice(choices)
        if what == "copy":
            copies.pop(rng.randrange(len(copies))).land()
        elif what == "commit":
            commits.pop(0).arrive()                            # MMAs end in order
        else:
            step = next(role, None)
            if step is None:
                del waits[role]
            else:
                waits[role] = step


@pytest.mark.parametrize("KB", [1, 2])
@pytest.mark.parametrize("codes", [2, 4, 6, 8])
def test_no_wait_passes_on_another_use(KB, codes):
    rng = random.Random(10 * KB + codes)
    for blocks in [*range(1, 42), 63, 64, 65, 100, 128]:
        run(blocks, KB, codes, rng)


def test_the_model_finds_a_stage_shared_by_groups():
    """With an odd number of code slots and steps of two blocks a group skips uses of a slot."""
    with pytest.raises(AssertionError):
        for seed in range(50):
            run(128, 2, 3, random.Random(seed))
