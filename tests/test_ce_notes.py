"""The vocabulary loss' notes (what a tile's epilogue wants of its tokens), on the
CPU: the order in which a workgroup brings them and reads them, stepped through for
items of any number of stages, finds each note still in its slot."""
import os
import re

import pytest

import fp8_scaled_matmul_amd as fm

SOURCE = os.path.join(os.path.dirname(fm.__file__), "csrc", "ce_gemm.h")


def overwritten(stages, ring, slots, items=40):
    """Items whose slot another's note has taken, or is on its way to, when their
    epilogue reads it.  The fills run `ring` stages ahead; the one that ends an item
    describes the next, whose note goes to the next slot."""
    slot_of, held, described = {}, {}, 0

    def describe():
        nonlocal described
        if described < items:
            slot_of[described] = described % slots
            held[described % slots] = described
        described += 1

    describe()
    filled = 0

    def fill():
        nonlocal filled
        if described <= items and (filled + 1) % stages == 0:
            describe()
        filled += 1

    for _ in range(ring):
        fill()
    bad = []
    for item in range(items):
        for _ in range(stages):
            fill()              # at the end of the stage, before an epilogue
        if held[slot_of[item]] != item:
            bad.append(item)
    return bad


def constants():
    text = open(SOURCE).read()
    ring = int(re.search(r"constexpr int kRing = (\d+);", text)[1])
    slots, least = re.search(r"constexpr int kNoteSlots = (\w+), kNoteStages = (\d+);", text).groups()
    return ring, ring if slots == "kRing" else int(slots), int(least)


def test_the_model_finds_a_slot_too_few():
    assert overwritten(1, 4, 5)             # each item with five behind it
    assert not overwritten(1, 4, 6)
    assert overwritten(2, 4, 3) and not overwritten(2, 4, 4)


@pytest.mark.parametrize("more", range(6))
def test_notes_stay_until_they_are_read(more):
    ring, slots, least = constants()
    assert least >= 1 and not overwritten(least + more, ring, slots)

