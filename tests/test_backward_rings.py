"""The backward kernel's rings of weights and operands, as a model on the CPU:
barriers that are waited for by parity, boxes that land in any order, roles that
run in any order.  A role that reads a slot has to find its own stage there,
landed.  The order in which the operand warps wait is taken from the kernel's
source."""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "q5_lm_head_gb300", "csrc", "backward.cu")
SIDES = 3          # operand slots
GROUPS = 2         # groups of operand warps, taking the stages in turn


def _operand_waits():
    """Barriers in the order in which the operand warps wait for them."""
    with open(SOURCE) as f:
        text = f.read()
    part = text[text.index("-- operands\n"):text.index("-- unpacking\n")]
    return re.findall(r"wait\(&(wfull|pempty)\[", part)


class _Barrier:
    """Phases completed so far; a wait for a parity passes while the last completed phase has that parity."""

    def __init__(self):
        self.done = 0

    def passes(self, parity):
        return (self.done & 1) != parity


def _run(order, slots, stages, rng):
    """One schedule; the stages that a role read before they were there."""
    wfull, wempty = [_Barrier() for _ in range(slots)], [_Barrier() for _ in range(slots)]
    pfull, pempty = [_Barrier() for _ in range(SIDES)], [_Barrier() for _ in range(SIDES)]
    held = [None] * slots                 # the stage whose box has landed in a slot
    flying, wrong = [], []

    def producer():
        for i in range(stages):
            s = i % slots
            while i >= slots and not wempty[s].passes((i // slots & 1) ^ 1):
                yield
            held[s] = None
            flying.append(i)
            yield

    def landing():
        landed = 0
        while landed < stages:
            if flying and rng.random() < 0.3:
                i = flying.pop(rng.randrange(len(flying)))
                held[i % slots] = i
                wfull[i % slots].done += 1
                landed += 1
            yield

    def operands(group):
        for i in range(group, stages, GROUPS):
            for bar in order:
                if bar == "wfull":
                    while not wfull[i % slots].passes(i // slots & 1):
                        yield
                else:
                    while i >= SIDES and not pempty[i % SIDES].passes((i // SIDES & 1) ^ 1):
                        yield
                yield
            if held[i % slots] != i:
                wrong.append(i)
            yield
            pfull[i % SIDES].done += 1

    def unpack():
        for i in range(stages):
            while not pfull[i % SIDES].passes(i // SIDES & 1):
                yield
            if held[i % slots] != i:
                wrong.append(i)
            yield
            wempty[i % slots].done += 1
            ready.append(i)

    def products():
        for i in range(stages):
            while i not in ready:
                yield
            yield
            pempty[i % SIDES].done += 1

    ready = []
    roles = [producer(), landing(), unpack(), products()] + [operands(g) for g in range(GROUPS)]
    for _ in range(200 * stages):
        if not roles:
            return wrong
        role = rng.choice(roles)
        try:
            next(role)
        except StopIteration:
            roles.remove(role)
        if wrong:
            return wrong
    raise AssertionError("the rings stand still")


@pytest.mark.parametrize("slots", [3, 4, 5, 6])
def test_no_role_reads_a_box_before_it_has_landed(slots):
    order = _operand_waits()
    assert sorted(order) == ["pempty", "wfull"]
    for seed in range(300):
        assert not _run(order, slots, 24, random.Random(seed)), f"schedule {seed}"


def test_the_model_finds_a_parity_taken_too_early():
    """Three slots, the weights waited for before the operands' slot: the slot's last user is the
    other group, and nothing shows that its box has landed."""
    assert any(_run(["wfull", "pempty"], 3, 24, random.Random(seed)) for seed in range(300))
