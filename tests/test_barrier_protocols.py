"""The barrier protocols of the cross-attention kernels on the host (tests/barrier_model.py), with the
numbers of slots and barriers that the kernels are compiled with (csrc/cross_phases.h)."""
import ctypes
import functools
import os
import shutil
import subprocess

import pytest

from geometry_aware_local_pack3d_b200 import build

from . import barrier_model as bm

DIMS = [48, 64, 96, 128]
WRAPPERS = """
#include "cross_phases.h"
using namespace p3d::xa;
extern "C" {
int fwd_slots_of(int d) { return fwd_slots(d); }
int fwd_bufs_of(int d) { return fwd_bufs(d); }
int fwd_ready() { return kFwdReady; }
int dq_slots_of(int d) { return dq_slots(d); }
int dq_own_of(int d) { return dq_own(d); }
int dq_ready() { return kDqReady; }
int dkv_stages_of(int d) { return dkv_stages(d); }
int dkv_five_of(int d) { return dkv_five(d); }
int dkv_turns() { return kDkvTurns; }
int short_turns() { return kShortTurns; }
}
"""


@pytest.fixture(scope="module")
def numbers(tmp_path_factory):
    """The header's numbers, compiled for the host."""
    at = tmp_path_factory.mktemp("phases")
    (at / "numbers.cpp").write_text(WRAPPERS)
    out = os.path.join(at, "numbers.so")
    subprocess.run([shutil.which("g++") or "g++", "-std=c++17", "-shared", "-fPIC", "-I", build.CSRC,
                    str(at / "numbers.cpp"), "-o", out], check=True)
    return ctypes.CDLL(out)


# ------------------------------------------------------------------ the model itself
def test_the_model_notices_an_early_an_overtaken_and_a_stuck_wait():
    def machine(*agents):
        m = bm.Machine()
        m.bar("a")
        for i, ops in enumerate(agents):
            m.agent(f"agent {i}", iter_ops(ops))
        return m

    def iter_ops(ops):
        for op in ops:
            yield op

    bm.check(lambda: machine([("arrive", "a")], [("wait", "a", 0)]))
    for ops in ([("arrive", "a"), ("arrive", "a")], []):  # overtaken, and never completed
        with pytest.raises(bm.Violation):
            bm.check(lambda: machine(ops, [("wait", "a", 0)]))
    with pytest.raises(bm.Violation):  # phase 1 looks complete before phase 0 is
        bm.check(lambda: machine([("arrive", "a"), ("arrive", "a")], [("wait", "a", 1)]))
    with pytest.raises(bm.Violation):  # a buffer that is still being written
        bm.check(lambda: machine([("copy", "K", "x", 1, "a"), ("read", "x", 1)]))


# ------------------------------------------------------------------ the kernels
@functools.cache
def holds(kernel, numbers, *args):
    """Checks a kernel once for head dims that share their numbers."""
    bm.check(lambda: kernel(dict(numbers), *args))


# (row tiles, state tiles) of the units of a CTA: one row tile alone, single state tiles, none
FORWARD_UNITS = [((2, 3), (1, 2), (2, 0), (2, 1), (2, 1), (1, 4), (2, 2)), ((1, 6), (1, 3), (1, 1))]


def forward_numbers(numbers, d):
    return (("slots", numbers.fwd_slots_of(d)), ("bufs", numbers.fwd_bufs_of(d)),
            ("ready", numbers.fwd_ready()))


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("units", FORWARD_UNITS)
def test_forward_kernel(numbers, d, masked, units):
    holds(bm.forward, forward_numbers(numbers, d), units, masked)


@pytest.mark.parametrize("d", DIMS)
def test_forward_ring_gives_k_and_v_slots_of_their_own(numbers, d):
    # whoever waits for K items alone (or V items alone) sees every phase of the slots they come to
    slots = numbers.fwd_slots_of(d)
    for first in (0, 1):
        seen = {}
        for item in range(first, 20 * slots, 2):
            slot, phase = item % slots, item // slots
            assert phase == seen.get(slot, -1) + 1
            seen[slot] = phase


@pytest.mark.parametrize("units", FORWARD_UNITS)
@pytest.mark.parametrize("masked", [False, True])
def test_an_odd_ring_is_noticed(units, masked):
    with pytest.raises(bm.Violation):
        bm.check(lambda: bm.forward(dict(slots=5, bufs=1, ready=8), units, masked))


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("units", [(5, 3, 1, 1, 2), (11,)])
def test_dq_kernel(numbers, d, masked, units):
    holds(bm.dq, (("slots", numbers.dq_slots_of(d)), ("ready", numbers.dq_ready()),
                  ("own", bool(numbers.dq_own_of(d)))), units, masked)


@pytest.mark.parametrize("run", [(5,), (1, 1, 1, 1), (3, 2, 4)])
def test_short_forward_kernel(numbers, run):
    holds(bm.forward_short, (("staged", numbers.short_turns()),), run)
    with pytest.raises(bm.Violation):  # one barrier for both buffers of rows is too few
        bm.check(lambda: bm.forward_short(dict(staged=1), run))


@pytest.mark.parametrize("bufs", [1, 2])
@pytest.mark.parametrize("run", [[5], [1, 1, 1, 1], [3, 2, 4]])
def test_short_backward_kernel(bufs, run):
    bm.check(lambda: bm.backward_short(dict(bufs=bufs), run))


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("steps", [1, 2, 3, 14])
def test_dk_dv_kernel(numbers, d, steps):
    holds(bm.dkv, (("stages", numbers.dkv_stages_of(d)), ("five", bool(numbers.dkv_five_of(d))),
                   ("turns", numbers.dkv_turns())), steps)


def test_two_barriers_in_turn_are_too_few_for_five_slots():
    with pytest.raises(bm.Violation):
        bm.check(lambda: bm.dkv(dict(stages=6, five=True, turns=2), 14))
