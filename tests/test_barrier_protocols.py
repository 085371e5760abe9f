"""The barrier protocols of the cross-attention kernels on the host (tests/barrier_model.py), with the
numbers of slots and barriers that the kernels are compiled with (csrc/cross_phases.h)."""
import ctypes
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
int dkv_stages_of(int d) { return dkv_stages(d); }
int dkv_five_of(int d) { return dkv_five(d); }
int dkv_turns() { return kDkvTurns; }
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
@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("steps", [1, 2, 3, 14])
def test_dk_dv_kernel(numbers, d, steps):
    c = dict(stages=numbers.dkv_stages_of(d), five=bool(numbers.dkv_five_of(d)), turns=numbers.dkv_turns())
    bm.check(lambda: bm.dkv(c, steps))


def test_two_barriers_in_turn_are_too_few_for_five_slots():
    with pytest.raises(bm.Violation):
        bm.check(lambda: bm.dkv(dict(stages=6, five=True, turns=2), 14))
