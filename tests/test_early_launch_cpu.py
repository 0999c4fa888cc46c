"""What kernels that start before the launch in front of them has ended must keep to, read in their sources
(CPU only)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "backward_optimizer_gb300", "csrc")


def _sources():
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".cu", ".cuh", ".h")):
            with open(os.path.join(CSRC, f)) as h:
                # without comments
                yield f, re.sub(r"//[^\n]*", "", h.read())


def test_nothing_is_read_as_constant():
    """__ldg and ld.global.nc promise that the value does not change while the kernel runs.  A kernel that starts
    early runs while the launch in front still writes, and the compiler may move such a load before the wait."""
    found = [f for f, text in _sources() if re.search(r"__ldg\s*\(|global\.nc|__restrict__", text)]
    assert found == []


def test_the_next_launch_is_let_go_only_behind_the_wait():
    """An early read (the weights of a few-token product) relies on it: all but one launch in front are done."""
    for f, text in _sources():
        for at in (m.start() for m in re.finditer("griddepcontrol.launch_dependents", text)):
            assert text[:at].endswith('griddepcontrol.wait;\\n\\t'), f
