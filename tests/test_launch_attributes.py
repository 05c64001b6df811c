"""No launcher keeps per-device launch state for the whole process.

cudaFuncSetAttribute acts on the current device, and a failure of it may pass: it has to be called at
every launch (or its success kept by device), never once for the process.  A second device cannot be
assumed where these tests run, so the sources are read instead.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(__file__)), "matrix_state_nonlinear_gb300", "csrc")
LAUNCHERS = [f for f in sorted(os.listdir(CSRC))
             if f.endswith(".cu") and "cudaFuncSetAttribute" in open(os.path.join(CSRC, f)).read()]


def test_there_are_launchers():
    assert len(LAUNCHERS) > 10


@pytest.mark.parametrize("name", LAUNCHERS)
def test_attributes_are_set_at_every_launch(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    for m in re.finditer(r"cudaFuncSetAttribute", text):
        before = text[:m.start()]
        body = before[before.rfind("\n}"):]  # from the end of the function before
        assert "call_once" not in body and "once_flag" not in body, name
        assert not re.search(r"static\s+(const\s+)?(bool|cudaError_t)\b[^;(]*;", body), name
        assert not re.search(r"static\s+const\s+\w+\s+\w+\s*=\s*$", body), name
