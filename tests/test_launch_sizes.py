"""A kernel's largest dynamic shared memory is one constant for all of its launches.

Set to a call's own size, it could lie too low for another host thread's call that is between its attribute and
its launch, which is then refused.  The sources are read, as in the test beside this one."""
import os
import re

import pytest

from test_launch_attributes import CSRC, LAUNCHERS

CONSTANT = re.compile(r"(\w+(<[\w, ]*>)?::)?k[A-Z]\w*$")
FIXED_LAYOUT = re.compile(r"const \w+ L = (\w+)(<\w+>)?\((\w*)\);")  # of nothing, or of a constant


@pytest.mark.parametrize("name", LAUNCHERS)
def test_the_limit_is_a_constant(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    values = re.findall(r"cudaFuncAttributeMaxDynamicSharedMemorySize,\s*([^;]*?)\);", text)
    assert values
    for v in values:
        if CONSTANT.match(v) or v == "c8_layout().total":
            continue
        assert v == "L.total", (name, v)
        layouts = FIXED_LAYOUT.findall(text)
        assert layouts and not re.search(r"\bL = \w+\(p\.", text) and not re.search(r"^  L = ", text, re.M), name
        assert all(not arg or re.search(rf"const(expr)? int {arg} = \d+;|\bint {arg}\)", text) for _, _, arg in layouts), name
