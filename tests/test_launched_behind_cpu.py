"""Kernels that may begin before the launch ahead of them has ended read what that launch writes
with loads that see it once it is waited for: none takes the read-only path, whose data must not
change while the kernel runs."""
import os
import re

import pytest

from test_paged_cpu import CSRC

FILES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))
               and "griddep_wait()" in open(os.path.join(CSRC, f)).read())


def test_there_are_such_kernels():
    assert "pages_reserve.cu" in FILES and "qk_rope.cu" in FILES


@pytest.mark.parametrize("name", FILES)
def test_no_read_only_loads(name):
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    for form in (r"\b__ldg\s*\(", r"\bld\.global(\.\w+)*\.nc\b",
                 # (the compiler takes that path by itself for these)
                 r"\bconst\s+[\w:]+\s*\*\s*(const\s+)?__restrict__"):
        assert not re.search(form, src), (name, form)
