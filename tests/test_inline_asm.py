"""Inline assembly names what it changes: a statement that sets m0 or makes
the hardware write LDS says so in its clobber list, and so does every wait
and barrier, so that no compiler version may move memory accesses or a value
of its own in m0 across them.  Read from the sources; no GPU is needed."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "combine_lds_atomic_amd", "csrc")


def statements():
    for f in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, f)).read()
        for m in re.finditer(r"\basm\s+volatile\s*\((.*?)\)\s*;", text, re.S):
            yield f"{f}:{text.count(chr(10), 0, m.start()) + 1}", m.group(1)


@pytest.mark.parametrize("where,body", [pytest.param(w, b, id=w) for w, b in statements()])
def test_clobbers(where, body):
    code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', body.split('":')[0] + '"'))
    clobbers = re.findall(r'"([^"]*)"', body.rsplit(":", 1)[1])
    if re.search(r"\bm0\b", code):
        assert "m0" in clobbers, where
    if re.search(r"load_lds|s_waitcnt|s_barrier", code):
        assert "memory" in clobbers, where


def test_the_sources_hold_such_statements():
    found = [b for _, b in statements()]
    assert sum("load_lds" in b for b in found) >= 2 and sum("s_barrier" in b for b in found) >= 1
