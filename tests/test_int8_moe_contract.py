"""What the int8 and routing sources and entry points promise, without a GPU."""
import os
import re

import pytest

import w4a16_gemv_amd as amd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w4a16_gemv_amd", "csrc")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(amd.LIB_PATH):
        from w4a16_gemv_amd import build
        build.build()
    return amd.load()


def test_assembly_that_writes_m0_says_so():
    """A statement that sets m0 without naming it leaves the compiler free to hold a value there across it."""
    found = 0
    for name in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, name), encoding="utf-8").read()
        for statement in re.findall(r"\basm\b(?:\s+volatile)?\s*\((.*?)\);", text, flags=re.S):
            if re.search(r"\b\w+\s+m0\s*,", statement):
                found += 1
                assert re.search(r'"m0"', statement.rsplit(":", 1)[1]), f"{name}: {statement}"
    assert found >= 2
