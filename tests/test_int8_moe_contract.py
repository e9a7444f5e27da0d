"""What the int8 and routing sources and entry points promise, without a GPU."""
import ctypes as C
import os
import re

import pytest

import w4a16_gemv_amd as amd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL = 1
P = C.c_void_p(0x1000)          # never dereferenced: validation fails first
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


def _up(n, to):
    return -(-n // to) * to


@pytest.mark.parametrize("M,N,K", [(3, 8, 64), (17, 100, 1), (138, 512, 8192), (310, 512, 11008), (128, 1024, 11008)])
def test_linear_needs_room_for_codes_and_scales(lib, M, N, K):
    need = _up(M * amd.int8_pitch(K), 256) + _up(4 * M, 256)
    assert lib.int8_linear_workspace_size(M, N, K) == need + lib.int8_gemm_workspace_size(M, N, K)
    for work, size in ((P, need - 1), (P, 0), (None, need)):
        assert lib.int8_linear(P, 0, P, P, M, N, K, P, 0, work, size, None) == EINVAL


@pytest.mark.parametrize("M,K", [(1, 0), (2, 0), (1, 64), (2, 11264)])
def test_linear_of_one_or_two_tokens_needs_no_workspace(lib, M, K):
    assert lib.int8_linear_workspace_size(M, 300, K) == 0
