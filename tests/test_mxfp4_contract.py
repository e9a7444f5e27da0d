"""How mxfp4_gemv and mxfp4_moe_mlp take rows, without a GPU: every plan has a kernel
and room in LDS, and the GPU tests reach every variant."""
import ctypes as C
import itertools
import os

import pytest

import w4a16_gemv_amd as amd
from tests import test_gpu_mxfp4_contract as on_gpu
from tests.test_gpu_mxfp4 import TYPES

LDS = 112 << 10         # for rows
KERNELS = {(8, 1), (8, 2), (8, 4), (4, 4), (2, 4), (1, 4)}      # waves, units of each


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(amd.LIB_PATH):
        from w4a16_gemv_amd import build
        build.build()
    return amd.load()


def sizes():
    """(T, top_k, experts, H, F) over the range; experts 0 is mxfp4_gemv of T rows of H."""
    lengths = sorted({n + d for n in (1, 128, 256, 384, 512, 640, 1024, 1152, 1280, 1664, 2048, 2304, 3584, 4096, 5120, 7168,
                                      8192, 11008, 16384, 1 << 20) for d in (0, 1) if n + d <= 1 << 20})
    for M, H, F in itertools.product(range(1, 17), lengths, (1, 500, 4200, 9000, 17000, 33000, 200000)):
        yield M, 1, 0, H, F
    for T, (k, E), H, F in itertools.product((1, 2, 3, 4, 8, 10, 13, 16, 20, 40, 64), ((1, 1), (2, 3), (2, 8), (8, 64), (32, 1024)),
                                             lengths, (1, 130, 1000, 11008)):
        yield T, k, E, H, F


def test_every_plan_has_a_kernel_and_room():
    parts = (1, 2, 3)
    for T, k, E, H, F in sizes():
        for dtype in TYPES:
            split, units, width, rows, down = on_gpu.rows_plan(T, k, E, H, F, dtype)
            case = (T, k, E, H, F, dtype)
            assert (split, units) in KERNELS, case
            if width == 0:
                assert E == 0, case
                continue
            # whole steps, at least one, and rows of them (16 bytes apart) that fit
            assert width > 0 and width % (128 * split * units) == 0, case
            assert rows * parts[TYPES.index(dtype)] * (2 * width + 16) <= LDS, case
            assert E > 0 or width >= H, case
            assert (E > 0) == (down >= 0), case


def variants(T, k, E, H, F, dtype):
    split, units, width, rows, down = on_gpu.rows_plan(T, k, E, H, F, dtype)
    if E == 0:
        return {(dtype, split, units) if width else (dtype, "wide", 1 if T <= 4 else 2 if T <= 8 else 4)}
    return {(dtype, "up", split, units, "whole" if width >= H else "in turns"), (dtype, "down", down)}


def test_the_gpu_tests_reach_every_variant():
    want, reached = set(), set()
    for s in sizes():
        for dtype in TYPES:
            want |= variants(*s, dtype)
    for dtype in TYPES:
        for M, N, K in on_gpu.GEMV:
            reached |= variants(M, 1, 0, K, N, dtype)
        for s in on_gpu.MLP:
            reached |= variants(*s, dtype)
    assert len(want) >= 3 * (6 + 3 + 6 + 4) and reached >= want, want - reached


def test_rows_probe_arguments(lib):
    a = (C.c_int32 * 5)()
    ask = lambda T=4, k=2, E=8, H=64, F=32, dt=0, a=a: lib.nf4_probe_mxfp4_rows(T, k, E, H, F, dt, a)  # noqa: E731
    assert ask() == 0 and ask(E=0) == 0 and a[4] == -1
    for bad in (dict(T=0), dict(k=0), dict(E=-1), dict(H=-1), dict(F=-1), dict(dt=3), dict(a=None), dict(E=0, T=17)):
        assert ask(**bad) == 1
    for large in (dict(T=65), dict(k=33), dict(E=1025), dict(H=(1 << 20) + 1), dict(E=0, H=(1 << 20) + 1), dict(E=0, F=1 << 31)):
        assert ask(**large) == 2


def test_the_gpu_tests_reach_every_share_of_large_tiles():
    """Of rows sorted by expert, on 256 compute units."""
    for counts, slots, N, K, kind in on_gpu.LARGE:
        assert on_gpu.plan(slots, N, K, len(counts)) == (5, 1) and on_gpu.shares(counts, N, 256) == kind
    assert {case[-1] for case in on_gpu.LARGE} >= {(True, "whole"), (True, "halves"), (True, "quarters"), (False, "halves")}
