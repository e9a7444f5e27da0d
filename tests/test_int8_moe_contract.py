"""What the int8 and routing sources and entry points promise, without a GPU."""
import ctypes as C
import os
import re

import pytest
import torch
from torch.autograd import forward_ad

import w4a16_gemv_amd as amd
from tests import test_gpu_int8, test_gpu_int8_moe_contract as on_gpu

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


def _codes(rows, K, **kw):
    """An Int8Tensor off the GPU, which only a call that has passed its first checks would notice."""
    t = amd.Int8Tensor.__new__(amd.Int8Tensor)
    t.data, t.scale, t.K = torch.zeros(rows, amd.int8_pitch(K), dtype=torch.int8), torch.ones(rows, **kw), K
    return t


def _route(T, k, E):
    r = amd.MoeRoute.__new__(amd.MoeRoute)
    r.offsets = torch.zeros(E + 1, dtype=torch.int32)
    r.order, r.pos = torch.zeros(T * k, dtype=torch.int32), torch.zeros(T, k, dtype=torch.int32)
    return r


SCALES = {
    "dequant": lambda leaf, other: amd.int8_dequant(leaf),
    "method": lambda leaf, other: leaf.dequant(),
    "gemm x": lambda leaf, other: amd.int8_gemm(leaf, other),
    "gemm w": lambda leaf, other: amd.int8_gemm(other, leaf),
    "linear w": lambda leaf, other: amd.int8_linear(torch.zeros(6, 70), leaf),
    "vector w": lambda leaf, other: leaf.gemm(torch.zeros(70)),
    "grouped x": lambda leaf, other: amd.int8_gemm_grouped(leaf, other, _route(6, 2, 3)),
    "grouped w": lambda leaf, other: amd.int8_gemm_grouped(other, leaf, _route(6, 2, 3)),
    "quantize out": lambda leaf, other: amd.int8_quantize(torch.zeros(6, 70), out=leaf),
}


@pytest.mark.parametrize("call", SCALES.values(), ids=SCALES.keys())
def test_scales_that_require_a_gradient_are_refused(call):
    """A learned scale would silently get none.  The flag may be set after the Int8Tensor was made."""
    leaf, other = _codes(6, 70), _codes(6, 70)
    leaf.scale.requires_grad_()
    with pytest.raises(ValueError, match="scale requires a gradient"):
        call(leaf, other)
    with torch.no_grad(), pytest.raises(Exception) as e:
        call(leaf, other)                      # past that check: these are not on the GPU
    assert "requires a gradient" not in str(e.value)


@pytest.mark.parametrize("call", SCALES.values(), ids=SCALES.keys())
def test_scales_with_a_tangent_are_refused(call):
    leaf, other = _codes(6, 70), _codes(6, 70)
    with forward_ad.dual_level(), torch.no_grad():
        leaf.scale = forward_ad.make_dual(leaf.scale, torch.ones(6))
        with pytest.raises(ValueError, match="scale has a forward-mode tangent"):
            call(leaf, other)


TANGENTS = {
    "quantize": lambda x: amd.int8_quantize(x),
    "linear": lambda x: amd.int8_linear(x, _codes(6, 8)),
    "gather": lambda x: amd.moe_gather(x, _route(4, 2, 3)),
    "combine": lambda x: amd.moe_combine(x, _route(2, 2, 3)),
    "gather_grad": lambda x: amd.moe_gather_grad(x, _route(2, 2, 3)),
    "combine_grad dy": lambda x: amd.moe_combine_grad(x, torch.zeros(8, 8), _route(4, 2, 3)),
}


@pytest.mark.parametrize("call", TANGENTS.values(), ids=TANGENTS.keys())
def test_values_with_a_tangent_are_refused(call):
    """The result would have none, in silence.  torch.no_grad() leaves forward mode on."""
    x = torch.zeros(4, 8)
    for context in (torch.enable_grad, torch.no_grad):
        with forward_ad.dual_level(), context():
            with pytest.raises(ValueError, match="forward-mode tangent"):
                call(forward_ad.make_dual(x, torch.ones(4, 8)))
            with pytest.raises(ValueError) as e:
                call(x)                        # a level alone is no reason
            assert "tangent" not in str(e.value)


# --- what the GPU tests reach ------------------------------------------------

# every variant of the dense products (plan, detail), splits of K as one, and of the grouped ones
DENSE = ({(-2, 4), (-2, 8), (-2, 11), (-1, 4), (-1, 8), (-1, 22)} | {(i, "whole K") for i in range(5)} |
         {(i, "split K") for i in range(5)} | {(5, shares) for shares in (1, 2, 3, 5)})
GROUPED = {(-1, 4), (-1, 8), (-1, 22)} | {(i, "whole K") for i in range(5)} | {(5, 1)}


def _variant(plan, detail):
    return (plan, detail) if plan < 0 or plan == 5 else (plan, "split K" if detail > 1 else "whole K")


def test_the_gpu_tests_reach_every_variant(lib):
    """A rule that is measured anew may send their sizes elsewhere; then they need others."""
    sizes = test_gpu_int8.TILINGS + [size for _, size in on_gpu.KERNELS]
    assert {_variant(*on_gpu.plan(*s)) for s in sizes} >= DENSE
    # (that of test_gpu_int8.py lies in the test's marks)
    marks = test_gpu_int8.test_gemm_grouped_tilings.pytestmark
    sizes = [m.args[1] for m in marks if m.name == "parametrize"][0] + [size for _, size in on_gpu.GROUPED]
    assert {_variant(*on_gpu.plan(rows, N, K, E)) for rows, E, N, K in sizes} >= GROUPED
    assert {on_gpu.plan(T * k, N, K, E)[0] for T, k, E, N, K in on_gpu.ABSENT} >= {-1, 0, 2, 4, 5}
    assert all(on_gpu.plan(*s)[1] > 1 for s in on_gpu.SPLITS)
    assert {on_gpu.plan(*s)[0] for s in on_gpu.SPLITS} == set(range(5))


def test_plan_arguments(lib):
    a, b = C.c_int32(), C.c_int32()
    ask = lambda M=4, N=8, K=64, E=0, a=C.byref(a), b=C.byref(b): lib.nf4_probe_int8_plan(M, N, K, E, 0, a, b)  # noqa: E731
    assert ask() == 0 and (a.value, b.value) == (-1, 4)
    for bad in (dict(M=0), dict(N=0), dict(K=-1), dict(E=-1), dict(a=None), dict(b=None)):
        assert ask(**bad) == EINVAL
    for large in (dict(M=1 << 31), dict(N=1 << 31), dict(K=131072), dict(E=1025)):
        assert ask(**large) == 2
