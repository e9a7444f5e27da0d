"""include/mxfp4.h without a GPU: what it declares is exported and bound,
host-side validation refuses bad arguments before anything is launched, the
binding refuses tensors it cannot take, and the GPU tests reach every kernel."""
import ctypes as C
import os
import re

import pytest
import torch
from torch.autograd import forward_ad

import w4a16_gemv_amd as amd
from tests import test_gpu_mxfp4 as on_gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, EUNSUPPORTED = 0, 1, 2
P = C.c_void_p(0x1000)          # never dereferenced: validation fails first
BIG = 1 << 62                   # a workspace size that is always enough


def at(address):
    return C.c_void_p(address)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(amd.LIB_PATH):
        from w4a16_gemv_amd import build
        build.build()
    return amd.load()


def test_every_declared_symbol_is_exported(lib):
    src = open(os.path.join(ROOT, "include", "mxfp4.h"), encoding="utf-8").read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = re.findall(r"^(?:nf4_status|size_t|int64_t)\s+(mxfp4_\w+)\s*\(", src, flags=re.M)
    assert len(names) == 12
    for name in names:
        assert hasattr(lib, name) and name in amd.EXPORTED, name


@pytest.mark.parametrize("K,pitch", [(-3, 0), (0, 0), (1, 64), (128, 64), (129, 128), (1501, 768), (4096, 2048)])
def test_pitch(lib, K, pitch):
    assert lib.mxfp4_pitch(K) == pitch == amd.mxfp4_pitch(K)


@pytest.mark.parametrize("rows,K,size", [(0, 64, 0), (3, 0, 0), (-1, 64, 0), (1, 1, 256), (32, 256, 256), (33, 256, 512),
                                         (32, 257, 512), (100, 1501, 4 * 6 * 256)])
def test_scale_size(lib, rows, K, size):
    assert lib.mxfp4_scale_size(rows, K) == size == amd.mxfp4_scale_size(rows, K)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), EINVAL), (dict(K=-1), EINVAL), (dict(dt=3), EINVAL), (dict(dt=-1), EINVAL),
    (dict(x=None), EINVAL), (dict(q=None), EINVAL), (dict(s=None), EINVAL),
    (dict(x=at(0x1001)), EINVAL), (dict(x=at(0x1002), dt=2), EINVAL),
    (dict(q=at(0x1008)), EINVAL), (dict(s=at(0x1004)), EINVAL),
    (dict(rows=1 << 31), EUNSUPPORTED), (dict(K=1 << 31), EUNSUPPORTED), (dict(rows=1 << 30, K=300), EUNSUPPORTED),
    (dict(rows=0, x=None, q=None, s=None), OK), (dict(K=0, x=None, q=None, s=None), OK)])
def test_quantize_and_dequant_arguments(lib, kw, status):
    a = dict(x=P, dt=0, rows=4, K=32, q=P, s=P) | kw
    assert lib.mxfp4_quantize(a["x"], a["dt"], a["rows"], a["K"], a["q"], a["s"], None) == status
    assert lib.mxfp4_dequant(a["q"], a["s"], a["rows"], a["K"], a["x"], a["dt"], None) == status


WEIGHTS = [
    (dict(M=-1), EINVAL), (dict(N=-1), EINVAL), (dict(K=-1), EINVAL), (dict(dt=3), EINVAL),
    (dict(wq=None), EINVAL), (dict(ws=None), EINVAL), (dict(y=None), EINVAL),
    (dict(wq=at(0x1008)), EINVAL), (dict(ws=at(0x1004)), EINVAL),
    (dict(y=at(0x1001)), EINVAL), (dict(y=at(0x1002), dt=2), EINVAL),
    (dict(K=(1 << 20) + 1), EUNSUPPORTED), (dict(N=1 << 31), EUNSUPPORTED),
    (dict(M=0, xq=None, x=None, wq=None, y=None), OK), (dict(N=0, wq=None, ws=None, y=None), OK)]
PRODUCT = WEIGHTS + [(dict(work=at(0x1080)), EINVAL), (dict(M=1 << 31), EUNSUPPORTED)]


@pytest.mark.parametrize("kw,status", PRODUCT + [
    (dict(xq=None), EINVAL), (dict(xs=None), EINVAL), (dict(xq=at(0x1008)), EINVAL), (dict(xs=at(0x1001)), EINVAL)])
def test_gemm_arguments(lib, kw, status):
    a = dict(xq=P, xs=P, wq=P, ws=P, M=4, N=8, K=64, y=P, dt=0, work=P) | kw
    assert lib.mxfp4_gemm(a["xq"], a["xs"], a["wq"], a["ws"], a["M"], a["N"], a["K"], a["y"], a["dt"],
                          a["work"], BIG, None) == status


@pytest.mark.parametrize("kw,status", PRODUCT + [
    (dict(x=None), EINVAL), (dict(x=at(0x1001)), EINVAL), (dict(xdt=3), EINVAL),
    (dict(M=3000, N=3000, work=None), EINVAL), (dict(M=3000, N=3000, bytes=255), EINVAL)])
def test_linear_arguments(lib, kw, status):
    a = dict(x=P, xdt=0, wq=P, ws=P, M=4, N=8, K=64, y=P, dt=0, work=P, bytes=BIG) | kw
    assert lib.mxfp4_linear(a["x"], a["xdt"], a["wq"], a["ws"], a["M"], a["N"], a["K"], a["y"], a["dt"],
                            a["work"], a["bytes"], None) == status


@pytest.mark.parametrize("kw,status", WEIGHTS + [
    (dict(M=17), EINVAL), (dict(x=None), EINVAL), (dict(x=at(0x1001)), EINVAL), (dict(xdt=3), EINVAL)])
def test_gemv_arguments(lib, kw, status):
    a = dict(x=P, xdt=0, wq=P, ws=P, M=4, N=8, K=64, y=P, dt=0) | kw
    assert lib.mxfp4_gemv(a["x"], a["xdt"], a["wq"], a["ws"], a["M"], a["N"], a["K"], a["y"], a["dt"], None) == status


@pytest.mark.parametrize("kw,status", WEIGHTS + [
    (dict(E=-1), EINVAL), (dict(k=0), EINVAL), (dict(xr=-1), EINVAL), (dict(offsets=None), EINVAL),
    (dict(offsets=at(0x1002)), EINVAL), (dict(order=at(0x1002)), EINVAL), (dict(xq=None), EINVAL),
    (dict(xs=None), EINVAL), (dict(xq=at(0x1008)), EINVAL), (dict(xs=at(0x1008)), EINVAL),
    (dict(E=1025), EUNSUPPORTED), (dict(M=1 << 31), EUNSUPPORTED), (dict(xr=1 << 31), EUNSUPPORTED),
    (dict(N=1 << 30, E=3), EUNSUPPORTED), (dict(E=0, offsets=None), OK)])
def test_grouped_arguments(lib, kw, status):
    a = dict(xq=P, xs=P, xr=4, order=P, k=2, wq=P, ws=P, offsets=P, E=3, M=8, N=8, K=64, y=P, dt=0) | kw
    assert lib.mxfp4_gemm_grouped(a["xq"], a["xs"], a["xr"], a["order"], a["k"], a["wq"], a["ws"], a["offsets"], a["E"],
                                  a["M"], a["N"], a["K"], a["y"], a["dt"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), EINVAL), (dict(k=0), EINVAL), (dict(E=-1), EINVAL), (dict(H=-1), EINVAL), (dict(F=-1), EINVAL),
    (dict(dt=3), EINVAL), (dict(bytes=2), EINVAL), (dict(x=None), EINVAL), (dict(y=None), EINVAL),
    (dict(ids=None), EINVAL), (dict(ids=at(0x1004), bytes=8), EINVAL), (dict(x=at(0x1001)), EINVAL),
    (dict(y=at(0x1002), dt=2), EINVAL), (dict(w=at(0x1002)), EINVAL), (dict(work=at(0x1010)), EINVAL),
    (dict(work=None), EINVAL), (dict(wbytes=255), EINVAL), (dict(w1q=None), EINVAL), (dict(w1s=None), EINVAL),
    (dict(w2q=None), EINVAL), (dict(w2s=None), EINVAL), (dict(w1q=at(0x1008)), EINVAL), (dict(w2s=at(0x1008)), EINVAL),
    (dict(T=65), EUNSUPPORTED), (dict(k=33), EUNSUPPORTED), (dict(E=1025), EUNSUPPORTED),
    (dict(H=(1 << 20) + 1), EUNSUPPORTED), (dict(F=(1 << 20) + 1), EUNSUPPORTED),
    (dict(H=1 << 20, E=1024, F=1 << 20), EUNSUPPORTED), (dict(E=1024, F=1 << 20), EUNSUPPORTED),
    (dict(T=0, x=None, y=None, ids=None), OK), (dict(H=0, x=None, y=None), OK)])
def test_moe_mlp_arguments(lib, kw, status):
    a = dict(x=P, dt=0, w1q=P, w1s=P, w2q=P, w2s=P, ids=P, bytes=4, w=P, T=3, k=2, E=8, H=64, F=32, gated=1, y=P, work=P,
             wbytes=BIG) | kw
    assert lib.mxfp4_moe_mlp(a["x"], a["dt"], a["w1q"], a["w1s"], a["w2q"], a["w2s"], a["ids"], a["bytes"], a["w"], a["T"],
                             a["k"], a["E"], a["H"], a["F"], a["gated"], a["y"], a["work"], a["wbytes"], None) == status


def test_workspace_sizes(lib):
    for f in (lib.mxfp4_gemm_workspace_size, lib.mxfp4_linear_workspace_size):
        for sizes in ((-1, 4, 4), (4, 4, 1 << 40), (1 << 40, 4, 4), (0, 4, 4), (4, 0, 4), (4, 4, 0)):
            assert f(*sizes) == 0
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    for M, N, K in ((3000, 3000, 64), (333, 4099, 1501), (8192, 11008, 4096)):
        need = up(M * amd.mxfp4_pitch(K)) + up(amd.mxfp4_scale_size(M, K))
        assert lib.mxfp4_linear_workspace_size(M, N, K) == need + lib.mxfp4_gemm_workspace_size(M, N, K)
        assert lib.mxfp4_linear(P, 0, P, P, M, N, K, P, 0, P, need - 1, None) == EINVAL
    assert lib.mxfp4_linear_workspace_size(1, 4096, 4096) == 0
    size = lib.mxfp4_moe_mlp_workspace_size
    for bad in ((65, 2, 4, 64, 64, 0), (4, 33, 4, 64, 64, 0), (-1, 2, 4, 64, 64, 0), (4, 2, 4, 64, 64, 3),
                (4, 2, 1025, 64, 64, 0), (4, 2, 4, (1 << 20) + 1, 64, 0), (4, 2, 4, 64, -1, 0)):
        assert size(*bad) == 0
    # what lies between the products (two bf16 numbers of each, three for fp32)
    assert size(3, 2, 4, 8192, 129, 0) == 6 * 2 * 256 * 2 and size(3, 2, 4, 8192, 129, 2) == 6 * 3 * 256 * 2


def _codes(rows, K):
    """An Mxfp4Tensor off the GPU, which only a call that has passed its first checks would notice."""
    t = amd.Mxfp4Tensor.__new__(amd.Mxfp4Tensor)
    t.data = torch.zeros(rows, amd.mxfp4_pitch(K), dtype=torch.uint8)
    t.scale, t.K = torch.zeros(amd.mxfp4_scale_size(rows, K), dtype=torch.uint8), K
    return t


def _route(T, k, E):
    r = amd.MoeRoute.__new__(amd.MoeRoute)
    r.offsets = torch.zeros(E + 1, dtype=torch.int32)
    r.order, r.pos = torch.zeros(T * k, dtype=torch.int32), torch.zeros(T, k, dtype=torch.int32)
    return r


def test_binding_refuses_shapes_and_types():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    for data, scale, K in ((u8(4, 64), u8(256), 129), (u8(4, 64), u8(255), 128), (u8(4, 64), u8(1, 256), 128),
                           (u8(64), u8(256), 128), (u8(4, 64), u8(256), -1)):
        with pytest.raises(ValueError, match="must"):
            amd.Mxfp4Tensor(data, scale, K)
    with pytest.raises(ValueError, match="on the GPU"):
        amd.Mxfp4Tensor(u8(4, 64), u8(256), 100)
    blocks = amd.Mxfp4Tensor.from_blocks
    for codes, scales, K in ((u8(4, 3, 8), u8(4, 3), None), (u8(4, 48), u8(4, 3), None), (u8(4, 3, 16), u8(4, 2), None),
                             (u8(4, 3, 16), u8(4, 3), 97), (u8(4, 3, 16), u8(4, 3), 64),
                             (u8(4, 3, 16).char(), u8(4, 3), None), (u8(4, 3, 16), u8(4, 3), 90)):
        with pytest.raises(ValueError):
            blocks(codes, scales, K)
    with pytest.raises(ValueError, match="bfloat16, float16 or float32"):
        amd.mxfp4_quantize(torch.zeros(4, 64, dtype=torch.float64))
    with pytest.raises(ValueError, match="dimension"):
        amd.mxfp4_quantize(torch.tensor(1.0))
    with pytest.raises(ValueError, match="x has K=64, w has K=65"):
        amd.mxfp4_gemm(_codes(4, 64), _codes(4, 65))
    for f in (amd.mxfp4_linear, amd.mxfp4_gemv):
        with pytest.raises(ValueError, match=r"x must be \[M, 64\]"):
            f(torch.zeros(4, 65), _codes(4, 64))
    with pytest.raises(ValueError, match="not a multiple of 3 experts"):
        amd.mxfp4_gemm_grouped(_codes(4, 64), _codes(4, 64), _route(4, 2, 3))
    with pytest.raises(ValueError, match="x has 5 rows, expected 4"):
        amd.mxfp4_gemm_grouped(_codes(5, 64), _codes(6, 64), _route(4, 2, 3))


CALLS = {
    "quantize": lambda x: amd.mxfp4_quantize(x),
    "linear": lambda x: amd.mxfp4_linear(x, _codes(6, 64)),
    "gemv": lambda x: amd.mxfp4_gemv(x, _codes(6, 64)),
    "mlp": lambda x: amd.mxfp4_moe_mlp(x, _codes(6, 64), _codes(128, 3), torch.zeros(4, 1, dtype=torch.int32)),
    "method": lambda x: _codes(6, 64).gemm(x),
}


@pytest.mark.parametrize("call", CALLS.values(), ids=CALLS.keys())
def test_gradients_and_tangents_are_refused(call):
    """The result would have none, in silence."""
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="requires a gradient"):
        call(x.clone().requires_grad_())
    with forward_ad.dual_level(), torch.no_grad():
        with pytest.raises(ValueError, match="forward-mode tangent"):
            call(forward_ad.make_dual(x, torch.ones(4, 64)))
    with torch.no_grad(), pytest.raises(ValueError, match="on the GPU"):
        call(x.clone().requires_grad_())


def test_plan_arguments(lib):
    a, b = C.c_int32(), C.c_int32()
    ask = lambda M=4, N=8, K=64, E=0, a=C.byref(a), b=C.byref(b): lib.nf4_probe_mxfp4_plan(M, N, K, E, 0, a, b)  # noqa: E731
    assert ask() == 0 and (a.value, b.value) == (-1, 4)
    for bad in (dict(M=0), dict(N=0), dict(K=-1), dict(E=-2), dict(a=None), dict(b=None)):
        assert ask(**bad) == EINVAL
    for large in (dict(M=1 << 31), dict(N=1 << 31), dict(K=(1 << 20) + 1), dict(E=1025)):
        assert ask(**large) == 2


def _variant(plan, detail):
    return (plan, detail) if plan < 0 or plan == 5 else (plan, "split K" if detail > 1 else "whole K")


def test_the_gpu_tests_reach_every_variant(lib):
    """A rule that is measured anew may send their sizes elsewhere; then they need others."""
    reached = {_variant(*on_gpu.plan(M, N, K, -1)) for M, N, K in on_gpu.LINEAR}
    want = {(-1, u) for u in (4, 8, 12, 22, -4, -2, -1)}
    assert reached >= want, want - reached
    reached = {_variant(*on_gpu.plan(M, N, K)) for M, N, K in on_gpu.DENSE}
    want = {(-1, 4)} | {(i, s) for i in range(5) for s in ("whole K", "split K")}
    want |= {(5, shares) for shares in (1, 2, 3, 4, 5)}
    assert reached >= want, want - reached
    reached = {_variant(*on_gpu.plan(T * k, N, K, E)) for T, k, E, N, K in on_gpu.GROUPED}
    want = {(-1, u) for u in (-4, -2, -1)} | {(i, "whole K") for i in (0, 2, 4)} | {(5, 1)}
    assert reached >= want, want - reached
