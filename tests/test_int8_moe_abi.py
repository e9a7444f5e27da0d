"""include/int8.h and include/moe.h without a GPU: what they declare is
exported and bound, host-side validation refuses bad arguments before anything
is launched, and the binding refuses tensors it cannot take."""
import ctypes as C
import os
import re

import pytest
import torch

import w4a16_gemv_amd as amd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, EUNSUPPORTED = 0, 1, 2
P = C.c_void_p(0x1000)          # never dereferenced: validation fails first
BIG = 1 << 62                   # a workspace size that is always enough


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(amd.LIB_PATH):
        from w4a16_gemv_amd import build
        build.build()
    return amd.load()


def test_every_declared_symbol_is_exported(lib):
    names = []
    for fn in ("int8.h", "moe.h"):
        src = open(os.path.join(ROOT, "include", fn), encoding="utf-8").read()
        src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
        names += re.findall(r"^(?:nf4_status|size_t|int64_t)\s+((?:int8|moe)_\w+)\s*\(", src, flags=re.M)
    assert len(names) == 13
    for name in names:
        assert hasattr(lib, name) and name in amd.EXPORTED, name


@pytest.mark.parametrize("K,pitch", [(-3, 0), (0, 0), (1, 64), (64, 64), (65, 128), (1501, 1536)])
def test_pitch(lib, K, pitch):
    assert lib.int8_pitch(K) == pitch == amd.int8_pitch(K)


def _quantize(lib, x=P, dt=0, rows=4, K=32, q=P, scale=P):
    return lib.int8_quantize(x, dt, rows, K, q, scale, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), EINVAL), (dict(K=-1), EINVAL), (dict(dt=3), EINVAL), (dict(dt=-1), EINVAL),
    (dict(x=None), EINVAL), (dict(q=None), EINVAL), (dict(scale=None), EINVAL),
    (dict(x=C.c_void_p(0x1001)), EINVAL), (dict(x=C.c_void_p(0x1002), dt=2), EINVAL),
    (dict(q=C.c_void_p(0x1008)), EINVAL), (dict(scale=C.c_void_p(0x1002)), EINVAL),
    (dict(rows=1 << 31), EUNSUPPORTED), (dict(K=1 << 31), EUNSUPPORTED),
    (dict(rows=0, x=None, q=None, scale=None), OK)])
def test_quantize_arguments(lib, kw, status):
    assert _quantize(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), EINVAL), (dict(K=-1), EINVAL), (dict(dt=3), EINVAL), (dict(out=None), EINVAL),
    (dict(q=None), EINVAL), (dict(scale=None), EINVAL), (dict(out=C.c_void_p(0x1001)), EINVAL),
    (dict(q=C.c_void_p(0x1008)), EINVAL), (dict(rows=1 << 31), EUNSUPPORTED),
    (dict(rows=0, q=None), OK), (dict(K=0, q=None), OK)])
def test_dequant_arguments(lib, kw, status):
    a = dict(q=P, scale=P, rows=4, K=32, out=P, dt=0, **{}) | kw
    assert lib.int8_dequant(a["q"], a["scale"], a["rows"], a["K"], a["out"], a["dt"], None) == status


PRODUCT = [
    (dict(M=-1), EINVAL), (dict(N=-1), EINVAL), (dict(K=-1), EINVAL), (dict(dt=3), EINVAL),
    (dict(wq=None), EINVAL), (dict(ws=None), EINVAL), (dict(y=None), EINVAL),
    (dict(wq=C.c_void_p(0x1008)), EINVAL), (dict(ws=C.c_void_p(0x1002)), EINVAL),
    (dict(y=C.c_void_p(0x1001)), EINVAL), (dict(y=C.c_void_p(0x1002), dt=2), EINVAL),
    (dict(work=C.c_void_p(0x1080)), EINVAL),
    (dict(K=131072), EUNSUPPORTED), (dict(N=1 << 31), EUNSUPPORTED), (dict(M=1 << 31), EUNSUPPORTED),
    (dict(M=0, xq=None, x=None, wq=None, y=None), OK), (dict(N=0, wq=None, ws=None, y=None), OK)]


@pytest.mark.parametrize("kw,status", PRODUCT + [
    (dict(xq=None), EINVAL), (dict(xs=None), EINVAL), (dict(xq=C.c_void_p(0x1008)), EINVAL),
    (dict(xs=C.c_void_p(0x1001)), EINVAL)])
def test_gemm_arguments(lib, kw, status):
    a = dict(xq=P, xs=P, wq=P, ws=P, M=4, N=8, K=64, y=P, dt=0, work=P) | kw
    assert lib.int8_gemm(a["xq"], a["xs"], a["wq"], a["ws"], a["M"], a["N"], a["K"], a["y"], a["dt"],
                         a["work"], BIG, None) == status


@pytest.mark.parametrize("kw,status", PRODUCT + [
    (dict(x=None), EINVAL), (dict(x=C.c_void_p(0x1001)), EINVAL), (dict(xdt=3), EINVAL),
    (dict(M=300, work=None), EINVAL), (dict(M=300, bytes=255), EINVAL)])
def test_linear_arguments(lib, kw, status):
    a = dict(x=P, xdt=0, wq=P, ws=P, M=4, N=8, K=64, y=P, dt=0, work=P, bytes=BIG) | kw
    assert lib.int8_linear(a["x"], a["xdt"], a["wq"], a["ws"], a["M"], a["N"], a["K"], a["y"], a["dt"],
                           a["work"], a["bytes"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), EINVAL), (dict(N=-1), EINVAL), (dict(K=-1), EINVAL), (dict(dt=3), EINVAL),
    (dict(E=-1), EINVAL), (dict(k=0), EINVAL), (dict(xr=-1), EINVAL), (dict(offsets=None), EINVAL),
    (dict(offsets=C.c_void_p(0x1002)), EINVAL), (dict(order=C.c_void_p(0x1002)), EINVAL),
    (dict(wq=None), EINVAL), (dict(ws=None), EINVAL), (dict(y=None), EINVAL), (dict(xq=None), EINVAL),
    (dict(xs=None), EINVAL), (dict(xq=C.c_void_p(0x1008)), EINVAL),
    (dict(wq=C.c_void_p(0x1008)), EINVAL), (dict(y=C.c_void_p(0x1001)), EINVAL),
    (dict(K=131072), EUNSUPPORTED), (dict(E=1025), EUNSUPPORTED), (dict(M=1 << 31), EUNSUPPORTED),
    (dict(xr=1 << 31), EUNSUPPORTED), (dict(N=1 << 31), EUNSUPPORTED),
    (dict(E=0, offsets=None), OK), (dict(M=0, y=None), OK), (dict(N=0, wq=None), OK)])
def test_grouped_arguments(lib, kw, status):
    a = dict(xq=P, xs=P, xr=4, order=P, k=2, wq=P, ws=P, offsets=P, E=3, M=8, N=8, K=64, y=P, dt=0) | kw
    assert lib.int8_gemm_grouped(a["xq"], a["xs"], a["xr"], a["order"], a["k"], a["wq"], a["ws"],
                                 a["offsets"], a["E"], a["M"], a["N"], a["K"], a["y"], a["dt"],
                                 None) == status


def test_workspace_sizes_are_zero_for_bad_sizes(lib):
    assert lib.int8_gemm_workspace_size(-1, 4, 4) == 0
    assert lib.int8_linear_workspace_size(-1, 4, 4) == 0
    assert lib.int8_linear_workspace_size(1 << 40, 4, 4) == 0
    assert lib.int8_linear_workspace_size(4, 4, 1 << 40) == 0
    assert lib.moe_sort_workspace_size(-1, 4, 4) == 0
    assert lib.moe_sort_workspace_size(1 << 40, 4, 4) == 0
    assert lib.moe_sort_workspace_size(8, 2, 4) == 0
    # a workspace of a large sort holds a count per workgroup and expert
    assert lib.moe_sort_workspace_size(1 << 20, 8, 64) >= 64 * 4


@pytest.mark.parametrize("kw,status", [
    (dict(bytes=3), EINVAL), (dict(T=-1), EINVAL), (dict(k=0), EINVAL), (dict(E=-1), EINVAL),
    (dict(ids=None), EINVAL), (dict(offsets=None), EINVAL), (dict(order=None), EINVAL),
    (dict(pos=None), EINVAL), (dict(ids=C.c_void_p(0x1004), bytes=8), EINVAL),
    (dict(offsets=C.c_void_p(0x1002)), EINVAL), (dict(work=C.c_void_p(0x1010)), EINVAL),
    (dict(T=1 << 16, work=None), EINVAL), (dict(T=1 << 16, wbytes=8), EINVAL),
    (dict(E=1025), EUNSUPPORTED), (dict(T=1 << 31), EUNSUPPORTED), (dict(T=1 << 29, k=3), EUNSUPPORTED)])
def test_sort_arguments(lib, kw, status):
    a = dict(ids=P, bytes=4, T=16, k=2, E=8, offsets=P, order=P, pos=P, work=P, wbytes=BIG) | kw
    assert lib.moe_sort(a["ids"], a["bytes"], a["T"], a["k"], a["E"], a["offsets"], a["order"], a["pos"],
                        a["work"], a["wbytes"], None) == status


MOVES = [(dict(T=-1), EINVAL), (dict(k=0), EINVAL), (dict(R=-1), EINVAL), (dict(H=-1), EINVAL),
         (dict(dt=3), EINVAL), (dict(pos=None), EINVAL), (dict(pos=C.c_void_p(0x1002)), EINVAL),
         (dict(T=1 << 31), EUNSUPPORTED), (dict(R=1 << 31), EUNSUPPORTED), (dict(H=1 << 31), EUNSUPPORTED),
         (dict(a=C.c_void_p(0x1001)), EINVAL), (dict(b=C.c_void_p(0x1002), dt=2), EINVAL),
         (dict(T=0, a=None, b=None, pos=None), OK)]


@pytest.mark.parametrize("kw,status", MOVES + [(dict(a=None), EINVAL), (dict(b=None), EINVAL),
                                               (dict(R=0, a=None, b=None), OK),
                                               (dict(H=0, a=None, b=None), OK)])
def test_gather_arguments(lib, kw, status):
    a = dict(a=P, dt=0, pos=P, T=4, k=2, R=8, H=16, b=P) | kw
    assert lib.moe_gather(a["a"], a["dt"], a["pos"], a["T"], a["k"], a["R"], a["H"], a["b"], None) == status


@pytest.mark.parametrize("kw,status", MOVES + [(dict(a=None), EINVAL), (dict(b=None), EINVAL),
                                               (dict(w=C.c_void_p(0x1002)), EINVAL),
                                               (dict(H=0, a=None, b=None), OK)])
def test_combine_arguments(lib, kw, status):
    a = dict(a=P, dt=0, w=P, pos=P, T=4, k=2, R=8, H=16, b=P) | kw
    assert lib.moe_combine(a["a"], a["dt"], a["w"], a["pos"], a["T"], a["k"], a["R"], a["H"], a["b"],
                           None) == status


@pytest.mark.parametrize("kw,status", MOVES + [(dict(a=None), EINVAL), (dict(g=None), EINVAL),
                                               (dict(w=C.c_void_p(0x1002)), EINVAL),
                                               (dict(dw=C.c_void_p(0x1002)), EINVAL),
                                               (dict(b=None, dw=None), OK)])
def test_combine_grad_arguments(lib, kw, status):
    a = dict(g=P, a=P, dt=0, w=P, pos=P, T=4, k=2, R=8, H=16, b=P, dw=P) | kw
    assert lib.moe_combine_grad(a["g"], a["a"], a["dt"], a["w"], a["pos"], a["T"], a["k"], a["R"], a["H"],
                                a["b"], a["dw"], None) == status


def test_binding_refuses_tensors_off_the_gpu():
    codes, scale = torch.zeros(4, 64, dtype=torch.int8), torch.ones(4)
    with pytest.raises(ValueError, match="on the GPU"):
        amd.Int8Tensor(codes, scale, 60)
    with pytest.raises(ValueError, match="on the GPU"):
        amd.int8_quantize(torch.zeros(4, 64))
    with pytest.raises(ValueError, match="on the GPU"):
        amd.moe_sort(torch.zeros(4, 2, dtype=torch.int32), 8)
    with pytest.raises(ValueError, match="on the GPU"):
        amd.MoeRoute(torch.zeros(9, dtype=torch.int32), torch.zeros(8, dtype=torch.int32),
                     torch.zeros(4, 2, dtype=torch.int32))


def test_binding_refuses_shapes_and_types_first():
    codes, scale = torch.zeros(4, 64, dtype=torch.int8), torch.ones(4)
    for K in (-1, 0, 65, 200):
        with pytest.raises(ValueError):
            amd.Int8Tensor(codes, scale, K)
    with pytest.raises(ValueError, match="bfloat16, float16 or float32"):
        amd.int8_quantize(torch.zeros(4, 64, dtype=torch.float64))
    with pytest.raises(ValueError, match="dimension"):
        amd.int8_quantize(torch.tensor(1.0))
    with pytest.raises(ValueError, match="requires a gradient"):
        amd.int8_quantize(torch.zeros(4, 64, requires_grad=True))
    with torch.no_grad(), pytest.raises(ValueError, match="on the GPU"):
        amd.int8_quantize(torch.zeros(4, 64, requires_grad=True))
    for ids in (torch.zeros(4, dtype=torch.int32), torch.zeros(4, 0, dtype=torch.int32)):
        with pytest.raises(ValueError, match="top_k"):
            amd.moe_sort(ids, 8)
    with pytest.raises(ValueError, match="negative"):
        amd.moe_sort(torch.zeros(4, 2, dtype=torch.int32), -1)
