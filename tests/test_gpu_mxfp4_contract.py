"""What include/mxfp4.h promises beside the values themselves: rows that leave each other alone."""
import pytest
import torch

import w4a16_gemv_amd as amd
from tests.test_gpu_mxfp4 import F32, TYPES, dev, exactly, random_rows, same
from tests.test_gpu_mxfp4_mlp import check, make

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    amd.load()


# --- rows whose step of sixteen units has no room in LDS ------------------------

# 14 to 16 rows in fp16 or 10 to 16 in fp32 of 257 to 512 elements, where four waves share a row
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K", [(16, 40, 400), (14, 100, 512), (10, 33, 257), (12, 700, 384), (16, 3000, 500)])
def test_gemv_nan_stays_in_its_row(M, N, K, dtype):
    """Rows stand side by side in LDS; what a wave reads past one must not be the next."""
    w, wt = random_rows(N, N, K, 127, 129)
    x = torch.randint(-8, 9, (M, K), device=dev()).to(dtype)
    want = exactly(x.double(), w, 0.5, F32)
    assert same(amd.mxfp4_gemv(x, wt, out_dtype=F32), want)
    for row in (1, M // 2, M - 1):
        hurt, some = x.clone(), want.clone()
        hurt[row], some[row] = NAN, NAN
        assert same(amd.mxfp4_gemv(hurt, wt, out_dtype=F32), some)


@pytest.mark.parametrize("gated", (True, False), ids=("gated", "plain"))
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,k,E,H,F", [(20, 3, 5, 257, 41), (16, 1, 1, 400, 60), (64, 2, 3, 512, 33), (13, 2, 2, 384, 64)])
def test_mlp_rows_of_257_to_512(T, k, E, H, F, dtype, gated):
    x, w1, t1, w2, t2, ids, weights = make(T + F, T, k, E, H, F, gated, dtype)
    check(amd.mxfp4_moe_mlp(x, t1, t2, ids, weights), x, w1, w2, ids, weights, E, gated)
