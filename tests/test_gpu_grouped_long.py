"""Long sums of the grouped products, which are taken in chunks: every kind of
tile they have, with differences that a lost, doubled or misplaced chunk makes."""

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import double_binary_tree_gb300 as vr  # noqa: E402
from tests import more_refs, operator_refs as refs  # noqa: E402
from tests.test_gpu_grouped import Case, untouched  # noqa: E402
from tests.test_gpu_operator_memory import Arena  # noqa: E402

# sums longer than these take chunks of 2048
LONG = {"fp16": 32768, "bf16": 262144}


def near(got, want, case, what):
    """In the 2-norm within the largest rounding to the type (one each, 1 / sqrt(3)
    of that on average at most, leaves room for what sums in 32 bits are off by).  A
    lost chunk of 2048 of 33000 terms is a quarter of the norm, one of 263000 a
    twelfth."""
    assert refs.norm_error(got, want) <= refs.U_T[case.ty], what


def linear(case):
    arena = Arena()
    got = case.linear(arena=arena)
    assert vr.vr_stream_status() == 0 and arena.intact()
    want, bound = more_refs.grouped(case.x, case.w, case.counts)
    near(got[:case.used], want[:case.used], case, "out")
    refs.assert_close(got[:case.used], want[:case.used], bound[:case.used], case.ty, "out")
    assert untouched(got[case.used:])
    assert torch.equal(got[:case.used], case.linear()[:case.used])


def gradients(case, dx=True, dw=True):
    arena = Arena()
    gx, gw = case.grad(arena=arena, dx=dx, dw=dw)
    assert vr.vr_stream_status() == 0 and arena.intact()
    wx, bx, ww, bw = more_refs.grouped_grad(case.dy, case.x, case.w, case.counts)
    again = case.grad(dx=dx, dw=dw)
    if dx:
        near(gx[:case.used], wx[:case.used], case, "dX")
        refs.assert_close(gx[:case.used], wx[:case.used], bx[:case.used], case.ty, "dX")
        assert untouched(gx[case.used:])
        assert torch.equal(gx[:case.used], again[0][:case.used])
    if dw:
        for e in range(case.E):
            near(gw[e], ww[e], case, "dW of group %d" % e)
        refs.assert_close(gw, ww, bw, case.ty, "dWeight")
        assert torch.equal(gw, again[1])


# few rows a group, one CTA, pairs of them (more than 128 rows of a weight)
FORWARD = [([7, 3], 16), ([40, 66], 8), ([600], 8), ([40, 0, 100, 65], 264), ([300, 257], 1000)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("counts,small", FORWARD, ids=lambda x: str(x).replace(" ", ""))
def test_rows(counts, small, dtype):
    n = LONG[dtype] + 8 * 37
    if dtype == "bf16" and small > 264:
        small = 392
    linear(Case(counts, n, small, dtype, spare=3, seed=small))
    gradients(Case(counts, small, n, dtype, spare=3, seed=small), dw=False)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("K,N", [(24, 32), (72, 128), (200, 136), (264, 520), (129, 131)])
@pytest.mark.parametrize("ends", [[0.3, 0.0, 0.4, 0.01, 0.2901], [0.999, 0.002], [0.1] * 11])
def test_weights(ends, K, N, dtype):
    """Groups whose ends are no multiples of anything, empty ones, and NaN in
    the rows behind the last."""
    counts = [int(LONG[dtype] * x) | 1 if x else 0 for x in ends]
    case = Case(counts, K, N, dtype, spare=70, seed=K)
    assert case.rows > LONG[dtype]
    case.x[case.used:] = math.nan
    case.dy[case.used:] = math.inf
    gradients(case, dx=K > 64)
    # (dX's sums are short)
