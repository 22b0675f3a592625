"""vr_orthogonalize of matrices with few rows or columns: a rounding in one of a few
directions does not average out over the others."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import double_binary_tree_gb300 as vr  # noqa: E402
from tests.test_gpu_orthogonalize import DT, call, compare, make  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("m", [1, 2, 3, 4, 6, 8, 12, 15, 16, 17])
@pytest.mark.parametrize("n", [0, 1, 30, 500, 2100])    # more columns than rows
def test_few_rows_or_columns(n, m, dtype):
    """Each of 32 matrices on its own, as rows or as columns."""
    code, ty = DT[dtype]
    rows, cols = (m, m + n) if n % 3 else (m + n, m)
    ms = make(32, rows, cols, ty, 100 * m + n)
    got = call(ms, code)
    assert vr.vr_stream_status() == 0
    compare(got, ms, ty)
