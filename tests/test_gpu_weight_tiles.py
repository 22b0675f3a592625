"""The weight's gradient of vr_linear_xent around the number of tokens where it
leaves its tiles through shared memory (an epilogue that stores tiles and loads
none) or row by row."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import double_binary_tree_gb300 as vr  # noqa: E402
from tests import operator_refs as refs  # noqa: E402
from tests.test_gpu_linear_xent import DT, IGNORE, call, compare, make  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [1, 1023, 1024, 1025])
@pytest.mark.parametrize("D,V", [(64, 1000), (1032, 260), (1048, 3001)])
def test_the_weight_gradient_alone(D, V, T, dtype):
    code, ty = DT[dtype]
    scale = 64.0 * T if dtype == "fp16" else 1.0
    h, w, y = make(T, D, V, ty, 31)
    got = call(h, w, y, code, scale=scale, dh=False)
    assert vr.vr_stream_status() == 0
    compare(got, refs.xent(h, w, y, IGNORE, True, scale), ty)
