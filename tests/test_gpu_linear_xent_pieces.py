"""vr_linear_xent with the vocabulary in pieces: because the workspace is the least
one, or because the tokens are many."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import double_binary_tree_gb300 as vr  # noqa: E402
from tests import operator_refs as refs  # noqa: E402
from tests.test_gpu_linear_xent import DT, IGNORE, call, compare, make  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,D,V", [(600, 640, 240000), (300, 512, 500000), (129, 160, 800001)])
def test_the_least_workspace_takes_pieces(T, D, V, dtype):
    code, ty = DT[dtype]
    h, w, y = make(T, D, V, ty, 51, ignored=0.2)
    full, least = (vr.vr_linear_xent_workspace_bytes(h, D, w, D, T, D, V, code, g) for g in (1, 2))
    # else the numerators were kept, and both calls were the same
    assert least < full
    scale = 64.0 * T if dtype == "fp16" else 1.0
    want = refs.xent(h, w, y, IGNORE, True, scale)
    kept = call(h, w, y, code, scale=scale)
    pieces = call(h, w, y, code, scale=scale, least=True)
    assert vr.vr_stream_status() == 0
    compare(kept, want, ty)
    compare(pieces, want, ty)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,D,V", [
    (2600, 65, 60000),     # rows that are no 16-byte units, through the padded weight
    (1024, 72, 140000), (1025, 72, 140000), (3000, 264, 50304)])
def test_more_tokens_than_dim(T, D, V, dtype):
    code, ty = DT[dtype]
    h, w, y = make(T, D, V, ty, 52, ignored=0.3)
    scale = 64.0 * T if dtype == "fp16" else 1.0
    got = call(h, w, y, code, scale=scale)
    assert vr.vr_stream_status() == 0
    compare(got, refs.xent(h, w, y, IGNORE, True, scale), ty)
    for dh, dw in ((True, False), (False, True)):
        part = call(h, w, y, code, scale=scale, dh=dh, dw=dw)
        assert all(p is None or torch.equal(a, p) for a, p in zip(got, part))
