"""vr_balance_loss over the range of its logits' types: rows of large equal or
far apart values are as exact as rows near zero."""

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import double_binary_tree_gb300 as vr  # noqa: E402
from tests import operator_refs as refs  # noqa: E402
from tests.test_gpu_balance import DT, call, draw  # noqa: E402


def bounds(x, f, coef, n):
    """Loss, gradients and bounds of an fp32 evaluation of exp(x - top): the
    difference is rounded once, its product with log2 e once, ex2 to 2 ulp
    (2^-22), the sums of E terms and the divisions to (E + 16) 2^-24."""
    E = x.shape[1]
    p = torch.softmax(x, 1)
    gap = (x.amax(1, keepdim=True) - x).clamp(max=200.0)   # beyond it both are 0
    rel = (3 * gap + 8 + E + 16) * refs.U32
    dot = (p * f).sum(1, keepdim=True)
    factor = coef * E / n
    loss = factor * float((f * p.sum(0)).sum())
    bound = factor * p * (f + dot) * 2 * (rel + rel.amax())
    # each p is off by rel p at most, E n of them are summed
    loss_bound = factor * float((f * (p * rel).sum(0)).sum()) + loss * (E + n + 16) * refs.U32
    return loss, loss_bound, factor * p * (f - dot), bound


@pytest.mark.parametrize("tokens", [9, 3000])      # one launch, and two
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("value", [1e4, 1e6, 3e7, 1e9, 1e10, 1e20, 1e30, 2e37])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_rows_of_large_logits(sign, value, dtype, tokens):
    """A router that masks with a large negative constant masks all experts of
    a token: equal probabilities.  And half of them at twice the distance."""
    code, ty = DT[dtype]
    E, k = 32, 2
    logits = draw(1, tokens, E, ty, 20)
    v = sign * value
    logits[0][1::7] = v
    logits[0][2::7] = v
    logits[0][2::7, 16:] = v - value
    if dtype == "fp32" and value <= 1e6:             # differences that count
        logits[0][3::7] = v - 0.25 * torch.arange(E, device="cuda")
    loss, counts, picks, out = call(logits, None, k, code, 1.0)
    assert vr.vr_stream_status() == 0
    assert picks[0][1].tolist() == [0, 1] and picks[0][2].tolist() == [0, 1]
    f = counts.cpu().double() / (k * tokens)
    want, loss_bound, grads, bound = bounds(logits[0].cpu().double(), f, 1.0, tokens)
    assert math.isfinite(float(loss)) and abs(float(loss) - want) <= loss_bound
    refs.assert_close(out[0].cpu(), grads, bound, ty, "dlogits")
