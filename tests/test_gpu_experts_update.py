"""The example's update of the experts, against the Newton-Schulz steps of its
momentum in 64 bits."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

from tests import operator_refs as refs  # noqa: E402
from tests.test_gpu_experts_step import _example  # noqa: E402


def test_experts_move_by_the_orthogonalised_momentum():
    """In the first step the momentum is the gradient.  An update of zero, or of
    another size or direction, fails."""
    ex = _example()
    step = ex.Step(seed=6)
    tokens, targets = step.batch()
    _, _, counts, grads = step.gradients(tokens, targets)
    assert int(counts.min()) > 0
    before = [w.clone() for w in (step.up, step.down)]
    step.update(grads, lr=0.01, expert_lr=0.02)
    for w, old, g in zip((step.up, step.down), before, grads[2:]):
        for e in range(ex.EXPERTS):
            want = refs.orthogonalize(g[e], 5, None, 1e-7, 1.0)
            move = (old[e].double() - w[e].double()) / 0.02
            norm = float(want.norm())
            # the operator's own error, and the rounding of w - step to bf16: half a
            # step of each entry, 2^-8 of it at most
            limit = refs.ortho_tolerance(torch.bfloat16, norm, 3.4445 ** 5) * norm
            limit += 2.0 ** -8 * float(w[e].double().norm()) / 0.02
            assert limit < 0.7 * norm  # (no move at all is off by the norm)
            assert float((move - want).norm()) <= limit, e
