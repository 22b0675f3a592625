"""The example's data-parallel step: the losses, the AllReduce of their
gradients and the orthogonalised update, run together."""

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

from tests.conftest import ROOT  # noqa: E402


def _example():
    path = os.path.join(ROOT, "examples", "training_step.py")
    spec = importlib.util.spec_from_file_location("training_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_the_losses_fall():
    history = _example().main(30)
    first, last = history[0], history[-1]
    assert last[0] < 0.8 * first[0]
    assert last[1] < first[1]


def test_the_first_step_against_autograd():
    """The gradients that the step makes of one batch, summed over the ranks,
    against torch's own of the whole batch in 32 bits."""
    ex = _example()
    step = ex.Step(seed=3)
    g = step.g.get_state()
    before = {k: getattr(step, k).clone() for k in ("hidden", "head", "router")}
    step.run(lr=0.0, head_lr=1.0, router_lr=0.0)
    step.g.set_state(g)
    tokens, targets = step.batch()
    head = before["head"].float().requires_grad_()
    x = step.embed[tokens.reshape(-1)].float()
    h = (x + x @ before["hidden"].float().t()).to(torch.bfloat16).float()
    loss = torch.nn.functional.cross_entropy(h @ head.t(), targets.reshape(-1), ignore_index=-100)
    loss.backward()
    moved = before["head"].float() - step.head.float()
    # bf16 steps: the weight's own rounding (2^-9 of its elements) over the
    # gradient's size is the largest error
    scale = float(head.grad.norm())
    slack = 2.0 ** -8 * float(before["head"].float().norm())
    assert float((moved - head.grad).norm()) <= 0.02 * scale + slack
