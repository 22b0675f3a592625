"""The example's step of a mixture of experts: embedding, router, grouped
products, cross entropy, AllReduce and both updates, run together."""

import importlib.util
import math
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

from tests.conftest import ROOT  # noqa: E402


def _example():
    path = os.path.join(ROOT, "examples", "experts_step.py")
    spec = importlib.util.spec_from_file_location("experts_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_steps_run():
    history = _example().main(3)
    assert len(history) == 3
    assert all(math.isfinite(a) and math.isfinite(b) for a, b in history)


def _reference(ex, step, tokens, targets, coef=0.01):
    """The step's loss by torch in 32 bits, with the step's own choice of
    experts and its roundings of what is passed on to bf16."""
    def b16(x):  # rounded, the gradient passed straight on
        return x + (x.to(torch.bfloat16).float() - x).detach()

    table, router, up, down = (w.float().detach().requires_grad_() for w in
                               (step.table, step.router, step.up, step.down))
    flat = tokens.reshape(-1)
    valid = flat >= 0
    h = b16(table[flat.clamp(min=0)] * valid[:, None] * ex.SCALE)
    logits = b16(h @ router.t())
    p = torch.softmax(logits, 1) * valid[:, None]
    # equal logits: the lower expert first, as a stable sort has them
    chosen = torch.argsort(logits.detach(), dim=1, descending=True, stable=True)[:, :ex.TOPK]
    n = valid.sum()
    f = torch.bincount(chosen[valid].reshape(-1), minlength=ex.EXPERTS) / (n * ex.TOPK)
    balance = coef * ex.EXPERTS * (f * p.sum(0) / n).sum()
    last = h
    for k in range(ex.TOPK):
        e = chosen[:, k]
        y = b16(torch.einsum("tfd,td->tf", up[e], h)).relu()
        z = b16(torch.einsum("tdf,tf->td", down[e], y))
        last = last + z / ex.TOPK * valid[:, None]
    last = b16(last)
    loss = torch.nn.functional.cross_entropy(last @ table.t(), targets.reshape(-1),
                                             ignore_index=ex.IGNORE)
    grads = torch.autograd.grad(loss + balance, (table, router, up, down))
    return float(loss.detach()), float(balance.detach()), chosen[valid], grads


def test_gradients_against_autograd():
    """Every gradient of one batch against torch's own in 32 bits."""
    ex = _example()
    step = ex.Step(seed=5)
    tokens, targets = step.batch()
    loss, balance, counts, grads = step.gradients(tokens, targets)
    want_loss, want_balance, chosen, want = _reference(ex, step, tokens, targets)
    assert counts.tolist() == torch.bincount(chosen.reshape(-1), minlength=ex.EXPERTS).tolist()
    # losses of logits below 2^5 from bf16 inputs that are the same on both
    # sides, but for a rounding of `last` here and there (2^-9 of it)
    assert abs(loss - want_loss) <= 2.0 ** -8 * want_loss
    assert abs(balance - want_balance) <= 2.0 ** -8 * want_balance
    # 2-norms: each gradient has passed up to six roundings to bf16 (of the
    # factors, dlast, dz, da, dx, dh and itself; a rounding is 2^-8 / sqrt(3) on
    # average at most, they add as independent errors: sqrt(7 / 3) 2^-8), and the
    # AllReduce of four ranks adds one of each rank's; twice that
    for name, got, ref in zip(("table", "router", "up", "down"), grads, want):
        off = float((got.float() - ref).norm() / ref.norm())
        assert off <= 2 * math.sqrt(8 / 3) * 2.0 ** -8, (name, off)


def test_update_is_what_the_operators_make():
    """The masters move against the gradient by lr in the first step (AdamW's
    first step is its sign), the experts by an orthogonal matrix."""
    ex = _example()
    step = ex.Step(seed=6)
    tokens, targets = step.batch()
    *_, grads = step.gradients(tokens, targets)
    before = [w.clone() for w in step.masters + [step.up, step.down]]
    step.update(grads, lr=0.01, expert_lr=0.02)
    for w, old, g in zip(step.masters, before, grads):
        live = g.float().abs() > 1e-4  # far above eps = 1e-8
        move = (old * (1 - 0.01 * 0.01) - w)[live] / 0.01
        # g / (|g| + 1e-8): within 1e-4; the masters below 1 are rounded, 2^-24
        # of them over a step of 0.01
        assert bool(((move - g.float()[live].sign()).abs() <= 1e-4 + 100 * 2.0 ** -23).all())
    for w, old in zip((step.up, step.down), before[2:]):
        d = (old.float() - w.float()) / 0.02
        s = torch.linalg.svdvals(d.double())
        # five Newton-Schulz steps leave singular values of about 0.7 to 1.2; the
        # matrices are rounded to bf16 on the way (2^-9 of entries of 0.06, 512
        # of them a row, over 0.02: below 0.2)
        assert float(s.max()) < 1.5
