"""The example's data-parallel step: the gradients of its hidden matrix and of its
router, summed over the ranks, against autograd's of the whole batch."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

from tests.test_gpu_training_step import _example  # noqa: E402


def test_hidden_matrix_and_router():
    ex = _example()
    step = ex.Step(seed=4)
    g = step.g.get_state()
    hidden, head, router = (getattr(step, k).clone() for k in ("hidden", "head", "router"))
    lr = 1000.0     # so that the bf16 router moves by more than its rounding
    step.run(lr=0.0, head_lr=0.0, router_lr=lr)
    step.g.set_state(g)
    tokens, targets = step.batch()
    x = step.embed[tokens.reshape(-1)].float()
    flat = targets.reshape(-1)

    # the hidden matrix: the momentum of the first step is its gradient
    m = hidden.float().requires_grad_()
    h = x + x @ m.t()
    torch.nn.functional.cross_entropy(h @ head.float().t(), flat, ignore_index=-100).backward()
    # bf16 states, gradients of the states, their products and the sum of four
    # ranks: eight roundings of 2^-9 on average at most
    scale = float(m.grad.norm())
    assert float((step.momentum - m.grad).norm()) <= 8 * 2.0 ** -9 * scale

    # the router: the balance loss over the tokens that count, their choice held
    r = router.float().requires_grad_()
    h = h.detach().to(torch.bfloat16).float()
    logits = (h @ r.t()).to(torch.bfloat16).float()
    count = flat >= 0
    p = torch.softmax(logits[count], 1)
    chosen = logits[count].argsort(dim=1, descending=True, stable=True)[:, :ex.TOPK]
    f = torch.bincount(chosen.reshape(-1), minlength=ex.EXPERTS).float() / chosen.numel()
    (0.01 * ex.EXPERTS * (f * p.mean(0)).sum()).backward()
    moved = (router.float() - step.router.float()) / lr
    # logits rounded to bf16 move p by up to 2^-9 of them (they reach 5 or so),
    # besides the roundings above and that of the weight itself
    slack = 2.0 ** -8 * float(router.float().norm() / lr + moved.norm())
    assert float((moved - r.grad).norm()) <= (5 + 8) * 2.0 ** -9 * float(r.grad.norm()) + slack
    assert float(r.grad.norm()) > 4 * slack
