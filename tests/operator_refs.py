"""The training operators in 64 bits on the CPU, from their definitions, and
bounds on what 32-bit arithmetic may differ by.  Shares no code with the
package."""

import math

import torch

U32 = 2.0 ** -24
U_T = {torch.float32: U32, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
MIN_T = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}


def balance(logits, masks, topk, coef, grad_scale):
    """logits: R CPU tensors (T, E); masks: R CPU tensors (T,) or None.
    Returns loss, counts, chosen, dlogits and, for each gradient, a bound of
    the fp32 evaluation's error before its final rounding."""
    R = len(logits)
    T, E = logits[0].shape
    x = torch.stack(logits).double()
    valid = torch.ones(R, T, dtype=torch.bool)
    if masks is not None:
        for r, m in enumerate(masks):
            if m is not None:
                valid[r] = m != 0
    valid &= ~(x == -math.inf).all(2)
    chosen = torch.full((R, T, topk), -1, dtype=torch.int64)
    counts = torch.zeros(E, dtype=torch.int64)
    for r in range(R):
        for t in range(T):
            if valid[r, t]:
                row = x[r, t].tolist()
                # NaN above +inf, equal values: the lower index first
                order = sorted(range(E), key=lambda e: (0, 0.0, e) if row[e] != row[e]
                               else (1, -row[e], e))[:topk]
                chosen[r, t] = torch.tensor(order)
                for e in order:
                    counts[e] += 1
    n = int(valid.sum())
    p = torch.zeros_like(x)
    if n:
        p[valid] = torch.softmax(x[valid], 1)
    f = counts.double() / max(1, n * topk)
    mean = p.sum((0, 1)) / max(1, n)
    loss = coef * E * float((f * mean).sum())
    factor = grad_scale * coef * E / max(1, n)
    dot = (p * f).sum(2, keepdim=True)
    grads = factor * p * (f - dot)
    # exp in fp32: the exponent x - lse is rounded to |x - lse| 2^-23 (the
    # difference, its product with log2 e, lse itself), ex2 to 2 ulp
    gap = torch.where(p > 0, -torch.log(p.clamp(min=1e-300)), torch.zeros_like(p))
    top = x.abs().where(x.abs() < math.inf, torch.zeros_like(x)).amax(2, keepdim=True)
    rel = (2 * gap + 2 * top + 8) * 2 * U32
    # p (f - dot): p's relative error twice over, dot's E-term sum
    bound = abs(factor) * p * (f + dot) * (2 * rel + (E + 8) * U32)
    worst = float(rel[valid].max()) if n else 0.0
    loss_bound = abs(loss) * (worst + (T * R + E + 16) * U32)
    return dict(loss=loss, loss_bound=loss_bound, counts=counts, chosen=chosen, grads=grads,
                bound=bound, n=n)


def assert_close(got, want, bound, dtype, what=""):
    """|got - want| within `bound`, widened by one rounding to dtype."""
    got = got.double()
    limit = bound + (want.abs() + bound) * U_T[dtype] + MIN_T[dtype]
    bad = ~((got - want).abs() <= limit)
    assert not bool(bad.any()), "%s: %d of %d outside, first got %r want %r limit %r" % (
        what, int(bad.sum()), bad.numel(), float(got[bad][0]), float(want[bad][0]),
        float(limit.expand_as(want)[bad][0]))


def xent(hidden, weight, targets, ignore, mean, grad_scale):
    """The cross entropy and its gradients in 64 bits, with bounds on what the
    operator's arithmetic may differ by: products exact, fp32 sums that may
    truncate (2^-23 a term), exp and log in fp32, softmax minus one-hot
    rounded to the type, its softmax part twice at most."""
    ty = hidden.dtype
    h, w = hidden.double(), weight.double()
    T, D = h.shape
    V = w.shape[0]
    valid = (targets != ignore) & (targets >= 0) & (targets < V)
    rows = valid.nonzero()[:, 0]
    l = h @ w.t()
    el = (D + 16) * 2.0 ** -23 * (h.abs() @ w.abs().t())
    big = l.abs().amax(1).nan_to_num(0.0)
    lse = torch.logsumexp(l, 1)
    # exponents rounded to 2^-22 of the logits, sums of up to 128 terms in a
    # row, then over the tiles
    el_row = el.amax(1)
    b_lse = el_row + (200 + V / 2048) * U32 + big * 2.0 ** -21 + lse.abs() * U32
    n = int(valid.sum())
    per = (1.0 / n if n else 0.0) if mean else 1.0
    losses = torch.zeros(T, dtype=torch.float64, device=h.device)
    hot = targets.clone()
    hot[~valid] = 0
    losses[valid] = (lse - l.gather(1, hot[:, None])[:, 0])[valid]
    b_losses = b_lse + el_row + (losses.abs() + big) * U32
    loss = float(losses[valid].sum()) * per
    b_loss = float(b_losses[valid].sum()) * per + abs(loss) * 4 * U32
    # gradients over the tokens that count
    hv, lv = h[rows], l[rows]
    p = torch.exp(lv - lse[rows, None])
    one = torch.zeros_like(p)
    one[torch.arange(len(rows), device=h.device), hot[rows]] = 1.0
    g = p - one
    bp = p * (el[rows] + b_lse[rows, None] + big[rows, None] * 2.0 ** -21 + 8 * U32)
    bg = bp + (p + g.abs() + 2 * bp) * U_T[ty] + (2.0 ** -39 if ty == torch.float16 else 2.0 ** -126)
    s = per * grad_scale
    dh = torch.zeros_like(h)
    b_dh = torch.zeros_like(h)
    dh[rows] = s * (g @ w)
    b_dh[rows] = abs(s) * ((bg + (V + 16) * 2.0 ** -23 * (g.abs() + bg)) @ w.abs())
    dw = s * (g.t() @ hv)
    b_dw = abs(s) * ((bg + (n + 16) * 2.0 ** -23 * (g.abs() + bg)).t() @ hv.abs())
    return dict(valid=valid, lse=lse, b_lse=b_lse, losses=losses, b_losses=b_losses, loss=loss,
                b_loss=b_loss, dh=dh, b_dh=b_dh, dw=dw, b_dw=b_dw)


def norm_error(got, want):
    """2-norm of the difference over the 2-norm of the result."""
    n = float(want.norm())
    d = float((got.double() - want).norm())
    return d / n if n else d


COEFS = (3.4445, -4.7750, 2.0315)


def orthogonalize(m, steps, coefs, eps, scale):
    x = m.double()
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.t()
    x = x / (x.norm() + eps)
    for k in range(steps):
        # the coefficients reach the operator as fp32
        a, b, c = (float(torch.tensor(v, dtype=torch.float32)) for v in
                   (coefs[3 * k:3 * k + 3] if coefs is not None else COEFS))
        g = x @ x.t()
        x = a * x + (b * g + c * (g @ g)) @ x
    return scale * (x.t() if tall else x)


def ortho_tolerance(ty, norm, gain):
    """2-norm of the error over that of the result.  X is held to 22 bits: a
    rounding of X (norm 1), amplified by at most `gain` (the product of the
    steps' a) in the directions of the smallest singular values, next to the
    norm of the result, and the
    chunks' sums (32 additions truncated to 2^-23 each, both ways).  fp16
    and bf16: the result's own rounding on top of that; bf16 operands are
    rounded to 2^-12 on average three times a step and scaled by
    |b A + c A A| <= 2.8."""
    exact = 2.0 ** -23 * (gain / norm + 64)
    if ty == torch.float32:
        return exact
    if ty == torch.float16:
        return exact + 2.0 ** -11
    return exact + 2.0 ** -9 + 2.0 ** -9
