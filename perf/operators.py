"""The operators of a data-parallel training step, measured: the two losses
whose gradients an AllReduce sums, and the update that is made of the sum.

* ``xent``     softmax cross entropy of a linear layer over a large
               vocabulary, its per-token losses and, for training, the
               gradients of the hidden states and of the weight;
* ``ortho``    a matrix (or several of one shape) orthogonalised by
               Newton-Schulz steps;
* ``balance``  the balance loss of R ranks' expert routers over the whole
               batch, with the per-expert counts, the chosen experts and the
               gradients of the logits.
"""

import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
COEFS = (3.4445, -4.7750, 2.0315)  # of the quintic Newton-Schulz step
STEPS = 5
EPS = 1e-7
IGNORE = -100


def listed():
    return [
        # one sampled token scored against its vocabulary: latency
        dict(name="xent one token", op="xent", tokens=1, dim=1024, vocab=32768, dtype="bf16",
             grads=False, ignored=0.0),
        # perplexity of a batch of documents: loss only
        dict(name="xent scoring", op="xent", tokens=4096, dim=2048, vocab=50304, dtype="bf16",
             grads=False, ignored=0.05),
        # a fine-tuning step on a ragged batch, the prompts' tokens ignored
        dict(name="xent ragged", op="xent", tokens=777, dim=1000, vocab=50001, dtype="bf16",
             grads=True, ignored=0.4),
        # a half-precision training step of a small vocabulary
        dict(name="xent half", op="xent", tokens=2048, dim=2048, vocab=32768, dtype="fp16",
             grads=True, ignored=0.0),
        # one rank's micro-batch of pre-training: large vocabulary
        dict(name="xent large", op="xent", tokens=4096, dim=4096, vocab=131072, dtype="bf16",
             grads=True, ignored=0.02),
        # the small projections of many layers in one call: latency
        dict(name="ortho small", op="ortho", count=8, rows=128, cols=128, dtype="bf16"),
        # a ragged matrix in full precision
        dict(name="ortho odd fp32", op="ortho", count=1, rows=500, cols=1003, dtype="fp32"),
        # the feed-forward matrices of a few layers
        dict(name="ortho layers", op="ortho", count=4, rows=1024, cols=4096, dtype="bf16"),
        # a tall matrix whose momentum is kept in 32 bits
        dict(name="ortho tall fp32", op="ortho", count=1, rows=4096, cols=1024, dtype="fp32"),
        # one wide feed-forward matrix
        dict(name="ortho large", op="ortho", count=1, rows=4096, cols=16384, dtype="bf16"),
        # four ranks that decode a few sequences each
        dict(name="balance small", op="balance", ranks=4, tokens=16, experts=8, topk=2,
             dtype="fp32", masked=0.1),
        # eight ranks' micro-batches over many experts
        dict(name="balance large", op="balance", ranks=8, tokens=16384, experts=256, topk=8,
             dtype="bf16", masked=0.05),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, grain=1):
    """The same as a multiple of `grain`."""
    while True:
        n = max(lo, min(hi, -(-_log(rng, lo, hi) // grain) * grain))
        if n != 3072:
            return n


def draw(rng):
    op = rng.choice(["xent", "xent", "ortho", "ortho", "balance"])
    if op == "xent":
        grads = rng.random() < 0.7
        tokens = _size(rng, 1, 8192)
        # three in four hidden sizes are multiples of eight, as models have them
        dim = _size(rng, 64, 4096, 8 if rng.random() < 0.75 else 1)
        vocab = _size(rng, 1000, 131072, 64 if rng.random() < 0.5 else 1)
        while tokens * dim * vocab > 4096 * 4096 * 131072 // 2:
            tokens = max(1, tokens // 2)
        return dict(op=op, tokens=tokens, dim=dim, vocab=vocab,
                    dtype=rng.choice(["bf16", "bf16", "fp16"]), grads=grads,
                    ignored=rng.choice([0.0, 0.1, 0.5]))
    if op == "ortho":
        rows = _size(rng, 32, 4096, 8 if rng.random() < 0.75 else 1)
        cols = _size(rng, 32, 8192, 8 if rng.random() < 0.75 else 1)
        count = _size(rng, 1, 16)
        m, n = min(rows, cols), max(rows, cols)
        while count > 1 and count * m * m * n > 2048 * 2048 * 8192:
            count //= 2
        return dict(op=op, count=count, rows=rows, cols=cols,
                    dtype=rng.choice(["bf16", "bf16", "fp32", "fp16"]))
    experts = _size(rng, 4, 512)
    topk = min(rng.choice([1, 2, 4, 6, 8]), experts)
    ranks = rng.choice([1, 2, 4, 7, 8])
    tokens = _size(rng, 1, 16384)
    return dict(op=op, ranks=ranks, tokens=tokens, experts=experts, topk=topk,
                dtype=rng.choice(["fp32", "bf16", "fp16"]), masked=rng.choice([0.0, 0.1]))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    dtype = DTYPES[case["dtype"]]
    # half-precision training scales its gradients into the type's range
    s = dict(case=case, dtype=dtype, grad_scale=1.0)
    if case["dtype"] == "fp16" and case["op"] != "ortho":
        s["grad_scale"] = 64.0 * case["tokens"] * case.get("ranks", 1)
    if case["op"] == "xent":
        T, D, V = case["tokens"], case["dim"], case["vocab"]
        # logits of deviation 2; every other token's target stands out by
        # about 8, as a partly trained model's does
        weight = (randn(V, D) * (2.0 / math.sqrt(D))).to(dtype)
        targets = torch.randint(0, V, (T,), generator=g, device="cuda")
        hidden = randn(T, D)
        hidden[::2] += 2.0 * weight[targets[::2]].float()
        targets[rand(T) < case["ignored"]] = IGNORE
        s.update(hidden=hidden.to(dtype), weight=weight, targets=targets,
                 losses=torch.empty(T, device="cuda"), lse=torch.empty(T, device="cuda"),
                 loss=torch.empty(1, device="cuda"))
        if case["grads"]:
            s.update(dhidden=torch.empty(T, D, device="cuda", dtype=dtype),
                     dweight=torch.empty(V, D, device="cuda", dtype=dtype))
    elif case["op"] == "ortho":
        n, r, c = case["count"], case["rows"], case["cols"]
        # a gradient's decaying spectrum over a floor of noise
        k = max(1, min(r, c) // 4)
        decay = torch.arange(1, k + 1, device="cuda").float().rsqrt()
        m = (randn(n, r, k) * decay) @ randn(n, k, c) / math.sqrt(k) + 0.3 * randn(n, r, c)
        m = (m * 0.01).to(dtype)
        s.update(matrices=[x.clone() for x in m], out=[torch.empty_like(x) for x in m])
    else:
        R, T, E = case["ranks"], case["tokens"], case["experts"]
        bias = randn(E)  # some experts are preferred
        logits = [(randn(T, E) + bias).to(dtype) for _ in range(R)]
        masks = [(rand(T) >= case["masked"]).to(torch.uint8) for _ in range(R)]
        s.update(logits=logits, masks=masks, coef=0.01,
                 loss=torch.empty(1, device="cuda"),
                 counts=torch.empty(E, device="cuda", dtype=torch.int32),
                 chosen=[torch.empty(T, case["topk"], device="cuda", dtype=torch.int32)
                         for _ in range(R)],
                 dlogits=[torch.empty_like(x) for x in logits])
    return s


# ---------------------------------------------------------------- plain forms
def _plain_xent(s):
    h, w, y, dtype = s["hidden"].float(), s["weight"].float(), s["targets"], s["dtype"]
    valid = y != IGNORE
    at = torch.where(valid, y, 0)[:, None]
    logits = h @ w.t()
    top = logits.max(dim=1, keepdim=True).values
    e = torch.exp(logits - top)
    total = e.sum(dim=1, keepdim=True)
    lse = torch.log(total) + top
    losses = torch.where(valid, (lse - logits.gather(1, at))[:, 0], 0.0)
    scale = 1.0 / valid.sum().clamp(min=1)
    out = {"losses": losses, "lse": lse[:, 0], "loss": (losses.sum() * scale)[None]}
    if s["case"]["grads"]:
        grad = e / total
        grad.scatter_add_(1, at, torch.full_like(losses, -1.0)[:, None])
        grad *= valid[:, None] * (scale * s["grad_scale"])
        out["dhidden"] = (grad @ w).to(dtype)
        out["dweight"] = (grad.t() @ h).to(dtype)
    return out


def _newton_schulz(x, steps):
    if steps == 0:
        return x
    a, b, c = COEFS
    gram = x @ x.transpose(1, 2)
    return _newton_schulz(a * x + (b * gram + c * (gram @ gram)) @ x, steps - 1)


def _plain_ortho(s):
    m = torch.stack(s["matrices"]).float()
    tall = m.shape[1] > m.shape[2]
    x = m.transpose(1, 2) if tall else m
    x = x / ((x * x).sum(dim=(1, 2), keepdim=True).sqrt() + EPS)
    x = _newton_schulz(x, STEPS)
    return list((x.transpose(1, 2) if tall else x).to(s["dtype"]).contiguous().unbind(0))


def _plain_balance(s):
    R, T, E, k = (s["case"][n] for n in ("ranks", "tokens", "experts", "topk"))
    x = torch.stack(s["logits"]).float()
    valid = torch.stack(s["masks"]) != 0
    n = valid.sum().clamp(min=1)
    # a stable sort gives ties to the lowest index
    chosen = torch.argsort(x, dim=2, descending=True, stable=True)[:, :, :k]
    chosen = torch.where(valid[:, :, None], chosen, -1)
    slots = torch.where(chosen < 0, E, chosen).reshape(-1)
    counts = torch.zeros(E + 1, device=x.device, dtype=torch.int64)
    counts = counts.scatter_add_(0, slots, torch.ones_like(slots))[:E]
    p = torch.exp(x - x.max(dim=2, keepdim=True).values)
    p = p / p.sum(dim=2, keepdim=True) * valid[:, :, None]
    share = counts / (n * k)
    mean = p.sum(dim=(0, 1)) / n
    loss = s["coef"] * E * (share * mean).sum()
    grad = (s["grad_scale"] * s["coef"] * E / n) * p * (share - (p @ share)[:, :, None])
    return {"loss": loss[None], "counts": counts.int(), "chosen": list(chosen.int().unbind(0)),
            "dlogits": list(grad.to(s["dtype"]).unbind(0))}


# ------------------------------------------------------ the framework's calls
def _work(s, size, *args):
    """The workspace that a program keeps for calls of one shape."""
    if "work" not in s:
        n = size(*args)
        s["work"], s["bytes"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"), n
    return s["work"], s["bytes"]


def _own_xent(s):
    import double_binary_tree_gb300 as vr
    c, h, w = s["case"], s["hidden"], s["weight"]
    T, D, V, grads = c["tokens"], c["dim"], c["vocab"], c["grads"]
    dtype = vr.VR_BFLOAT16 if c["dtype"] == "bf16" else vr.VR_FLOAT16
    work, size = _work(s, vr.vr_linear_xent_workspace_bytes, h, D, w, D, T, D, V, dtype, grads)
    vr.vr_linear_xent(h, D, w, D, s["targets"], T, D, V, dtype, IGNORE, True, s["grad_scale"],
                      s["losses"], s["lse"], s["loss"], s.get("dhidden"), s.get("dweight"),
                      work, size, torch.cuda.current_stream())
    return {k: s[k] for k in ("losses", "lse", "loss") + (("dhidden", "dweight") if grads else ())}


def _own_ortho(s):
    import double_binary_tree_gb300 as vr
    c = s["case"]
    dtype = {"fp32": vr.VR_FLOAT32, "fp16": vr.VR_FLOAT16, "bf16": vr.VR_BFLOAT16}[c["dtype"]]
    n, r, k = c["count"], c["rows"], c["cols"]
    work, size = _work(s, vr.vr_orthogonalize_workspace_bytes, n, r, k, dtype)
    vr.vr_orthogonalize(s["matrices"], s["out"], n, r, k, dtype, STEPS, None, EPS, 1.0, work, size,
                        torch.cuda.current_stream())
    return s["out"]


def _own_balance(s):
    import double_binary_tree_gb300 as vr
    c = s["case"]
    dtype = {"fp32": vr.VR_FLOAT32, "fp16": vr.VR_FLOAT16, "bf16": vr.VR_BFLOAT16}[c["dtype"]]
    R, T, E = c["ranks"], c["tokens"], c["experts"]
    work, size = _work(s, vr.vr_balance_loss_workspace_bytes, R, T, E)
    vr.vr_balance_loss(s["logits"], E, s["masks"], R, T, E, c["topk"], dtype, s["coef"],
                       s["grad_scale"], s["loss"], s["counts"], s["chosen"], s["dlogits"],
                       work, size, torch.cuda.current_stream())
    return {k: s[k] for k in ("loss", "counts", "chosen", "dlogits")}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"xent": _own_xent, "ortho": _own_ortho, "balance": _own_balance}[op](state)
    return {"xent": _plain_xent, "ortho": _plain_ortho, "balance": _plain_balance}[op](state)


def work(case):
    if case["op"] == "xent":
        T, D, V = case["tokens"], case["dim"], case["vocab"]
        one = (T * D + V * D) * 2
        # the logits; with gradients two more products of the same size and
        # both gradients written
        return {"bytes": one * (2 if case["grads"] else 1) + T * 16 + 4,
                "flops": (6 if case["grads"] else 2) * T * D * V}
    if case["op"] == "ortho":
        n, m, k = case["count"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
        size = 4 if case["dtype"] == "fp32" else 2
        # per step: two symmetric products, half of each computed, and a whole one
        return {"bytes": 2 * n * m * k * size, "flops": STEPS * n * (3 * m * m * k + m ** 3)}
    R, T, E, k = (case[n] for n in ("ranks", "tokens", "experts", "topk"))
    size = 4 if case["dtype"] == "fp32" else 2
    return {"bytes": R * T * (2 * E * size + 1 + 4 * k) + 4 * E + 4, "flops": 12 * R * T * E}


# ------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "xent":
        T, V, y = case["tokens"], case["vocab"], s["targets"]
        h, w = s["hidden"].double(), s["weight"].double()
        count = max(1, int((y >= 0).sum()))
        losses, lse = torch.zeros(T, **_f64()), torch.zeros(T, **_f64())
        dh = torch.zeros_like(h) if case["grads"] else None
        dw = torch.zeros_like(w) if case["grads"] else None
        keep = (y >= 0).double()
        hot = y.clamp(min=0)
        for lo in range(0, T, 1024):  # tokens at a time
            hi = min(T, lo + 1024)
            z = torch.mm(h[lo:hi], w.T)
            lse[lo:hi] = torch.logsumexp(z, 1)
            rows = torch.arange(hi - lo, device="cuda")
            losses[lo:hi] = (lse[lo:hi] - z[rows, hot[lo:hi]]) * keep[lo:hi]
            if case["grads"]:
                z = z.sub_(lse[lo:hi, None]).exp_()
                z[rows, hot[lo:hi]] -= 1.0
                z *= (keep[lo:hi] / count * s["grad_scale"])[:, None]
                dh[lo:hi] = torch.mm(z, w)
                dw.addmm_(z.T, h[lo:hi])
        out = {"losses": losses, "lse": lse, "loss": losses.sum()[None] / count}
        if case["grads"]:
            out.update(dhidden=dh, dweight=dw)
        return out
    if case["op"] == "ortho":
        a, b, c = COEFS
        got = []
        for m in s["matrices"]:
            x = m.double()
            x = x / (torch.linalg.norm(x) + EPS)
            for _ in range(STEPS):  # the same polynomial from the shorter side
                if x.shape[0] <= x.shape[1]:
                    q = torch.mm(x, x.T)
                    x = a * x + b * torch.mm(q, x) + c * torch.mm(q, torch.mm(q, x))
                else:
                    q = torch.mm(x.T, x)
                    x = a * x + b * torch.mm(x, q) + c * torch.mm(torch.mm(x, q), q)
            got.append(x)
        return got
    E, k = case["experts"], case["topk"]
    x = torch.cat(s["logits"]).double()
    valid = torch.cat(s["masks"]).bool()
    n = max(1, int(valid.sum()))
    p = torch.softmax(x, 1) * valid[:, None]
    left, hits = x.clone(), torch.zeros(E, **_f64())
    for _ in range(k):  # the largest one left, the first of equals
        at = _first_largest(left)
        hits += torch.bincount(at[valid], minlength=E).double()
        left[torch.arange(len(left), device="cuda"), at] = -math.inf
    f = hits / (n * k)
    grad = p * f - p * (p * f).sum(1, keepdim=True)
    T = case["tokens"]
    return {"loss": (s["coef"] * E * (f * p.sum(0) / n).sum())[None], "counts": None,
            "chosen": None, "dlogits": list((grad * (s["grad_scale"] * s["coef"] * E / n)).split(T))}


def _f64():
    return dict(dtype=torch.float64, device="cuda")


def _first_largest(x):
    """The lowest index of each row's largest value."""
    index = torch.arange(x.shape[1], device=x.device)
    return torch.where(x == x.max(1, keepdim=True).values, index, x.shape[1]).min(1).values
