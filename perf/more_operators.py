"""The operators that complete a training step, measured: where it begins (the
embedding of its tokens), what stands between the router and its experts, and
the update of everything that is not orthogonalised.

* ``embed``    rows of an embedding table by token, scaled; or the gradient of
               the table, the sums over equal tokens, written whole or added
               to the gradient of an output layer that shares the table;
* ``adamw``    one AdamW step over many tensors at once, with states of 32 or
               of 8 bits, with or without a 32-bit master copy;
* ``experts``  rows sorted by expert times the weights of their expert, with
               any number of rows per expert; or the gradients of such a
               product.
"""

import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
IGNORE = -100
BLOCK = 256  # elements of an 8-bit state that share a scale


def _f32(x):
    return float(torch.tensor(x, dtype=torch.float32))


# the optimiser's numbers are 32-bit numbers
LR, BETA1, BETA2, ADAM_EPS, DECAY = (_f32(x) for x in (3e-4, 0.9, 0.95, 1e-8, 0.1))
SEED = 0x5EED0123456789


def listed():
    return [
        # the token that a decoding step has just sampled: latency
        dict(name="embed one token", op="embed", tokens=1, dim=1024, vocab=32768, dtype="bf16",
             grads=False, add=False, ignored=0.0),
        # a rank's micro-batch
        dict(name="embed prompt", op="embed", tokens=16384, dim=4096, vocab=131072, dtype="bf16",
             grads=False, add=False, ignored=0.0),
        # a fine-tuning step on a ragged batch with padding, the table shared
        # with the output layer, whose gradient is there already
        dict(name="embed ragged grads", op="embed", tokens=777, dim=1000, vocab=50001,
             dtype="bf16", grads=True, add=True, ignored=0.4),
        # one rank's micro-batch of pre-training, a few words far more frequent
        # than the others
        dict(name="embed large grads", op="embed", tokens=16384, dim=4096, vocab=131072,
             dtype="bf16", grads=True, add=False, ignored=0.02),
        # the gains of the norms of many layers, in full precision: latency
        dict(name="adamw gains", op="adamw", dtype="fp32", grad="fp32", bits=32, master=False,
             small=48, layers=0, dim=1024, inner=0, vocab=0),
        # a model in 16 bits with master copies and states in full precision
        dict(name="adamw masters", op="adamw", dtype="bf16", grad="bf16", bits=32, master=True,
             small=24, layers=12, dim=1024, inner=4096, vocab=32768),
        # odd sizes, states in 8 bits
        dict(name="adamw 8 bits", op="adamw", dtype="bf16", grad="bf16", bits=8, master=True,
             small=17, layers=8, dim=1000, inner=4004, vocab=50001),
        # one token decoded, its experts' weights read once: latency
        dict(name="experts one token", op="experts", tokens=1, topk=8, groups=64, dim=2048,
             out=1024, dtype="bf16", grads=False, spare=0),
        # a decoding step of many sequences: every expert has a few rows
        dict(name="experts decode", op="experts", tokens=64, topk=4, groups=64, dim=2048,
             out=4096, dtype="bf16", grads=False, spare=0),
        # a ragged batch in half precision, with its gradients, in a buffer
        # that has room for more
        dict(name="experts ragged grads", op="experts", tokens=1501, topk=2, groups=12, dim=1000,
             out=1512, dtype="fp16", grads=True, spare=19),
        # a prompt through many experts
        dict(name="experts prompt", op="experts", tokens=4096, topk=8, groups=64, dim=2048,
             out=4096, dtype="bf16", grads=False, spare=0),
        # one rank's micro-batch of pre-training: both gradients
        dict(name="experts train", op="experts", tokens=16384, topk=4, groups=32, dim=4096,
             out=2048, dtype="bf16", grads=True, spare=0),
    ]


def _log(rng, lo, hi, grain=1):
    """A whole number spread over the logarithm of [lo, hi], a multiple of
    `grain`."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, -(-n // grain) * grain))


def draw(rng):
    op = rng.choice(["embed", "adamw", "experts", "experts"])
    if op == "embed":
        grads = rng.random() < 0.6
        return dict(op=op, tokens=_log(rng, 1, 32768),
                    # three in four widths are multiples of eight, as models have them
                    dim=_log(rng, 64, 4096, 8 if rng.random() < 0.75 else 1),
                    vocab=_log(rng, 1000, 131072, 64 if rng.random() < 0.5 else 1),
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), grads=grads,
                    add=grads and rng.random() < 0.4, ignored=rng.choice([0.0, 0.1, 0.5]))
    if op == "adamw":
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        dim = _log(rng, 64, 2048, 8 if rng.random() < 0.75 else 1)
        return dict(op=op, dtype=dtype, grad=rng.choice([dtype, dtype, "fp32"]),
                    bits=rng.choice([8, 32]), master=dtype != "fp32" and rng.random() < 0.7,
                    small=_log(rng, 1, 64), layers=_log(rng, 1, 8), dim=dim,
                    inner=_log(rng, dim, 4 * dim), vocab=_log(rng, 1000, 50000))
    groups = _log(rng, 1, 128)
    topk = min(rng.choice([1, 2, 4, 8]), groups)
    c = dict(op=op, tokens=_log(rng, 1, 16384), topk=topk, groups=groups,
             dim=_log(rng, 64, 4096, 8 if rng.random() < 0.8 else 1),
             out=_log(rng, 64, 4096, 8 if rng.random() < 0.8 else 1),
             dtype=rng.choice(["bf16", "bf16", "fp16"]), grads=rng.random() < 0.5,
             spare=rng.choice([0, 0, 33]))
    while c["tokens"] * topk * c["dim"] * c["out"] > 65536 * 4096 * 1024:
        c["tokens"] //= 2
    while groups * c["dim"] * c["out"] > 64 * 4096 * 2048:
        c["dim"] = max(64, c["dim"] // 2)
    return c


def _tensors(c):
    """Sizes of the tensors of a model: the table, each layer's matrices, the
    gains of the norms."""
    d, i = c["dim"], c["inner"]
    sizes = [c["vocab"] * d] if c["vocab"] else []
    return sizes + [d * d, d * i, i * d] * c["layers"] + [d] * c["small"]


def _starts(sizes):
    """Each tensor begins at a multiple of BLOCK elements of one buffer."""
    at, starts = 0, []
    for n in sizes:
        starts.append(at)
        at += -(-n // BLOCK) * BLOCK
    return starts, at


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 29)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    dtype = DTYPES[case["dtype"]]
    s = dict(case=case, dtype=dtype)
    if case["op"] == "embed":
        T, D, V = case["tokens"], case["dim"], case["vocab"]
        # words by frequency: the n-th in proportion to 1 / n
        ids = (torch.exp(rand(T) * math.log(V + 1)) - 1).long().clamp(0, V - 1)
        ids[rand(T) < case["ignored"]] = IGNORE
        s.update(ids=ids, scale=math.sqrt(D))
        if case["grads"]:
            s["scale"] = 0.5
            s["dout"] = randn(T, D).to(dtype)
            there = randn(V, D).to(dtype) if case["add"] else torch.zeros(V, D, device="cuda",
                                                                          dtype=dtype)
            s["dweight"] = there
        else:
            s.update(weight=(randn(V, D) * 0.02).to(dtype),
                     out=torch.empty(T, D, device="cuda", dtype=dtype))
    elif case["op"] == "adamw":
        sizes = _tensors(case)
        starts, n = _starts(sizes)
        live = torch.zeros(n, device="cuda")
        for a, k in zip(starts, sizes):
            live[a:a + k] = 1.0
        # tensors whose gradients differ by orders of magnitude, and in each
        # some elements that have hardly any
        size = torch.exp(randn(n // BLOCK) * 1.5).repeat_interleave(BLOCK) * live
        grad = randn(n) * size * torch.where(rand(n) < 0.1, 1e-3, 1e-2)
        s.update(sizes=sizes, starts=starts, step=100, grad=grad.to(DTYPES[case["grad"]]))
        value = randn(n) * 0.02 * live
        s["param"] = value.to(dtype)
        s["master"] = value if case["master"] else None
        m, v = randn(n) * size * 3e-3, (size * 1e-2 * (0.5 + rand(n))) ** 2
        if case["bits"] == 8:
            s["m"], s["mscale"] = _encode_m(m, torch.zeros(n, dtype=torch.int32, device="cuda"))
            s["v"], s["vscale"] = _encode_v(v, torch.zeros(n, dtype=torch.int32, device="cuda"))
            s["mvalues"], s["vvalues"] = torch.zeros_like(m), torch.zeros_like(v)
        else:
            s.update(m=m, v=v)
    else:
        T, k, E = case["tokens"], case["topk"], case["groups"]
        K, N = case["dim"], case["out"]
        # each token's experts, some of them preferred
        score = randn(T, E) + 0.7 * randn(E)
        chosen = torch.topk(score, k, dim=1).indices.reshape(-1)
        counts = torch.bincount(chosen, minlength=E).int()
        rows = T * k + case["spare"]
        s.update(counts=counts, rows=rows, most=int(counts.max()),
                 weight=(randn(E, N, K) / math.sqrt(K)).to(dtype), x=randn(rows, K).to(dtype))
        if case["grads"]:
            s.update(dout=randn(rows, N).to(dtype),
                     dx=torch.zeros(rows, K, device="cuda", dtype=dtype),
                     dweight=torch.empty(E, N, K, device="cuda", dtype=dtype))
        else:
            s["out"] = torch.zeros(rows, N, device="cuda", dtype=dtype)
    return s


# ---------------------------------------------------------------- plain forms
def _plain_embed(s):
    ids, dtype = s["ids"], s["dtype"]
    valid = ids >= 0
    at = torch.where(valid, ids, 0)
    if not s["case"]["grads"]:
        return {"out": (s["weight"][at].float() * s["scale"] * valid[:, None]).to(dtype)}
    rows = s["dout"].float() * (valid[:, None] * s["scale"])
    total = s["dweight"].float() if s["case"]["add"] else torch.zeros_like(s["dweight"],
                                                                          dtype=torch.float32)
    s["dweight"].copy_(total.index_add_(0, at, rows))
    return {"dweight": s["dweight"]}


# A state of 8 bits is a number of three binary digits behind the point and an
# exponent, by which the digits of a 32-bit number are cut off behind the third:
# the lowest exponents become those of 32-bit denormals.  `cut` (20 bits, random)
# is added to what is cut off.  Blocks of 256 share a power of two as scale.
def _power(e):
    """2**e of whole numbers e in [-126, 127], exactly."""
    return ((e + 127) << 23).int().view(torch.float32)


def _block_exponent(x):
    top = x.abs().view(-1, BLOCK).max(dim=1).values
    e = (top.view(torch.int32) >> 23) - 127
    return e.clamp(min=-110), torch.isfinite(top)


def _encode(x, cut, lift, bias):
    e, fine = _block_exponent(x)
    up = _power(lift - e).repeat_interleave(BLOCK)
    code = ((x.abs() * up * 2.0 ** -bias).view(torch.int32) + cut) >> 20
    code = torch.where(fine.repeat_interleave(BLOCK), code, 0)
    return code, torch.where(fine, _power(e - lift), math.nan)


def _encode_m(m, cut):
    code, scale = _encode(m, cut, 7, 120)
    return (code | torch.where((m < 0) & (code > 0), 128, 0)).to(torch.uint8), scale


def _encode_v(v, cut):
    code, scale = _encode(v, cut, 15, 112)
    return torch.where(v > 0, code.clamp(min=1), code).to(torch.uint8), scale


def _value_m(code, scale):
    code = code.int()
    x = ((code & 127) << 20).view(torch.float32) * 2.0 ** 120 * scale.repeat_interleave(BLOCK)
    return torch.where(code > 127, -x, x)


def _value_v(code, scale):
    return (code.int() << 20).view(torch.float32) * 2.0 ** 112 * scale.repeat_interleave(BLOCK)


def _mix(x):
    """A bijection of 32-bit numbers that stirs their bits (in 64-bit ones)."""
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random(n, step):
    """32 random bits of each element, by the seed, the step and its place."""
    key = SEED & 0xFFFFFFFF
    key = _mix(_mix(_mix(_mix(key) ^ (SEED >> 32)) ^ (step & 0xFFFFFFFF)) ^ (step >> 32))
    at = torch.arange(n, device="cuda")
    return _mix(_mix(key ^ (at >> 32)) ^ (at & 0xFFFFFFFF))


def _plain_adamw(s):
    c = s["case"]
    s["step"] += 1
    g = s["grad"].float()
    few = c["bits"] == 8
    m = _value_m(s["m"], s["mscale"]) if few else s["m"]
    v = _value_v(s["v"], s["vscale"]) if few else s["v"]
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + g * g * (1.0 - BETA2)
    p = (s["master"] if c["master"] else s["param"]).float()
    up = LR / (1.0 - BETA1 ** s["step"])
    down = (v / (1.0 - BETA2 ** s["step"])).sqrt() + ADAM_EPS
    p = p * (1.0 - LR * DECAY) - up * m / down
    if few:
        r = _random(m.numel(), s["step"])
        s["m"], s["mscale"] = _encode_m(m, ((r & 0xFFFF) << 4).int())
        s["v"], s["vscale"] = _encode_v(v, ((r >> 16) << 4).int())
    else:
        s["m"], s["v"] = m, v
    s["param"] = p.to(s["dtype"])
    out = {"param": s["param"], "m": _value_m(s["m"], s["mscale"]) if few else m,
           "v": _value_v(s["v"], s["vscale"]) if few else v}
    if c["master"]:
        s["master"] = out["master"] = p
    return out


def _plain_experts(s):
    E, counts, most = s["case"]["groups"], s["counts"].long(), s["most"]
    last = counts.cumsum(0)
    row = torch.arange(s["rows"], device="cuda")
    live = row < last[-1]
    group = (row[:, None] >= last).sum(1).clamp(max=E - 1)
    slot = torch.where(live, row - (last - counts)[group], 0)
    # each expert's rows side by side, with zeros up to the longest
    place = (last - counts)[:, None] + torch.arange(most, device="cuda")
    there = (torch.arange(most, device="cuda") < counts[:, None])[:, :, None]
    place = place.clamp(max=s["rows"] - 1)
    w = s["weight"].float()
    x = torch.where(there, s["x"][place].float(), 0.0)
    if not s["case"]["grads"]:
        y = x @ w.transpose(1, 2)
        return {"out": torch.where(live[:, None], y[group, slot], 0.0).to(s["dtype"])}
    dy = torch.where(there, s["dout"][place].float(), 0.0)
    dx = torch.where(live[:, None], (dy @ w)[group, slot], 0.0)
    return {"dx": dx.to(s["dtype"]), "dweight": (dy.transpose(1, 2) @ x).to(s["dtype"])}


# ------------------------------------------------------ the framework's calls
def _code(vr, name):
    return {"fp32": vr.VR_FLOAT32, "fp16": vr.VR_FLOAT16, "bf16": vr.VR_BFLOAT16}[name]


def _work(s, size, *args):
    """The workspace that a program keeps for calls of one shape."""
    if "work" not in s:
        n = size(*args)
        s["work"], s["bytes"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"), n
    return s["work"], s["bytes"]


def _own_embed(s):
    import double_binary_tree_gb300 as vr
    c = s["case"]
    T, D, V, dtype = c["tokens"], c["dim"], c["vocab"], _code(vr, c["dtype"])
    stream = torch.cuda.current_stream()
    if not c["grads"]:
        vr.vr_embedding(s["weight"], D, s["ids"], T, D, V, dtype, IGNORE, s["scale"], s["out"], D,
                        stream)
        return {"out": s["out"]}
    work, size = _work(s, vr.vr_embedding_grad_workspace_bytes, T, D, V, dtype)
    vr.vr_embedding_grad(s["dout"], D, s["ids"], T, D, V, dtype, IGNORE, s["scale"], c["add"],
                         s["dweight"], work, size, stream)
    return {"dweight": s["dweight"]}


def _parts(s, flat, unit=1):
    """The tensors of one flat buffer (`unit` elements of them to one of it)."""
    return None if flat is None else [flat[a // unit:a // unit + -(-n // unit)]
                                      for a, n in zip(s["starts"], s["sizes"])]


def _own_adamw(s):
    import double_binary_tree_gb300 as vr
    c = s["case"]
    if "lists" not in s:  # the program's tensors, listed once for all steps
        parts = [_parts(s, s[k]) for k in ("param", "grad", "m", "v")]
        parts += [_parts(s, s.get(k), BLOCK) for k in ("mscale", "vscale")]
        parts += [_parts(s, s.get(k)) for k in ("master", "mvalues", "vvalues")]
        s["lists"] = [vr.pointer_array(p) for p in parts]
        s["counts"] = vr.size_array(s["sizes"])
    p, g, m, v, ms, vs, master, mvalues, vvalues = s["lists"]
    s["step"] += 1
    sizes, n = s["counts"], len(s["sizes"])
    stream = torch.cuda.current_stream()
    vr.vr_adamw(p, g, m, v, ms, vs, master, sizes, n, _code(vr, c["dtype"]),
                _code(vr, c["grad"]), c["bits"], LR, BETA1, BETA2, ADAM_EPS, DECAY, s["step"], 1.0,
                SEED, None, stream)
    out = {"param": s["param"], "m": s["m"], "v": s["v"]}
    if c["bits"] == 8:
        vr.vr_adamw_values(m, v, ms, vs, sizes, n, mvalues, vvalues, stream)
        out.update(m=s["mvalues"], v=s["vvalues"])
    if c["master"]:
        out["master"] = s["master"]
    return out


def _own_experts(s):
    import double_binary_tree_gb300 as vr
    c, x, w, rows = s["case"], s["x"], s["weight"], s["rows"]
    K, N, E, dtype = c["dim"], c["out"], c["groups"], _code(vr, c["dtype"])
    stream = torch.cuda.current_stream()
    if not c["grads"]:
        work, size = _work(s, vr.vr_grouped_linear_workspace_bytes, x, K, w, rows, K, N, E, dtype)
        vr.vr_grouped_linear(x, K, w, s["counts"], rows, K, N, E, dtype, s["out"], N, work, size,
                             stream)
        return {"out": s["out"]}
    dy = s["dout"]
    work, size = _work(s, vr.vr_grouped_linear_grad_workspace_bytes, dy, N, x, K, w, rows, K, N, E,
                       dtype)
    vr.vr_grouped_linear_grad(dy, N, x, K, w, s["counts"], rows, K, N, E, dtype, s["dx"],
                              s["dweight"], work, size, stream)
    return {"dx": s["dx"], "dweight": s["dweight"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"embed": _own_embed, "adamw": _own_adamw, "experts": _own_experts}[op](state)
    return {"embed": _plain_embed, "adamw": _plain_adamw, "experts": _plain_experts}[op](state)


def work(case):
    size = {"fp32": 4, "fp16": 2, "bf16": 2}
    b = size[case["dtype"]]
    if case["op"] == "embed":
        T, D, V = case["tokens"], case["dim"], case["vocab"]
        # tokens that count; distinct ones, by the frequencies 1 / (n log(V + 1))
        T = max(1, round(T * (1 - case["ignored"])))
        top = math.log(V + 1)
        rows, n = 0.0, 1
        while n <= V:  # words n to 2 n - 1 are about as frequent as the middle one
            k = min(n, V + 1 - n)
            rows += k * -math.expm1(T * math.log1p(-1 / (top * 1.44 * n + 1)))
            n *= 2
        if not case["grads"]:
            return {"bytes": T * 8 + rows * D * b + case["tokens"] * D * b, "flops": T * D}
        # added to: those rows read and written; else every row written
        return {"bytes": T * 8 + T * D * b + (2 * rows if case["add"] else V) * D * b,
                "flops": 2 * T * D}
    if case["op"] == "adamw":
        n = sum(_tensors(case))
        state = 2 * (4 if case["bits"] == 32 else 1 + 4 / BLOCK)
        each = size[case["grad"]] + 2 * state + (b + 8 if case["master"] else 2 * b)
        if case["bits"] == 8:  # its values are written as well
            each += 8
        return {"bytes": n * each, "flops": n * 16}
    R, K, N = case["tokens"] * case["topk"], case["dim"], case["out"]
    E = min(case["groups"], R)  # experts that have rows
    if not case["grads"]:
        return {"bytes": (R * (K + N) + E * K * N) * b, "flops": 2 * R * K * N}
    return {"bytes": (R * (2 * K + N) + (E + case["groups"]) * K * N) * b, "flops": 4 * R * K * N}


# ------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embed":
        ids, k = s["ids"].tolist(), s["scale"]
        live = [i for i, t in enumerate(ids) if t != IGNORE]
        if not case["grads"]:
            out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
            if live:
                rows = torch.tensor(live, device="cuda")
                out[rows] = torch.index_select(s["weight"], 0, s["ids"][rows]).double().mul(k)
            return {"out": out}
        out = s["dweight"].double() if case["add"] else torch.zeros(
            case["vocab"], case["dim"], dtype=torch.float64, device="cuda")
        if live:
            # running sums over the tokens in order of their words, taken at the
            # end of each word's run, a few columns at a time
            word, order = torch.sort(s["ids"][s["ids"] != IGNORE], stable=True)
            order = torch.nonzero(s["ids"] != IGNORE)[:, 0][order]
            words, runs = torch.unique_consecutive(word, return_counts=True)
            ends = torch.cumsum(runs, 0) - 1
            for lo in range(0, case["dim"], 256):
                part = torch.cumsum(s["dout"][order, lo:lo + 256].double(), 0)[ends]
                part[1:] -= part[:-1].clone()
                out[words, lo:lo + 256] += k * part
        return {"dweight": out}
    if case["op"] == "adamw":
        few, g = case["bits"] == 8, s["grad"].double()
        m, v = s["m"], s["v"]
        if few:
            m = (m.view(torch.float8_e4m3fn).double().view(-1, BLOCK) * s["mscale"][:, None]).view(-1)
            power, digits = torch.div(v, 8, rounding_mode="floor").double(), (v % 8).double()
            v = torch.where(power > 0, (8 + digits) * torch.exp2(power - 18), digits * 2.0 ** -17)
            v = (v.view(-1, BLOCK) * s["vscale"][:, None]).view(-1)
        m, v = m.double(), v.double()
        p = (s["master"] if case["master"] else s["param"]).double()
        t = s["step"] + 1
        m = torch.lerp(g, m, BETA1)
        v = torch.lerp(g.square(), v, BETA2)
        p = p - LR * DECAY * p
        p = torch.addcdiv(p, m / (1 - BETA1 ** t), (v / (1 - BETA2 ** t)).sqrt() + ADAM_EPS,
                          value=-LR)
        out = {"param": p, "m": None if few else m, "v": None if few else v}
        if case["master"]:
            out["master"] = p
        return out
    counts, w, x = s["counts"].tolist(), s["weight"], s["x"]
    if case["grads"]:
        dx = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(w.shape, dtype=torch.float64, device="cuda")
    else:
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lo = 0
    for e, n in enumerate(counts):
        part = slice(lo, lo + n)
        if case["grads"]:
            dy = s["dout"][part].double()
            dx[part] = torch.mm(dy, w[e].double())
            dw[e] = torch.mm(dy.T, x[part].double())
        else:
            out[part] = torch.mm(x[part].double(), w[e].double().T)
        lo += n
    return {"dx": dx, "dweight": dw} if case["grads"] else {"out": out}
