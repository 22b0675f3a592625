"""Embedding, AdamW and grouped products in 64 bits (8-bit states: in 32, each
operation rounded by itself, as they are defined), with bounds on what the
operators' arithmetic may differ by.  Shares no code with the package."""

import numpy as np
import torch

U32 = 2.0 ** -24


def embedding(weight, ids, scale):
    """Rows of valid ids (others zero) and a bound before the last rounding:
    one multiplication in fp32."""
    V = weight.shape[0]
    valid = (ids >= 0) & (ids < V)
    out = weight.double()[ids.clamp(0, V - 1)] * scale
    out[~valid] = 0.0
    return out, out.abs() * U32


def embedding_grad(dout, ids, vocab, scale, old=None):
    """The table's gradient and a bound: n terms summed in fp32 in any order
    (n - 1 roundings), scaled and added to what was there (two more)."""
    valid = (ids >= 0) & (ids < vocab)
    at, rows = ids[valid], dout[valid].double()
    shape = (vocab, dout.shape[1])
    total = torch.zeros(shape, dtype=torch.float64, device=dout.device)
    size = torch.zeros_like(total)
    n = torch.zeros(vocab, dtype=torch.float64, device=dout.device)
    for t in range(len(at)) if len(at) < 64 else ():
        total[at[t]] += rows[t]
        size[at[t]] += rows[t].abs()
        n[at[t]] += 1
    if len(at) >= 64:
        total.index_add_(0, at, rows)
        size.index_add_(0, at, rows.abs())
        n.index_add_(0, at, torch.ones(len(at), dtype=torch.float64, device=dout.device))
    bound = abs(scale) * size * (n + 2)[:, None] * U32
    total = total * scale
    if old is not None:
        total = total + old.double()
        bound = bound + total.abs() * U32
    return total, bound


def mix(x):
    x = np.asarray(x, dtype=np.uint64)
    x = x ^ (x >> np.uint64(16))
    x = (x * np.uint64(0x6a09e667)) & np.uint64(0xffffffff)
    x = x ^ (x >> np.uint64(15))
    x = (x * np.uint64(0xbb67ae85)) & np.uint64(0xffffffff)
    return x ^ (x >> np.uint64(16))


def random_bits(seed, step, first, n):
    """32 random bits of the elements first .. first + n - 1."""
    key = mix(mix(seed & 0xffffffff) ^ np.uint64(seed >> 32))
    key = mix(mix(key ^ np.uint64(step & 0xffffffff)) ^ np.uint64(step >> 32))
    at = np.arange(first, first + n, dtype=np.uint64)
    return mix(mix(key ^ (at >> np.uint64(32))) ^ (at & np.uint64(0xffffffff)))


# m: e4m3, largest value of a block in [2^7, 2^8); v: five bits of exponent
# and three of mantissa, largest in [2^15, 2^16)
TOP = {"m": 7, "v": 15}
BIAS = {"m": 7, "v": 15}


def values(kind, codes, scales):
    """What codes stand for, from the formats' definition, in 64 bits."""
    c = codes.astype(np.int64)
    sign = np.where((c & 128) != 0, -1.0, 1.0) if kind == "m" else 1.0
    c = c & 127 if kind == "m" else c
    e, f = c >> 3, c & 7
    x = np.where(e > 0, (8.0 + f) * 2.0 ** (e - 3.0 - BIAS[kind]), f * 2.0 ** (-2.0 - BIAS[kind]))
    return sign * x * np.repeat(scales.astype(np.float64), 256)[:len(codes)]


def encode(kind, x, cut):
    """Codes and scales of fp32 values x: the neighbours of each value in the
    format, the upper one if the rest, in 2^-16 steps of... `cut` decides (16
    random bits)."""
    n = len(x)
    blocks = -(-n // 256)
    codes = np.zeros(n, dtype=np.uint8)
    scales = np.zeros(blocks, dtype=np.float32)
    for b in range(blocks):
        part = x[b * 256:(b + 1) * 256]
        if not np.isfinite(part).all():
            scales[b] = np.nan
            continue
        top = float(np.abs(part).max())
        e = max(int(np.floor(np.log2(top))) if top >= 2.0 ** -126 else -127, -110)
        scales[b] = np.float32(2.0 ** (e - TOP[kind]))
        # in units of the lowest code, exactly: 2^-20 of them are kept
        y = np.abs(part.astype(np.float64)) * 2.0 ** (TOP[kind] - e)
        ex = np.maximum(np.floor(np.log2(np.maximum(y, 2.0 ** -200))), 1.0 - BIAS[kind])
        units = y * 2.0 ** (3.0 - ex)                 # spacing of codes here is 1
        # digits below 2^-20 of the spacing: rounded to it where the format's
        # numbers are denormal, none elsewhere
        units = np.rint(units * 2.0 ** 20) * 2.0 ** -20
        c = np.floor(units + cut[b * 256:b * 256 + len(part)].astype(np.float64) * 2.0 ** -16)
        c = c + (ex + BIAS[kind] - 1.0) * 8.0          # 8 codes to an exponent
        if kind == "v":
            c = np.where(part > 0, np.maximum(c, 1), c)
        else:
            c = np.where(np.signbit(part), c + 128, c)  # (a zero keeps its sign)
        codes[b * 256:b * 256 + len(part)] = c.astype(np.uint8)
    return codes, scales


def adamw(p, g, m, v, lr, b1, b2, eps, wd, step, gs):
    """One step in 64 bits of fp32 inputs, new m and v in fp32 with each
    operation rounded, and a bound on p before its rounding to a type."""
    f = np.float32
    with np.errstate(all="ignore"):
        x = g.astype(f) * f(gs)
        m32 = m.astype(f) * f(b1) + x * (f(1) - f(b1))
        v32 = v.astype(f) * f(b2) + (x * x) * (f(1) - f(b2))
        b1, b2, lr, eps, wd, gs = (float(f(t)) for t in (b1, b2, lr, eps, wd, gs))
        x = g.astype(np.float64) * gs
        m64 = m.astype(np.float64) * b1 + x * (1 - b1)
        v64 = v.astype(np.float64) * b2 + x * x * (1 - b2)
        # states are 32-bit numbers: what overflows there is infinite (a square
        # of a gradient above 1.8e20 with 1 - b2 = 0.01), and p is made of that
        m64, v64 = (np.where(np.isfinite(t32), t64, t32)
                    for t32, t64 in ((m32, m64), (v32, v64)))
        up, root = lr / (1 - b1 ** step), np.sqrt(v64 / (1 - b2 ** step))
        move = up * m64 / (root + eps)
        p64 = p.astype(np.float64)
        want = p64 * (1 - lr * wd) - move
        # m: three roundings of terms that may cancel; v: five of positive
        # ones, halved by the root; the root and the division, 2 ulp each, and
        # four factors; p: its factor and the last sum
        size = np.abs(m.astype(np.float64)) * b1 + np.abs(x) * (1 - b1)
        bound = abs(up) * 3 * U32 * size / (root + eps) + np.abs(move) * 16 * U32
        bound = bound + (np.abs(p64) * 3 + np.abs(want)) * U32 + 1e-44
    return want, bound, m32, v32


def grouped(x, weight, counts):
    """Rows of each group times its weight, and a bound: fp32 sums that may
    truncate, 2^-23 a term."""
    K = x.shape[1]
    out = torch.zeros(x.shape[0], weight.shape[1], dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(out)
    lo = 0
    for e, n in enumerate(counts):
        a, b = x[lo:lo + n].double(), weight[e].double()
        out[lo:lo + n] = a @ b.t()
        bound[lo:lo + n] = (K + 16) * 2.0 ** -23 * (a.abs() @ b.abs().t())
        lo += n
    return out, bound


def grouped_grad(dout, x, weight, counts):
    dx, bx = grouped(dout, weight.transpose(1, 2), counts)
    dw = torch.zeros(weight.shape, dtype=torch.float64, device=x.device)
    bw = torch.zeros_like(dw)
    lo = 0
    for e, n in enumerate(counts):
        a, b = dout[lo:lo + n].double(), x[lo:lo + n].double()
        dw[e] = a.t() @ b
        bw[e] = (n + 16) * 2.0 ** -23 * (a.abs().t() @ b.abs())
        lo += n
    return dx, bx, dw, bw
