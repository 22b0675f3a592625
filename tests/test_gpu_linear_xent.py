"""vr_linear_xent against its definition in 64 bits (operator_refs.py)."""

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import double_binary_tree_gb300 as vr  # noqa: E402
from tests import operator_refs as refs  # noqa: E402

DT = {"fp16": (vr.VR_FLOAT16, torch.float16), "bf16": (vr.VR_BFLOAT16, torch.bfloat16)}
IGNORE = -100


def make(T, D, V, ty, seed, ignored=0.0, spread=2.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = torch.randn(T, D, generator=g, device="cuda").to(ty)
    w = (torch.randn(V, D, generator=g, device="cuda") * (spread / math.sqrt(D))).to(ty)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y[torch.rand(T, generator=g, device="cuda") < ignored] = IGNORE
    return h, w, y


def call(h, w, y, code, mean=True, scale=1.0, dh=True, dw=True, ignore=IGNORE, stream=None,
         least=False):
    T, D = h.shape
    V = w.shape[0]
    losses = torch.full((T,), math.nan, device="cuda")
    lse = torch.full((T,), math.nan, device="cuda")
    loss = torch.full((1,), math.nan, device="cuda")
    gh = torch.full((T, D), math.nan, device="cuda", dtype=h.dtype) if dh else None
    gw = torch.full((V, D), math.nan, device="cuda", dtype=h.dtype) if dw else None
    hs, ws = max(h.stride(0), D), max(w.stride(0), D)
    n = vr.vr_linear_xent_workspace_bytes(h, hs, w, ws, T, D, V, code,
                                          0 if not (dh or dw) else 2 if least else 1)
    # a workspace that holds NaN at the start
    work = torch.full((n,), 255, device="cuda", dtype=torch.uint8)
    vr.vr_linear_xent(h, hs, w, ws, y, T, D, V, code, ignore, mean, scale, losses, lse, loss, gh,
                      gw, work, n, stream or torch.cuda.current_stream())
    return losses, lse, loss, gh, gw


def compare(got, want, ty, norm=True):
    """`norm`: the 2-norm of the gradients' errors too -- for inputs without
    cancellation only.  Where softmax minus one-hot is itself a difference of
    nearly equal numbers, or a column of the weight is the same for all
    rows (the sum of a row of factors is zero, that of the rounded ones is
    not), the elementwise bound is the one that holds."""
    losses, lse, loss, gh, gw = got
    refs.assert_close(lse, want["lse"], want["b_lse"], torch.float32, "lse")
    refs.assert_close(losses, want["losses"], want["b_losses"], torch.float32, "losses")
    assert abs(float(loss) - want["loss"]) <= want["b_loss"] + 1e-30
    # norm: three independent roundings to the type at most, each u / sqrt(3)
    # at most on average
    if gh is not None:
        refs.assert_close(gh, want["dh"], want["b_dh"], ty, "dHidden")
        assert not norm or refs.norm_error(gh, want["dh"]) <= refs.U_T[ty]
    if gw is not None:
        refs.assert_close(gw, want["dw"], want["b_dw"], ty, "dWeight")
        assert not norm or refs.norm_error(gw, want["dw"]) <= refs.U_T[ty]


def check(h, w, y, dtype, mean=True, scale=1.0, norm=True, **kw):
    code, ty = DT[dtype]
    got = call(h, w, y, code, mean, scale, **kw)
    assert vr.vr_stream_status() == 0
    want = refs.xent(h, w, y, kw.get("ignore", IGNORE), mean, scale)
    compare(got, want, ty, norm)
    return got, want


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,D,V", [
    (1, 8, 1), (1, 64, 1000), (2, 128, 256), (5, 72, 257), (64, 64, 128), (127, 200, 511),
    (128, 256, 512), (129, 320, 1025), (300, 1024, 4099), (513, 96, 2000), (1000, 512, 777)])
def test_matches_the_definition(T, D, V, dtype):
    h, w, y = make(T, D, V, DT[dtype][1], T + D + V)
    check(h, w, y, dtype, scale=64.0 * T if dtype == "fp16" else 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,D,V", [(3, 1, 5), (33, 7, 300), (130, 65, 1000), (200, 333, 1111)])
def test_sizes_that_are_no_multiple_of_eight(T, D, V, dtype):
    h, w, y = make(T, D, V, DT[dtype][1], T + D + V)
    check(h, w, y, dtype, mean=False, scale=64.0 if dtype == "fp16" else 1.0)


def test_several_pieces_of_the_vocabulary():
    """40 000 x 4096 gradient factors are more than one piece; T is ragged."""
    h, w, y = make(4001, 64, 40000, torch.bfloat16, 3, ignored=0.1)
    check(h, w, y, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,D,V", [(1, 64, 700), (100, 264, 3000), (700, 130, 2500)])
def test_the_least_workspace(T, D, V, dtype):
    """Without room for the numerators the vocabulary goes in pieces; the loss
    is the same to the bit."""
    h, w, y = make(T, D, V, DT[dtype][1], 21, ignored=0.2)
    scale = 64.0 * T if dtype == "fp16" else 1.0
    a, _ = check(h, w, y, dtype, scale=scale, least=True)
    b = call(h, w, y, DT[dtype][0], scale=scale)
    assert all(torch.equal(x, z) for x, z in zip(a[:3], b[:3]))


@pytest.mark.parametrize("ignored", [0.3, 0.9])
def test_ignored_tokens_are_left_out_whatever_they_hold(ignored):
    h, w, y = make(400, 136, 1500, torch.bfloat16, 4, ignored=ignored)
    rows = (y == IGNORE).nonzero()[:, 0]
    clean = h.clone()
    h[rows[0]] = math.nan
    h[rows[1]] = math.inf
    h[rows[2]] = torch.finfo(h.dtype).min
    got = call(h, w, y, vr.VR_BFLOAT16)
    want = refs.xent(clean, w, y, IGNORE, True, 1.0)
    keep = torch.ones(400, dtype=torch.bool, device="cuda")
    keep[rows[:3]] = False
    refs.assert_close(got[1][keep], want["lse"][keep], want["b_lse"][keep], torch.float32, "lse")
    refs.assert_close(got[0], want["losses"], want["b_losses"], torch.float32, "losses")
    refs.assert_close(got[3], want["dh"], want["b_dh"], torch.bfloat16, "dHidden")
    refs.assert_close(got[4], want["dw"], want["b_dw"], torch.bfloat16, "dWeight")
    assert not got[3][rows].any()


def test_nothing_counts():
    h, w, y = make(50, 64, 500, torch.bfloat16, 5)
    y[:] = IGNORE
    losses, lse, loss, gh, gw = call(h, w, y, vr.VR_BFLOAT16)
    assert float(loss) == 0.0 and not losses.any() and not gh.any() and not gw.any()
    refs.assert_close(lse, *[refs.xent(h, w, y, IGNORE, True, 1.0)[k] for k in ("lse", "b_lse")],
                      torch.float32)


def test_no_tokens():
    h, w, y = make(1, 64, 500, torch.bfloat16, 6)
    losses, lse, loss, gh, gw = call(h[:0], w, y[:0], vr.VR_BFLOAT16)
    assert float(loss) == 0.0 and not gw.any()


def test_a_target_outside_the_vocabulary_is_reported_and_ignored():
    h, w, y = make(20, 64, 500, torch.bfloat16, 7)
    y[3], y[4] = 500, -1
    assert vr.vr_stream_status() == 0
    got = call(h, w, y, vr.VR_BFLOAT16)
    assert vr.vr_stream_status() == vr.VR_ERR_INVALID_ARGUMENT
    compare(got, refs.xent(h, w, y, IGNORE, True, 1.0), torch.bfloat16)


def test_ignore_index_inside_the_vocabulary():
    h, w, y = make(90, 64, 50, torch.bfloat16, 8)
    check(h, w, y, "bf16", ignore=7)


@pytest.mark.parametrize("dh,dw", [(True, False), (False, True), (False, False)])
def test_gradients_are_optional(dh, dw):
    h, w, y = make(140, 128, 900, torch.bfloat16, 9, ignored=0.2)
    full = call(h, w, y, vr.VR_BFLOAT16)
    part = call(h, w, y, vr.VR_BFLOAT16, dh=dh, dw=dw)
    for f, p in zip(full, part):
        assert p is None or torch.equal(f, p)


@pytest.mark.parametrize("stride,offset", [(80, 0), (80, 8), (83, 0), (64, 1), (72, 3)])
def test_strides_and_alignment(stride, offset):
    T, D, V = 70, 64, 300
    bh = torch.randn(T * stride + 16, device="cuda").to(torch.bfloat16)
    bw = torch.randn(V * stride + 16, device="cuda").to(torch.bfloat16)
    h = bh.as_strided((T, D), (stride, 1), offset)
    w = bw.as_strided((V, D), (stride, 1), offset)
    y = torch.randint(0, V, (T,), device="cuda")
    check(h, w, y, "bf16")


@pytest.mark.parametrize("case", ["sure", "far apart", "very negative"])
def test_extreme_logits(case):
    h, w, y = make(60, 64, 700, torch.bfloat16, 10)
    if case == "sure":            # targets far above the rest: losses near 0
        h += 8 * w[y]
    elif case == "far apart":     # logits of thousands
        h *= 64
    else:                         # every logit far below zero
        w[:, 0] = -40.0
        h[:, 0] = 40.0
    check(h, w, y, "bf16", norm=False)


def test_another_stream_and_the_same_bits_twice():
    h, w, y = make(700, 256, 3001, torch.bfloat16, 11, ignored=0.1)
    a = call(h, w, y, vr.VR_BFLOAT16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = call(h, w, y, vr.VR_BFLOAT16, stream=side)
    side.synchronize()
    assert all(torch.equal(x, z) for x, z in zip(a, b))


def test_in_a_graph():
    h, w, y = make(300, 128, 1000, torch.bfloat16, 12)
    want = call(h, w, y, vr.VR_BFLOAT16)
    out = [torch.zeros_like(x) for x in want]
    n = vr.vr_linear_xent_workspace_bytes(h, 128, w, 128, 300, 128, 1000, vr.VR_BFLOAT16, True)
    work = torch.empty(n, device="cuda", dtype=torch.uint8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vr.vr_linear_xent(h, 128, w, 128, y, 300, 128, 1000, vr.VR_BFLOAT16, IGNORE, True, 1.0,
                          *out, work, n, torch.cuda.current_stream())
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, z) for x, z in zip(want, out))


def test_gradient_against_differences():
    """Central differences of the 64-bit loss, along random directions."""
    T, D, V = 24, 64, 200
    h, w, y = make(T, D, V, torch.bfloat16, 13)
    _, _, _, gh, gw = call(h, w, y, vr.VR_BFLOAT16)

    def value(a, b):
        l = a @ b.t()
        return float((torch.logsumexp(l, 1) - l.gather(1, y[:, None])[:, 0]).mean())

    hd, wd, eps = h.double(), w.double(), 1e-4
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for _ in range(4):
        a = torch.randn(T, D, generator=g, device="cuda", dtype=torch.float64)
        b = torch.randn(V, D, generator=g, device="cuda", dtype=torch.float64)
        num = (value(hd + eps * a, wd + eps * b) - value(hd - eps * a, wd - eps * b)) / (2 * eps)
        mine = float((gh.double() * a).sum() + (gw.double() * b).sum())
        # each gradient element is off by at most two roundings of the type
        slack = 2 * 2.0 ** -8 * float((gh.double() * a).norm() + (gw.double() * b).norm())
        assert abs(num - mine) <= 4 * slack + 1e-6
