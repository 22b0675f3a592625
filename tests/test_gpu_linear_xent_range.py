"""vr_linear_xent where the logits are far from zero: confident tokens and large
offsets lose no digits but those of the logits themselves.  The inputs are made
so that every logit is exact in fp32 (few bits, no rounding in any order of
summation), so the bounds hold what the softmax adds alone."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import double_binary_tree_gb300 as vr  # noqa: E402
from tests import operator_refs as refs  # noqa: E402
from tests.test_gpu_linear_xent import DT, IGNORE, call  # noqa: E402


def bounds(h, w, y, scale):
    """From exact logits, in 64 bits: x = l - max is exact or rounded once, its
    product with log2 e once, ex2 to 2 ulp; a row's sum takes at most 40 fp32
    additions and products one after the other (16 columns a chain, chains,
    lanes) and one for every 1024 columns (parts of a lane)."""
    ty = h.dtype
    h, w = h.double(), w.double()
    T, V = len(y), w.shape[0]
    l = h @ w.t()
    x = l - l.amax(1, keepdim=True)
    e = torch.exp(x)
    total = e.sum(1, keepdim=True)
    rel = (3 * x.abs().clamp(max=200.0) + 8) * refs.U32       # of each e
    # the largest term is exact: ex2 of zero
    sums = ((e * rel).sum(1, keepdim=True) - 8 * refs.U32).clamp(min=0) / total + (40 + V / 1024) * refs.U32
    p = e / total
    one = torch.zeros_like(p)
    rows = torch.arange(T, device=h.device)
    one[rows, y] = 1.0
    # 1 - p of the target: what the others hold
    others = (e * (1 - one)).sum(1, keepdim=True) / total
    g = torch.where(one > 0, -others, p)
    losses = (x.logsumexp(1) - x[rows, y])
    b_losses = sums[:, 0] + (rel[rows, y] + 4 * refs.U32) * losses.abs() + refs.U32 * x[rows, y].abs()
    bg = p * (rel + sums) + g.abs() * 8 * refs.U32
    bg = bg + (2 * g.abs() + 2 * bg) * refs.U_T[ty] + \
        (2.0 ** -38 if ty == torch.float16 else 2.0 ** -126)
    s = scale / T
    more = lambda n: (n + 16) * 2.0 ** -23 * (g.abs() + bg)   # noqa: E731
    return dict(losses=losses, b_losses=b_losses, lse=torch.logsumexp(l, 1),
                loss=float(losses.mean()), b_loss=float(b_losses.mean()) * (1 + 4 * refs.U32) +
                float(losses.mean()) * 4 * refs.U32,
                dh=s * (g @ w), b_dh=s * ((bg + more(V)) @ w.abs()),
                dw=s * (g.t() @ h), b_dw=s * ((bg + more(T)).t() @ h.abs()))


def check(got, want, ty):
    losses, lse, loss, gh, gw = got
    refs.assert_close(losses, want["losses"], want["b_losses"], torch.float32, "losses")
    # lse itself is one fp32 number (a sum of two, the second rounded too)
    refs.assert_close(lse, want["lse"], want["lse"].abs() * 2 * refs.U32 + want["b_losses"],
                      torch.float32, "lse")
    assert abs(float(loss) - want["loss"]) <= want["b_loss"] + 1e-30
    if gh is not None:
        refs.assert_close(gh, want["dh"], want["b_dh"], ty, "dHidden")
        refs.assert_close(gw, want["dw"], want["b_dw"], ty, "dWeight")


def sure(T, V, ty, root, seed):
    """Logits root^2 + multiples of 1/2, the target's about 20 above the rest."""
    D = 64
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = 0.25 * torch.randint(-1, 2, (V, D), generator=g, device="cuda").float()
    y = torch.randperm(V, generator=g, device="cuda")[:T]
    h = 8 * w[y]
    h[:, 0] = root
    w[:, 0] = root
    return h.to(ty), w.to(ty), y


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("root", [0.0, 8.0, 32.0, 128.0])
@pytest.mark.parametrize("T,V,grads", [(12, 700, True), (300, 700, True), (5, 700, False),
                                       (300, 700, False)])
def test_confident_tokens(T, V, grads, root, dtype):
    code, ty = DT[dtype]
    h, w, y = sure(T, V, ty, root, 3)
    scale = 64.0 * T if dtype == "fp16" else 1.0
    want = bounds(h, w, y, scale)
    assert 1e-7 < float(want["losses"].median()) < 1e-3
    got = call(h, w, y, code, scale=scale, dh=grads, dw=grads)
    assert vr.vr_stream_status() == 0
    check(got, want, ty)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("root", [8.0, 128.0])
def test_confident_tokens_with_the_vocabulary_in_pieces(root, dtype):
    T, V = 300, 380000
    code, ty = DT[dtype]
    h, w, y = sure(T, V, ty, root, 4)
    scale = 64.0 * T if dtype == "fp16" else 1.0
    got = call(h, w, y, code, scale=scale)
    assert vr.vr_stream_status() == 0
    check(got, bounds(h, w, y, scale), ty)


@pytest.mark.parametrize("grads", [True, False])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("power", [10, 14, 17, 20, 30])
def test_large_equal_logits(power, sign, grads):
    """All logits 2^(2 power), from 1e6 to 1e18: a uniform softmax."""
    T, D, V = 40, 16, 700
    h = torch.zeros(T, D, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(V, D, device="cuda", dtype=torch.bfloat16)
    h[:, 3] = 2.0 ** power
    w[:, 3] = sign * 2.0 ** power
    y = torch.arange(T, device="cuda") * 17
    got = call(h, w, y, vr.VR_BFLOAT16, dh=grads, dw=grads)
    check(got, bounds(h, w, y, 1.0), torch.bfloat16)
