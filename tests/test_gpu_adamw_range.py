"""vr_adamw over its whole range: blocks of 8-bit states with every exponent,
none that becomes infinite, second moments near the largest number, decays far
below an ulp of 1, and what a control block may change."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import double_binary_tree_gb300 as vr  # noqa: E402
from tests import more_refs, operator_refs as refs  # noqa: E402
from tests.test_gpu_adamw import HYPER, SEED, Model, check, same  # noqa: E402

EXPONENTS = torch.arange(-110, 128)


def check_blocks(model, before, **hyper):
    """8-bit states bit for bit; parameters as `check` has them where they are
    32-bit numbers.  (A loaded v of code 0 beside an m of 2^100 moves a parameter
    by lr m / eps: what is 2^128 and more in 64 bits is infinite in 32, and what is
    above 2^127 may be, with the bound's 16 roundings.)"""
    h = dict(HYPER, **hyper)
    assert vr.vr_stream_status() == 0 and model.arena.intact()
    p, g, m, v, ms, vs, _ = (x and x[0] for x in before)
    after = [x and x[0] for x in model.host()]
    m0, v0 = (more_refs.values(*x).astype(np.float32) for x in (("m", m, ms), ("v", v, vs)))
    want, bound, m1, v1 = more_refs.adamw(p, g, m0, v0, **h)
    bits = more_refs.random_bits(SEED, h["step"], 0, len(p))
    for kind, x, cut, code, scale in (("m", m1, bits & np.uint64(0xffff), 2, 4),
                                      ("v", v1, bits >> np.uint64(16), 3, 5)):
        codes, scales = more_refs.encode(kind, x, cut)
        assert same(after[code], codes) and same(after[scale], scales), kind
    small, large = np.abs(want) <= 2.0 ** 127, np.abs(want) >= 2.0 ** 128 * (1 + 2.0 ** -18)
    assert np.isinf(after[0][large]).all()
    assert np.array_equal(np.sign(after[0][large]), np.sign(want[large]))
    refs.assert_close(torch.from_numpy(after[0][small]), torch.from_numpy(want[small]),
                      torch.from_numpy(bound[small]), torch.float32, "parameters")
    return after


def test_loaded_blocks_of_every_exponent():
    """States whose largest values begin at 2^-110 to 2^127, kept by a step
    without a gradient.  (A step number at which 1 - beta^t is 1.)"""
    n = len(EXPONENTS)
    model = Model([256 * n], "fp32", "fp32", 8, False)
    model.ms[0].copy_(torch.exp2(EXPONENTS.double() - 7))
    model.vs[0].copy_(torch.exp2(EXPONENTS.double() - 15))
    model.g[0].zero_()
    before = model.host()
    model.step(step=1 << 20)
    after = check_blocks(model, before, step=1 << 20)
    assert all(np.isfinite(after[i]).all() for i in (4, 5))


@pytest.mark.parametrize("wide", [False, True])
def test_blocks_of_gradients_of_every_exponent(wide):
    """v = g^2 and m = g (both betas 0): the largest squares begin at 2^-110 to
    2^127, none of them infinite; the others as large, or smaller by up to 2^40."""
    n = len(EXPONENTS)
    model = Model([256 * n], "fp32", "fp32", 8, False)
    g = torch.Generator()
    g.manual_seed(7)
    u = torch.rand(n, 256, generator=g, dtype=torch.float64)
    square = torch.exp2(EXPONENTS.double())[:, None] * (1.0 + 0.7 * u)
    if wide:
        square[:, 1:] *= torch.exp2(-40 * torch.rand(n, 255, generator=g, dtype=torch.float64))
    sign = torch.randint(0, 2, (n, 256), generator=g) * 2 - 1
    model.g[0].copy_((square.sqrt() * sign).reshape(-1))
    before = model.host()
    assert np.isfinite(before[1][0] * before[1][0]).all()
    model.step(b1=0.0, b2=0.0, gs=1.0, step=1)
    after = check_blocks(model, before, b1=0.0, b2=0.0, gs=1.0, step=1)
    assert np.isfinite(after[5]).all()
    # a second moment is its code's value, an eighth of it above or below at most
    # (from 8 of the lowest code on, where codes are 1 apart, an eighth; what is just
    # below may be rounded up to code 8, a seventh)
    v = more_refs.values("v", after[3], after[5])
    x = np.square(before[1][0].astype(np.float64))
    live = after[3] > 8
    assert live.any() and (np.abs(v - x)[live] <= x[live] / 8).all()


def test_finite_states_stay_finite():
    """Values between the largest code's below 2^128 and 2^128 are not rounded
    up to infinity."""
    model = Model([512], "fp32", "fp32", 8, False)
    for t in (model.m[0], model.v[0], model.ms[0], model.vs[0]):
        t.zero_()
    g = torch.Generator()
    g.manual_seed(8)
    u = 1.88 + 0.11 * torch.rand(512, generator=g, dtype=torch.float64)
    x = torch.cat([(u[:256] * 2.0 ** 127).sqrt(), u[256:] * 2.0 ** 127])  # v's block, m's block
    sign = torch.randint(0, 2, (512,), generator=g) * 2 - 1
    model.g[0].copy_(x * sign)
    grad = model.g[0].cpu().numpy()
    with np.errstate(over="ignore"):
        assert np.isfinite((grad * grad)[:256]).all()
    model.step(b1=0.0, b2=0.0, gs=1.0, step=1)
    out = [torch.empty(512, device="cuda") for _ in range(2)]
    vr.vr_adamw_values(model.m, model.v, model.ms, model.vs, [512], 1, out[:1], out[1:],
                       torch.cuda.current_stream())
    assert vr.vr_stream_status() == 0 and model.arena.intact()
    assert bool(torch.isfinite(out[0]).all()) and bool(torch.isfinite(out[1][:256]).all())
    # otherwise as the definition says: its code above the largest becomes that
    bits = more_refs.random_bits(SEED, 1, 0, 512)
    with np.errstate(over="ignore"):
        for kind, x, cut, got, most in (("m", grad, bits & np.uint64(0xffff), model.m[0], 0x77),
                                        ("v", (grad * grad)[:256], (bits >> np.uint64(16))[:256],
                                         model.v[0][:256], 0xf7)):
            codes, _ = more_refs.encode(kind, x, cut)
            digits = codes & 0x7f if kind == "m" else codes
            # (m's first block lies lower and keeps its codes)
            top = np.abs(x) >= 2.0 ** 127
            assert (digits[top] > most).any()
            want = np.where(top, np.minimum(digits, most), digits) + (codes - digits)
            assert same(got.cpu().numpy(), want.astype(np.uint8)), kind


def test_second_moments_near_the_largest_number():
    """v / (1 - beta2^t) may pass 2^128 in the first steps; its root does not."""
    model = Model([5000], "fp32", "fp32", 32, False)
    model.v[0].copy_(2.0 ** 127 * (0.4 + 1.5 * torch.rand(5000, device="cuda")))
    model.m[0].mul_(2.0 ** 62)
    model.g[0].zero_()
    before = model.host()
    model.step(step=1)
    after = check(model, before, step=1)
    assert float(np.abs(after[0][0] - before[0][0]).mean()) > 1e-4


@pytest.mark.parametrize("control", [False, True])
@pytest.mark.parametrize("dtype,bits,master", [("fp32", 32, False), ("bf16", 32, True),
                                               ("bf16", 8, True)])
@pytest.mark.parametrize("lr,wd", [(1e-6, 0.01), (3e-6, 0.01), (1e-5, 0.01), (2e-7, 0.1)])
def test_small_decays(lr, wd, dtype, bits, master, control):
    """lr * weightDecay below or about an ulp of 1: a parameter's change is
    right on average."""
    n = 1 << 20
    model = Model([n], dtype, dtype, bits, master)
    start = (model.master or model.p)[0]
    start.copy_(0.5 + 0.5 * torch.rand(n, device="cuda"))
    if bits == 8:  # (the steps are a few lr, hundreds of ulp at most)
        model.m[0].copy_(0x30 + 128 * torch.randint(0, 2, (n,), device="cuda"))
        model.v[0].copy_(0x70 + torch.randint(0, 8, (n,), device="cuda"))
        model.ms[0].fill_(1.0)
        model.vs[0].fill_(1.0)
    else:
        model.v[0].add_(0.1)
    model.g[0].copy_(torch.randn(n, device="cuda"))
    before = model.host()
    hyper = dict(lr=lr, wd=wd, step=5000, gs=1.0)
    block = torch.tensor([lr, 5000.0, 1.0], device="cuda") if control else None
    model.step(control=block, **hyper)
    assert vr.vr_stream_status() == 0
    after = model.host()
    p = (before[6] or before[0])[0].astype(np.float64)
    if bits == 8:
        m, v = (more_refs.values(k, c[0], s[0]).astype(np.float32)
                for k, c, s in (("m", before[2], before[4]), ("v", before[3], before[5])))
    else:
        m, v = before[2][0], before[3][0]
    want, *_ = more_refs.adamw(p.astype(np.float32), before[1][0], m, v, lr, 0.9, 0.99, 1e-8, wd,
                               5000, 1.0)
    off = float(np.mean((after[6] or after[0])[0].astype(np.float64) - want))
    # p is rounded once: to 2^-24 below 1 (2^-23 for what passes 1), an error between
    # -2^-25 and 2^-25 with a deviation of 2^-25 / sqrt(3), of the mean's 2^10
    # times less: six of those, and 20 roundings of the step's terms (the control
    # block's factors are made in 32 bits: 2^-20)
    move = float(np.mean(np.abs(want - p)))
    assert abs(off) <= 6 * 2.0 ** -24 / math.sqrt(3 * n) + 2.0 ** -19 * move
    assert 6 * 2.0 ** -24 / math.sqrt(3 * n) + 2.0 ** -19 * move < 0.2 * lr * wd * 0.75


@pytest.mark.parametrize("bits", [8, 32])
def test_infinite_parameters_stay(bits):
    """A parameter of minus infinity (a mask) without a gradient stays one."""
    model = Model([600], "fp32", "fp32", bits, False)
    model.p[0][5:300:7] = -math.inf
    model.p[0][1] = math.inf
    for t in (model.m[0], model.g[0]):
        t[:300].zero_()
    before = model.host()
    for wd in (0.1, 0.0):
        model.step(wd=wd)
        got = model.host()[0][0]
        for x in (math.inf, -math.inf):
            assert np.array_equal(got == x, before[0][0] == x)
        assert not np.isnan(got).any()


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("fp16", "fp32")])
def test_control_changes_factors_only(dtype, grad, bits):
    """Steps with their numbers in device memory and as arguments: the same
    states bit for bit, masters within the factors' precision."""
    model, other = (Model([5000, 77, 300], dtype, grad, bits, True) for _ in range(2))
    moved = [torch.zeros_like(w) for w in other.master]
    for step, lr, gs in ((1, 1e-3, 1.0), (2, 1e-3, 0.5), (3, 2e-3, 2.0), (4, 5e-4, 0.25)):
        old = [w.clone() for w in other.master]
        model.step(control=torch.tensor([lr, float(step), gs], device="cuda"))
        other.step(lr=lr, step=step, gs=gs)
        for a, w, o in zip(moved, other.master, old):
            a.add_((w - o).abs())
    assert vr.vr_stream_status() == 0
    for i in (2, 3, 4, 5):
        for x, y in zip(model.host()[i] or [], other.host()[i] or []):
            assert same(x, y), i
    for i, (x, y) in enumerate(zip(model.master, other.master)):
        # 1 - beta^t: the logarithm, its product with t, expm1 (1 ulp) and the
        # division, 2^-21 in all, of the two factors; decay's factor one
        # rounding; a rounding of p each step on both sides
        bound = moved[i] * 2.0 ** -20 + 8 * 2.0 ** -24 * (y.abs() + moved[i])
        assert bool(((x - y).abs() <= bound).all())
        assert torch.equal(model.p[i], x.to(model.p[i].dtype))
