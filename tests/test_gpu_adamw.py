"""vr_adamw against its definition (more_refs.py): states bit for bit, the
parameters in 64 bits."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import double_binary_tree_gb300 as vr  # noqa: E402
from tests import more_refs, operator_refs as refs  # noqa: E402
from tests.test_gpu_operator_memory import Arena  # noqa: E402

DT = {"fp32": (vr.VR_FLOAT32, torch.float32), "fp16": (vr.VR_FLOAT16, torch.float16),
      "bf16": (vr.VR_BFLOAT16, torch.bfloat16)}
HYPER = dict(lr=3e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.1, step=3, gs=0.5)
SEED = 0x123456789abcdef


class Model:
    """Tensors of the given sizes between guard bytes."""

    def __init__(self, sizes, dtype, grad, bits, master, seed=0, offset=0):
        self.arena, self.sizes, self.bits = Arena(), sizes, bits
        self.codes = DT[dtype][0], DT[grad][0]
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def tensors(ty, make, unit=1):
            size = torch.empty(0, dtype=ty).element_size()
            out = []
            for n in sizes:
                t = self.arena.like((-(-n // unit),), ty, offset * size)
                t.copy_(make(-(-n // unit)))
                out.append(t)
            return out

        def randn(n):
            return torch.randn(n, generator=g, device="cuda")

        self.p = tensors(DT[dtype][1], lambda n: 0.1 * randn(n))
        self.g = tensors(DT[grad][1], lambda n: randn(n) * torch.exp(2 * randn(n)))
        self.master = tensors(torch.float32, lambda n: 0.1 * randn(n)) if master else None
        if bits == 8:
            u8 = lambda top: lambda n: torch.randint(0, top, (n,), generator=g,  # noqa: E731
                                                     device="cuda")
            # (codes up to the largest that a block holds, both signs of m)
            self.m = tensors(torch.uint8, lambda n: u8(0x78)(n) + 128 * u8(2)(n))
            self.v = tensors(torch.uint8, u8(0xf8))
            self.ms = tensors(torch.float32, lambda n: torch.exp2(u8(6)(n) - 9.0), 256)
            self.vs = tensors(torch.float32, lambda n: torch.exp2(u8(6)(n) - 17.0), 256)
        else:
            self.m = tensors(torch.float32, randn)
            self.v = tensors(torch.float32, lambda n: randn(n) ** 2)
            self.ms = self.vs = None

    def host(self):
        def down(ts):
            return None if ts is None else [t.float().cpu().numpy() if t.is_floating_point()
                                            else t.cpu().numpy() for t in ts]
        return [down(x) for x in (self.p, self.g, self.m, self.v, self.ms, self.vs, self.master)]

    def step(self, control=None, stream=None, **hyper):
        h = dict(HYPER, **hyper)
        vr.vr_adamw(self.p, self.g, self.m, self.v, self.ms, self.vs, self.master, self.sizes,
                    len(self.sizes), *self.codes, self.bits, h["lr"], h["b1"], h["b2"], h["eps"],
                    h["wd"], h["step"], h["gs"], SEED, control,
                    stream or torch.cuda.current_stream())


def same(a, b):
    """Bit for bit, any NaN equal to any other."""
    return np.array_equal(a, b, equal_nan=a.dtype.kind == "f")


def check(model, before, **hyper):
    h = dict(HYPER, **hyper)
    assert vr.vr_stream_status() == 0
    assert model.arena.intact()
    p, g, m, v, ms, vs, master = before
    after = model.host()
    first = 0
    for i, n in enumerate(model.sizes):
        if model.bits == 8:
            with np.errstate(all="ignore"):
                m0 = more_refs.values("m", m[i], ms[i]).astype(np.float32)
                v0 = more_refs.values("v", v[i], vs[i]).astype(np.float32)
        else:
            m0, v0 = m[i], v[i]
        start = (master or p)[i]
        want, bound, m1, v1 = more_refs.adamw(start, g[i], m0, v0, **h)
        if model.bits == 8:
            bits = more_refs.random_bits(SEED, h["step"], first, n)
            for kind, x, cut, code, scale in (("m", m1, bits & np.uint64(0xffff), 2, 4),
                                              ("v", v1, bits >> np.uint64(16), 3, 5)):
                codes, scales = more_refs.encode(kind, x, cut)
                assert same(after[code][i], codes), (kind, i)
                assert same(after[scale][i], scales), (kind, i)
        else:
            assert same(after[2][i], m1) and same(after[3][i], v1), i
        fine = np.isfinite(want)
        got = torch.from_numpy((after[6] or after[0])[i])
        ty = torch.float32 if after[6] else model.p[i].dtype
        assert np.array_equal(np.isfinite(got.numpy()), fine)
        refs.assert_close(got[torch.from_numpy(fine)], torch.from_numpy(want[fine]),
                          torch.from_numpy(bound[fine]), ty, "tensor %d" % i)
        if after[6]:  # the parameters are the copies, rounded
            assert torch.equal(model.p[i], model.master[i].to(model.p[i].dtype))
        first += -(-n // 256) * 256
    return after


COMBOS = [("fp32", "fp32", False), ("fp32", "bf16", False), ("fp32", "fp16", False),
          ("bf16", "bf16", False), ("bf16", "bf16", True), ("bf16", "fp32", True),
          ("bf16", "fp16", False), ("fp16", "fp16", True), ("fp16", "fp32", False),
          ("fp16", "bf16", True)]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("dtype,grad,master", COMBOS)
def test_matches_the_definition(dtype, grad, master, bits):
    model = Model([1, 7, 0, 255, 256, 257, 4096, 3 * 4096 + 5], dtype, grad, bits, master)
    before = model.host()
    model.step()
    check(model, before)


@pytest.mark.parametrize("bits", [8, 32])
def test_many_tensors(bits):
    """More than one launch takes, a large one among them."""
    sizes = [3 + 37 * i for i in range(60)] + [700001] + [512] * 60
    model = Model(sizes, "bf16", "bf16", bits, True, seed=1)
    before = model.host()
    model.step(step=70000)
    check(model, before, step=70000)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("dtype,grad,master", COMBOS[:1] + COMBOS[4:6])
@pytest.mark.parametrize("offset", [1, 4, 8])
def test_alignment(offset, dtype, grad, master, bits):
    model = Model([9000, 33], dtype, grad, bits, master, offset=offset)
    before = model.host()
    model.step()
    check(model, before)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("hyper", [
    dict(b1=0.0), dict(b2=0.0), dict(wd=0.0), dict(gs=0.0), dict(eps=1e-3), dict(lr=0.0),
    dict(step=1), dict(step=1 << 33), dict(gs=2.0 ** -40), dict(gs=2.0 ** 30)])
def test_hyperparameters(hyper, bits):
    model = Model([1000], "fp32", "fp32", bits, False)
    before = model.host()
    model.step(**hyper)
    check(model, before, **hyper)


def test_values_of_8_bit_states():
    sizes = [1, 300, 5000, 0, 256]
    model = Model(sizes, "bf16", "bf16", 8, False)
    arena = Arena()
    out = [[arena.like((n,), torch.float32) for n in sizes] for _ in range(2)]
    vr.vr_adamw_values(model.m, model.v, model.ms, model.vs, sizes, len(sizes), *out,
                       torch.cuda.current_stream())
    assert vr.vr_stream_status() == 0 and arena.intact()
    for kind, codes, scales, got in (("m", model.m, model.ms, out[0]),
                                     ("v", model.v, model.vs, out[1])):
        for c, s, x in zip(codes, scales, got):
            want = more_refs.values(kind, c.cpu().numpy(), s.cpu().numpy())
            assert np.array_equal(x.cpu().numpy().astype(np.float64), want)
    one = [torch.empty(n, device="cuda") for n in sizes]
    vr.vr_adamw_values(None, model.v, None, model.vs, sizes, len(sizes), None, one,
                       torch.cuda.current_stream())
    assert all(torch.equal(a, b) for a, b in zip(one, out[1]))
    # m's bytes are the e4m3 format
    want = model.m[2].view(torch.float8_e4m3fn).float() * model.ms[2].repeat_interleave(256)[:5000]
    assert torch.equal(want, out[0][2])


def test_states_of_zero():
    """From nothing, and elements that never have a gradient."""
    model = Model([600], "fp32", "fp32", 8, False)
    for t in (model.m[0], model.v[0], model.ms[0], model.vs[0]):
        t.zero_()
    model.g[0][100:400] = 0.0
    for step in range(1, 4):
        before = model.host()
        model.step(step=step)
        check(model, before, step=step)
    assert not model.m[0][100:400].any() and not model.v[0][100:400].any()
    assert bool((model.v[0][:100] > 0).all())


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_gradient_that_is_not_finite_shows(bad, bits):
    model = Model([1000], "fp32", "fp32", bits, False)
    model.g[0][300] = bad
    before = model.host()
    model.step()
    after = check(model, before)
    if bits == 8:
        assert math.isnan(after[4][0][1]) and math.isfinite(after[4][0][0])


def test_tiny_and_huge_blocks():
    model = Model([256 * 6], "fp32", "fp32", 8, False)
    for b, x in enumerate((1e-30, 1e-19, 1e-10, 1e10, 1e18, 0.0)):
        model.g[0][b * 256:(b + 1) * 256] *= x
    for t in (model.ms[0], model.vs[0]):
        t.zero_()
    before = model.host()
    model.step(gs=1.0)
    check(model, before, gs=1.0)


def test_rounding_is_right_on_average():
    """A second moment whose steps are far smaller than its codes' distance
    still moves as the formula says: over 400 steps of 0.001 of itself the
    mean of 4096 elements follows within a few parts in a hundred; rounded to
    the nearest it would not move at all."""
    model = Model([4096], "fp32", "fp32", 8, False)
    for t in (model.m[0], model.v[0], model.ms[0], model.vs[0]):
        t.zero_()
    model.g[0].fill_(1.0)
    b2 = float(np.float32(0.999))
    for step in range(1, 401):
        model.step(step=step, b2=0.999, gs=1.0, lr=0.0)
        if step == 100:
            model.g[0].fill_(2.0)
    v = sum((1 - b2) * b2 ** (400 - s) * (1.0 if s <= 100 else 4.0) for s in range(1, 401))
    out = torch.empty(4096, device="cuda")
    vr.vr_adamw_values(None, model.v, None, model.vs, [4096], 1, None, [out],
                       torch.cuda.current_stream())
    # one element: each step rounds a change of at most c = 4 (1 - b2) to
    # codes that are at most an eighth of v <= 1.1 apart, a variance of at
    # most distance * change = 0.14 * 0.004 a step, 0.22 over 400 steps; the
    # mean of 4096 has a deviation of sqrt(0.22 / 4096) = 0.0074 at most: five
    assert abs(float(out.double().mean()) - v) <= 5 * 0.0074
    # the errors of neighbours are their own
    assert 0.001 < float(out.double().std()) < math.sqrt(0.22) * 2


@pytest.mark.parametrize("bits", [8, 32])
def test_control_from_device_memory(bits):
    """A captured step, replayed with other rates, steps and scales."""
    model, other = (Model([5000, 77], "bf16", "bf16", bits, True) for _ in range(2))
    control = torch.tensor([1e-3, 1.0, 1.0], device="cuda")
    model.step(control=control)  # (the library loads its kernels)
    other.step(lr=1e-3, step=1, gs=1.0)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        model.step(control=control)
    for step, lr, gs in ((2, 1e-3, 0.5), (3, 2e-3, 2.0), (4, 5e-4, 0.25)):
        control.copy_(torch.tensor([lr, float(step), gs]))
        graph.replay()
        other.step(lr=lr, step=step, gs=gs)
    assert vr.vr_stream_status() == 0
    for a, b in zip(model.host(), other.host()):
        for x, y in zip(a or [], b or []):
            if x.dtype == np.uint8:
                assert np.array_equal(x, y)
            else:
                # the factors are made on the device in 32 bits, 1 - beta^t
                # within 2^-21; the parameters, below 1, are rounded to bf16
                # (half a step is 2^-9; one that falls the other way, 2^-8)
                assert np.allclose(x, y, rtol=2.0 ** -7, atol=1e-6)
    saved = model.host()
    for bad in (math.nan, math.inf):
        control.copy_(torch.tensor([1e-3, 5.0, bad]))
        graph.replay()
    assert vr.vr_stream_status() == 0
    for a, b in zip(model.host(), saved):
        for x, y in zip(a or [], b or []):
            assert np.array_equal(x, y)


def test_lists_prepared_once_and_another_stream():
    model, other = (Model([5000, 0, 77], "bf16", "fp32", 8, True) for _ in range(2))
    lists = [vr.pointer_array(x) for x in (model.p, model.g, model.m, model.v, model.ms, model.vs,
                                           model.master)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for step in range(1, 3):
        vr.vr_adamw(*lists, vr.size_array(model.sizes), 3, *model.codes, 8, 3e-3, 0.9, 0.99, 1e-8,
                    0.1, step, 0.5, SEED, None, side)
        other.step(step=step)
    side.synchronize()
    for a, b in zip(model.host(), other.host()):
        assert all(np.array_equal(x, y) for x, y in zip(a, b))
