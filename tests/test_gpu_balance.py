"""vr_balance_loss against its definition in 64 bits (operator_refs.py)."""

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import double_binary_tree_gb300 as vr  # noqa: E402
from tests import operator_refs as refs  # noqa: E402

DT = {"fp32": (vr.VR_FLOAT32, torch.float32), "fp16": (vr.VR_FLOAT16, torch.float16),
      "bf16": (vr.VR_BFLOAT16, torch.bfloat16)}


def call(logits, masks, topk, dtype, coef=0.01, scale=1.0, grads=True, chosen=True, stride=None,
         out=None, stream=None):
    R, (T, E) = len(logits), logits[0].shape
    loss = torch.full((1,), math.nan, device="cuda")
    counts = torch.full((E,), -7, device="cuda", dtype=torch.int32)
    picks = [torch.full((T, topk), -7, device="cuda", dtype=torch.int32) for _ in range(R)]
    if out is None:
        out = [torch.full_like(x, math.nan) for x in logits]
    n = vr.vr_balance_loss_workspace_bytes(R, T, E)
    # a workspace that holds NaN at the start
    work = torch.full((n,), 255, device="cuda", dtype=torch.uint8)
    vr.vr_balance_loss(logits, stride or E, masks, R, T, E, topk, dtype, coef, scale, loss, counts,
                       picks if chosen else None, out if grads else None, work, n,
                       stream or torch.cuda.current_stream())
    return loss, counts, picks, out


def check(logits, masks, topk, dtype, coef=0.01, scale=1.0, **kw):
    code, ty = DT[dtype]
    loss, counts, picks, out = call(logits, masks, topk, code, coef, scale, **kw)
    assert vr.vr_stream_status() == 0
    want = refs.balance([x.cpu() for x in logits],
                        None if masks is None else [None if m is None else m.cpu() for m in masks],
                        topk, coef, scale)
    assert counts.cpu().tolist() == want["counts"].tolist()
    for r in range(len(logits)):
        assert torch.equal(picks[r].cpu().long(), want["chosen"][r])
        refs.assert_close(out[r].cpu(), want["grads"][r], want["bound"][r], ty, "rank %d" % r)
    assert abs(float(loss) - want["loss"]) <= want["loss_bound"] + 1e-30
    return want


def draw(R, T, E, ty, seed, spread=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(spread * torch.randn(T, E, generator=g, device="cuda")).to(ty) for _ in range(R)]


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("R,T,E,k", [
    (1, 1, 1, 1), (1, 1, 8, 2), (4, 16, 8, 2), (3, 5, 7, 7), (2, 33, 60, 8), (7, 9, 64, 6),
    (2, 40, 65, 4), (2, 70, 128, 8), (1, 200, 256, 8), (2, 31, 257, 3), (1, 37, 512, 32),
    (2, 19, 1000, 5), (1, 11, 1024, 8), (64, 3, 16, 1), (2, 3000, 24, 2)])
def test_matches_the_definition(R, T, E, k, dtype):
    code, ty = DT[dtype]
    logits = draw(R, T, E, ty, 31 * R + T + E)
    scale = float(64 * T * R) if dtype == "fp16" else 1.0
    check(logits, None, k, dtype, scale=scale)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_masked_tokens_are_left_out_whatever_they_hold(dtype):
    code, ty = DT[dtype]
    logits = draw(3, 50, 96, ty, 5)
    masks = [(torch.rand(50, device="cuda") < 0.6).to(torch.uint8) for _ in range(2)] + [None]
    for r in range(2):
        rows = (masks[r] == 0).nonzero()[:, 0]
        logits[r][rows[0]] = math.nan
        logits[r][rows[1]] = math.inf
        logits[r][rows[2]] = torch.finfo(ty).min
    logits[2][7] = -math.inf          # no expert open: does not count
    logits[2][8, 3:] = -math.inf      # three experts open
    logits[2][9] = torch.finfo(ty).min
    want = check(logits, masks, 4, dtype)
    assert (want["chosen"][2, 7] == -1).all()


def test_nothing_counts():
    logits = draw(2, 12, 16, torch.float32, 6)
    masks = [torch.zeros(12, device="cuda", dtype=torch.uint8) for _ in range(2)]
    loss, counts, picks, out = call(logits, masks, 2, vr.VR_FLOAT32)
    assert float(loss) == 0.0 and not counts.any()
    assert all(bool((p == -1).all()) for p in picks) and not any(bool(o.any()) for o in out)


def test_no_tokens():
    logits = [torch.empty(0, 16, device="cuda")]
    loss, counts, _, _ = call(logits, None, 2, vr.VR_FLOAT32)
    assert float(loss) == 0.0 and not counts.any()


def test_a_nan_that_counts_shows():
    logits = draw(1, 12, 16, torch.float32, 7)
    logits[0][3, 5] = math.nan
    loss, counts, picks, out = call(logits, None, 2, vr.VR_FLOAT32)
    assert math.isnan(float(loss)) and int(picks[0][3, 0]) == 5
    assert int(counts.sum()) == 24


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
def test_ties_go_to_the_lowest_expert(dtype):
    code, ty = DT[dtype]
    logits = draw(2, 64, 130, ty, 8)
    logits = [torch.round(x) for x in logits]   # many equal logits, 0 and -0 among them
    check(logits, None, 8, dtype, scale=64.0)


@pytest.mark.parametrize("offset,stride", [(0, 40), (1, 41), (3, 32), (8, 48)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_strides_and_alignment(offset, stride, dtype):
    """Rows inside a wider buffer: what lies between them is not touched."""
    code, ty = DT[dtype]
    T, E = 21, 32
    base = draw(1, 1, T * stride + offset, ty, 9)[0][0]
    x = base[offset:].as_strided((T, E), (stride, 1), offset)
    outBase = torch.full_like(base, 7.0)
    out = outBase.as_strided((T, E), (stride, 1), offset)
    check([x], None, 2, dtype, stride=stride, out=[out])
    left = torch.ones_like(base, dtype=torch.bool)
    left.as_strided((T, E), (stride, 1), offset)[:] = False
    assert bool((outBase[left] == 7.0).all())


def test_ranks_side_by_side_in_one_matrix():
    """Column slices of one matrix as the ranks' logits, gradients in place."""
    wide = draw(1, 30, 64, torch.float32, 10)[0]
    logits = [wide[:, :32], wide[:, 32:]]
    keep = [x.clone() for x in logits]
    want = refs.balance([x.cpu() for x in keep], None, 2, 0.01, 1.0)
    call(logits, None, 2, vr.VR_FLOAT32, stride=64, out=logits)
    for r in range(2):
        refs.assert_close(logits[r].cpu(), want["grads"][r], want["bound"][r], torch.float32)


def test_optional_outputs_and_other_stream():
    logits = draw(2, 500, 64, torch.float32, 11)
    full = call(logits, None, 4, vr.VR_FLOAT32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        part = call(logits, None, 4, vr.VR_FLOAT32, grads=False, chosen=False, stream=side)
    side.synchronize()
    assert torch.equal(full[0], part[0]) and torch.equal(full[1], part[1])


def test_the_same_bits_twice():
    logits = draw(8, 2000, 256, torch.bfloat16, 12)
    a, b = (call(logits, None, 8, vr.VR_BFLOAT16) for _ in range(2))
    assert torch.equal(a[0], b[0]) and all(torch.equal(x, y) for x, y in zip(a[3], b[3]))


def test_gradient_against_differences():
    """Central differences of the loss in 64 bits with the counts held."""
    logits = draw(1, 6, 10, torch.float32, 13)
    loss, counts, _, out = call(logits, None, 2, vr.VR_FLOAT32, coef=1.0)
    f = counts.cpu().double() / 12
    x = logits[0].cpu().double()

    def value(z):
        return 10 * float((f * torch.softmax(z, 1).mean(0)).sum())

    h = 1e-4
    for t, e in [(0, 0), (2, 9), (5, 4)]:
        z = x.clone()
        z[t, e] += h
        up = value(z)
        z[t, e] -= 2 * h
        num = (up - value(z)) / (2 * h)
        # truncation h^2 |f'''| / 6 <= 1e-8, cancellation 1e-15 / h = 1e-11,
        # fp32 evaluation 1e-6 of values below 1
        assert abs(num - float(out[0][t, e])) <= 2e-6


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
def test_a_row_at_the_lowest_value_is_uniform(dtype):
    """A router that masks with the type's lowest value, all experts of a
    token: equal probabilities, the first topK experts."""
    code, ty = DT[dtype]
    E, T = 32, 6
    logits = draw(1, T, E, ty, 14)
    logits[0][2] = torch.finfo(ty).min
    logits[0][4, 1:] = torch.finfo(ty).min
    scale = float(64 * T) if dtype == "fp16" else 1.0
    loss, counts, picks, out = call(logits, None, 2, code, 1.0, scale)
    f = counts.cpu().double() / (2 * T)
    factor = scale * E / T
    uniform = factor / E * (f - f.mean())
    # exp and the sum of 32 terms in fp32, one rounding to the type
    tol = uniform.abs().max() * (2.0 ** -18 + refs.U_T[ty]) + refs.MIN_T[ty]
    assert float((out[0][2].cpu().double() - uniform).abs().max()) <= float(tol)
    assert picks[0][2].tolist() == [0, 1]
    # the other's only open expert has probability one: no gradient
    assert float(out[0][4].cpu().double().abs().max()) <= factor * 2.0 ** -20
