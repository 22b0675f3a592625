"""vr_orthogonalize against its definition in 64 bits (operator_refs.py)."""

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
EPS = 1e-7


def make(count, rows, cols, ty, seed, rank=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if rank:
        x = (torch.randn(count, rows, rank, generator=g, device="cuda")
             @ torch.randn(count, rank, cols, generator=g, device="cuda"))
    else:
        x = torch.randn(count, rows, cols, generator=g, device="cuda")
    return [m.clone() for m in (x * 0.01).to(ty)]


def call(ms, code, steps=5, coefs=None, eps=EPS, scale=1.0, out=None, stream=None):
    rows, cols = ms[0].shape
    if out is None:
        out = [torch.full_like(m, math.nan) for m in ms]
    n = vr.vr_orthogonalize_workspace_bytes(len(ms), rows, cols, code)
    work = torch.full((n,), 255, device="cuda", dtype=torch.uint8)   # NaN at the start
    vr.vr_orthogonalize(ms, out, len(ms), rows, cols, code, steps, coefs, eps, scale, work, n,
                        stream or torch.cuda.current_stream())
    return out


def compare(got, ms, ty, steps=5, coefs=None, eps=EPS, scale=1.0):
    gain = 1.0
    for k in range(steps):
        gain *= abs(coefs[3 * k] if coefs is not None else refs.COEFS[0])
    for g, m in zip(got, ms):
        want = refs.orthogonalize(m, steps, coefs, eps, scale)
        tol = refs.ortho_tolerance(ty, float(want.norm()) / abs(scale), gain)
        assert refs.norm_error(g, want) <= tol
        # elements: errors of a few deviations, next to the larger of the
        # element and the result's rms
        rms = float(want.norm()) / math.sqrt(want.numel())
        assert bool(((g.double() - want).abs() <= 8 * tol * want.abs().clamp(min=rms)).all())


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("count,rows,cols", [
    (1, 1, 1), (2, 1, 37), (1, 64, 1), (3, 8, 8), (2, 32, 64), (1, 65, 33), (8, 128, 128),
    (2, 127, 129), (1, 129, 500), (3, 500, 129), (1, 256, 1000), (1, 777, 333), (2, 384, 640),
    # one launch of a cluster per matrix up to 128 x 2048, and just above
    (2, 100, 257), (1, 256, 128), (3, 90, 513), (1, 1025, 128), (2, 2048, 77), (1, 128, 2048),
    (1, 128, 2049), (1, 2100, 64), (2, 5, 1800), (40, 16, 1030)])
def test_matches_the_definition(count, rows, cols, dtype):
    code, ty = DT[dtype]
    ms = make(count, rows, cols, ty, rows + cols)
    got = call(ms, code)
    assert vr.vr_stream_status() == 0
    compare(got, ms, ty)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_larger_matrices(dtype):
    code, ty = DT[dtype]
    for rows, cols in [(1024, 4100), (2050, 1030)]:
        ms = make(1, rows, cols, ty, rows)
        compare(call(ms, code), ms, ty)


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
def test_few_large_singular_values(dtype):
    """A matrix of rank 4 plus a little noise: most directions are tiny."""
    code, ty = DT[dtype]
    ms = make(1, 200, 300, torch.float32, 1, rank=4)
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    ms = [(m + 1e-4 * torch.randn(200, 300, generator=g, device="cuda")).to(ty) for m in ms]
    compare(call(ms, code), ms, ty)


def test_more_matrices_than_one_launch_takes():
    ms = make(70, 24, 40, torch.float32, 2)
    compare(call(ms, vr.VR_FLOAT32), ms, torch.float32)


@pytest.mark.parametrize("steps", [1, 2, 12])
def test_other_coefficients(steps):
    """The cubic (1.5, -0.5, 0): converges to an orthogonal factor."""
    coefs = [1.5, -0.5, 0.0] * steps
    ms = make(1, 16, 400, torch.float32, 3)
    got = call(ms, vr.VR_FLOAT32, steps=steps, coefs=coefs, scale=2.0)
    compare(got, ms, torch.float32, steps, coefs, scale=2.0)
    if steps == 12:
        x = got[0].double() / 2
        assert float((x @ x.t() - torch.eye(16, device="cuda")).abs().max()) <= 1e-4


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_in_place_and_unaligned(dtype):
    code, ty = DT[dtype]
    base = torch.randn(2 * 50 * 61 + 8, device="cuda").to(ty)
    ms = [base[1:1 + 50 * 61].view(50, 61), base[3 + 50 * 61:3 + 2 * 50 * 61].view(50, 61)]
    keep = [m.clone() for m in ms]
    compare(call(ms, code, out=ms), keep, ty)


def test_a_zero_matrix_and_a_bad_one_stay_by_themselves():
    ms = make(4, 40, 70, torch.float32, 4)
    ms[1].zero_()
    ms[2][3, 5] = math.nan
    ms[3][0, 0] = math.inf
    got = call(ms, vr.VR_FLOAT32)
    compare(got[:1], ms[:1], torch.float32)
    assert not got[1].any()
    assert bool(got[2].isnan().all()) and bool(got[3].isnan().all())


def test_scales_of_the_input_do_not_matter():
    m = make(1, 60, 90, torch.float32, 5)[0]
    for by in (1e-12, 1e12):
        compare(call([m * by], vr.VR_FLOAT32, eps=0.0), [m * by], torch.float32, eps=0.0)


def test_another_stream_a_graph_and_the_same_bits():
    ms = make(3, 200, 260, torch.bfloat16, 6)
    a = call(ms, vr.VR_BFLOAT16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = call(ms, vr.VR_BFLOAT16, stream=side)
    side.synchronize()
    out = [torch.zeros_like(m) for m in ms]
    n = vr.vr_orthogonalize_workspace_bytes(3, 200, 260, vr.VR_BFLOAT16)
    work = torch.empty(n, device="cuda", dtype=torch.uint8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vr.vr_orthogonalize(ms, out, 3, 200, 260, vr.VR_BFLOAT16, 5, None, EPS, 1.0, work, n,
                            torch.cuda.current_stream())
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(a, b, out):
        assert torch.equal(x, y) and torch.equal(x, z)
