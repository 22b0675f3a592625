"""Refusals of embedding, AdamW and grouped products: reported on the host,
before anything is enqueued.  The pointers are never dereferenced."""

import math
import random

import pytest

import double_binary_tree_gb300 as vr
from tests.test_operators_host import A, INV, STEP, code

BIG = 1 << 62


def lookup_args(**kw):
    a = dict(weight=A, weightStride=64, ids=A + STEP, tokens=100, dim=64, vocab=500,
             dtype=vr.VR_BFLOAT16, ignoreIndex=-100, scale=1.0, out=A + 2 * STEP, outStride=64)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(dim=0), dict(vocab=0), dict(tokens=1 << 31), dict(tokens=BIG),
    dict(vocab=1 << 31), dict(vocab=BIG), dict(dim=1 << 25, weightStride=1 << 25, outStride=1 << 25),
    dict(weightStride=63), dict(outStride=63), dict(weightStride=1 << 40), dict(outStride=BIG),
    dict(weight=0), dict(ids=0), dict(out=0), dict(weight=A + 1), dict(out=A + 2 * STEP + 1),
    dict(ids=A + STEP + 4), dict(out=A), dict(out=A + STEP), dict(out=A + 64 * 500),
    dict(tokens=1, dim=4, out=A + STEP),  # a row of eight bytes over the one id
])
def test_embedding_refusals(bad):
    assert code(vr.vr_embedding, *lookup_args(**bad)) == INV


def embedding_grad_args(**kw):
    a = dict(dOut=A, dOutStride=64, ids=A + STEP, tokens=100, dim=64, vocab=500,
             dtype=vr.VR_BFLOAT16, ignoreIndex=-100, scale=1.0, accumulate=0,
             dWeight=A + 2 * STEP, workspace=A + 3 * STEP, workspaceBytes=1 << 20)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad", [
    dict(dtype=-1), dict(dim=0), dict(vocab=0), dict(tokens=1 << 31), dict(vocab=1 << 31),
    dict(dim=1 << 25, dOutStride=1 << 25), dict(dOutStride=63), dict(dOutStride=1 << 32),
    dict(dOut=0), dict(ids=0), dict(dWeight=0), dict(workspace=0), dict(workspaceBytes=1000),
    dict(workspace=A + 3 * STEP + 8), dict(dOut=A + 1), dict(dWeight=A + 2 * STEP + 1),
    dict(ids=A + STEP + 2), dict(dWeight=A), dict(dWeight=A + STEP), dict(workspace=A),
    dict(workspace=A + 2 * STEP + 16), dict(workspace=A + STEP),
])
def test_embedding_grad_refusals(bad):
    assert code(vr.vr_embedding_grad, *embedding_grad_args(**bad)) == INV


def test_embedding_grad_workspace():
    size = vr.vr_embedding_grad_workspace_bytes
    B = vr.VR_BFLOAT16
    assert code(size, 10, 0, 100, B) == INV
    assert code(size, 10, 10, 100, 7) == INV
    assert 0 < size(0, 1, 1, B) <= size(100, 64, 100, B) < size(100000, 64, 100, B)
    # it does not grow with the vocabulary
    assert size(100, 64, 100, B) == size(100, 64, 1 << 30, B)


def linear_args(**kw):
    a = dict(x=A, xStride=64, weight=A + STEP, counts=A + 2 * STEP, rows=100, dim=64, outDim=72,
             groups=4, dtype=vr.VR_BFLOAT16, out=A + 3 * STEP, outStride=72,
             workspace=A + 4 * STEP, workspaceBytes=1 << 20)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad", [
    dict(dtype=vr.VR_FLOAT32), dict(dtype=8), dict(dim=0), dict(outDim=0), dict(groups=0),
    dict(groups=1025), dict(rows=1 << 31), dict(rows=BIG), dict(dim=1 << 25, xStride=1 << 25),
    dict(outDim=1 << 25, outStride=1 << 25), dict(xStride=63), dict(outStride=71),
    dict(xStride=1 << 32), dict(outStride=BIG), dict(x=0), dict(weight=0), dict(counts=0),
    dict(out=0), dict(workspace=0), dict(workspace=A + 4 * STEP + 8), dict(workspaceBytes=0),
    dict(x=A + 1), dict(weight=A + STEP + 1), dict(out=A + 3 * STEP + 1),
    dict(counts=A + 2 * STEP + 2), dict(out=A), dict(out=A + STEP), dict(out=A + 2 * STEP),
    dict(out=A + 4 * STEP), dict(workspace=A), dict(workspace=A + STEP),
    dict(rows=1, outDim=8, groups=4, out=A + 2 * STEP),  # a row of 16 bytes over the counts
    # rows that are no 16-byte units need a copy: more than is there
    dict(x=A + 2, rows=10000), dict(xStride=65, rows=10000),
])
def test_grouped_linear_refusals(bad):
    assert code(vr.vr_grouped_linear, *linear_args(**bad)) == INV


def linear_grad_args(**kw):
    a = dict(dOut=A, dOutStride=72, x=A + STEP, xStride=64, weight=A + 2 * STEP,
             counts=A + 3 * STEP, rows=100, dim=64, outDim=72, groups=4, dtype=vr.VR_FLOAT16,
             dX=A + 4 * STEP, dWeight=A + 5 * STEP, workspace=A + 6 * STEP, workspaceBytes=1 << 20)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad", [
    dict(dtype=vr.VR_FLOAT32), dict(dim=0), dict(outDim=0), dict(groups=0), dict(groups=1025),
    dict(rows=1 << 31), dict(dOutStride=71), dict(xStride=63), dict(dOutStride=1 << 33),
    dict(dOut=0), dict(x=0), dict(weight=0), dict(counts=0), dict(dX=0, dWeight=0),
    dict(workspace=0), dict(workspace=A + 6 * STEP + 4), dict(workspaceBytes=100),
    dict(dOut=A + 1), dict(x=A + STEP + 1), dict(weight=A + 2 * STEP + 1), dict(counts=A + 3),
    dict(dX=A + 4 * STEP + 1), dict(dWeight=A + 5 * STEP + 1), dict(dX=A), dict(dX=A + STEP),
    dict(dWeight=A + 2 * STEP), dict(dWeight=A + 4 * STEP), dict(dX=A + 3 * STEP),
    dict(workspace=A + 5 * STEP + 16),
])
def test_grouped_linear_grad_refusals(bad):
    assert code(vr.vr_grouped_linear_grad, *linear_grad_args(**bad)) == INV


def test_grouped_workspaces():
    size, grad = vr.vr_grouped_linear_workspace_bytes, vr.vr_grouped_linear_grad_workspace_bytes
    B = vr.VR_BFLOAT16
    assert code(size, A, 64, A, 10, 64, 64, 0, B) == INV
    assert code(grad, A, 64, A, 63, A, 10, 64, 64, 1, B) == INV
    least = size(A, 64, A, 1000, 64, 72, 8, B)
    assert 0 < least <= 1024
    x_copy = size(A, 65, A, 1000, 64, 72, 8, B)
    assert x_copy - least >= 1000 * 64 * 2
    assert size(A, 64, A + 2, 1000, 64, 72, 8, B) - least >= 8 * 72 * 64 * 2
    assert size(A, 65, A, 1000, 65, 72, 8, B) > x_copy
    assert grad(A, 72, A, 64, A, 1000, 64, 72, 8, B) == least
    assert grad(A, 73, A, 64, A, 1000, 64, 73, 8, B) - least >= 1000 * 73 * 2


def adamw_args(**kw):
    at = iter(range(100))

    def two():
        return [A + next(at) * STEP for _ in range(2)]

    a = dict(params=two(), grads=two(), m=two(), v=two(), mScales=two(), vScales=two(),
             masters=two(), sizes=[1000, 300], count=2, dtype=vr.VR_BFLOAT16,
             gradDtype=vr.VR_BFLOAT16, stateBits=8, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8,
             weightDecay=0.1, step=1, gradScale=1.0, seed=1, control=None)
    for k, v in kw.items():
        if callable(v):
            v = v(a)
        a[k] = v
    return list(a.values())


@pytest.mark.parametrize("bad", [
    dict(count=0), dict(count=-1), dict(dtype=3), dict(gradDtype=-1), dict(stateBits=16),
    dict(dtype=vr.VR_FLOAT32), dict(mScales=None), dict(vScales=None), dict(stateBits=32),
    dict(params=None), dict(grads=None), dict(m=None), dict(v=None),
    dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=math.nan), dict(eps=-1.0),
    dict(eps=math.inf), dict(eps=1e-40), dict(lr=math.nan), dict(gradScale=math.inf), dict(weightDecay=math.inf),
    dict(step=0), dict(step=-5), dict(sizes=[1000, 1 << 41]), dict(control=A + 50 * STEP + 2),
    dict(params=[A, 0]), dict(grads=[0, A + STEP]), dict(masters=[A + 12 * STEP, 0]),
    dict(mScales=[A + 8 * STEP, 0]), dict(params=[A + 1, A + STEP]),
    dict(grads=[A + 2 * STEP, A + 3 * STEP + 1]), dict(masters=[A + 12 * STEP + 2, A + 13 * STEP]),
    dict(vScales=[A + 10 * STEP + 1, A + 11 * STEP]),
    dict(grads=lambda a: a["params"]), dict(v=lambda a: a["m"]),
    dict(params=[A, A + 1998]), dict(control=A),
    dict(m=lambda a: [a["m"][0], a["m"][0] + 999]),
])
def test_adamw_refusals(bad):
    assert code(vr.vr_adamw, *adamw_args(**bad)) == INV


def test_adamw_takes_gradients_that_share_memory():
    """Read only: two tensors' gradients may be the same (the refusal here is
    another one, the last that is checked)."""
    same = dict(grads=[A + 40 * STEP] * 2)
    assert code(vr.vr_adamw, *adamw_args(**same, params=[A, A + 2])) == INV


def values_args(**kw):
    two = [[A + (2 * i + j) * STEP for j in range(2)] for i in range(6)]
    a = dict(m=two[0], v=two[1], mScales=two[2], vScales=two[3], sizes=[1000, 300], count=2,
             mValues=two[4], vValues=two[5])
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad", [
    dict(count=0), dict(sizes=[1 << 41, 1]), dict(m=None), dict(vScales=None),
    dict(mValues=None, vValues=None), dict(m=[A, 0]), dict(vValues=[A + 10 * STEP, 0]),
    dict(mValues=[A, A + 9 * STEP]), dict(mValues=[A + 8 * STEP, A + 8 * STEP + 3996]),
    dict(mValues=[A + 8 * STEP + 2, A + 9 * STEP]), dict(vScales=[A + 6 * STEP + 1, A + 7 * STEP]),
])
def test_adamw_values_refusals(bad):
    assert code(vr.vr_adamw_values, *values_args(**bad)) == INV


def test_adamw_overlaps_as_a_plain_statement_says():
    """Random layouts: refused exactly when a written buffer touches another
    one.  (What is not refused goes on to the device: none here.)"""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("the pointers are not real")
    rng = random.Random(4)
    seen = set()
    for _ in range(3000):
        n = rng.randint(1, 4)
        sizes = [rng.randint(1, 900) for _ in range(n)]
        space = rng.choice([20000, 60000, 400000])
        if rng.random() < 0.5:  # slices of a few buffers, as programs have them
            def place(unit):
                at, out = A + rng.randint(0, space) * 256, []
                for k in sizes:
                    out.append(at)
                    at += (k * unit + 255) // 256 * 256 + rng.choice([0, 0, 0, 256])
                return out
        else:
            def place(unit):
                return [A + rng.randint(0, space) * 4 for _ in sizes]
        p, g, m, v = (place(4) for _ in range(4))
        extents = [(a, a + 4 * k, w) for ps, w in ((p, True), (g, False), (m, True), (v, True))
                   for a, k in zip(ps, sizes)]
        bad = any((x[2] or y[2]) and x[0] < y[1] and y[0] < x[1]
                  for i, x in enumerate(extents) for y in extents[:i])
        got = code(vr.vr_adamw, p, g, m, v, None, None, None, sizes, n, vr.VR_FLOAT32,
                   vr.VR_FLOAT32, 32, 1e-3, 0.9, 0.99, 1e-8, 0.1, 1, 1.0, 1, None)
        assert (got == INV) == bad, (extents, got)
        seen.add(bad)
    assert seen == {True, False}
