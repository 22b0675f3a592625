"""Refusals of the training operators: argument errors are reported on the
host, before anything is enqueued.  The pointers are never dereferenced."""

import pytest

import double_binary_tree_gb300 as vr

INV, UNS = vr.VR_ERR_INVALID_ARGUMENT, vr.VR_ERR_UNSUPPORTED
A = 0x10000000   # distinct buffers, far apart
STEP = 0x1000000


def code(fn, *args):
    before = vr.vr_launch_count()
    with pytest.raises(vr.VrError) as ei:
        fn(*args)
    assert vr.vr_launch_count() == before
    return ei.value.code


def balance_args(**kw):
    a = dict(logits=[A, A + STEP], rowStride=16, masks=None, R=2, tokens=10, experts=16, topK=2,
             dtype=vr.VR_FLOAT32, coef=1.0, gradScale=1.0, loss=A + 2 * STEP, counts=A + 3 * STEP,
             chosen=[A + 4 * STEP, A + 5 * STEP], dlogits=[A + 6 * STEP, A + 7 * STEP],
             workspace=A + 8 * STEP, workspaceBytes=4 << 20)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad", [
    dict(R=0), dict(R=65), dict(experts=0), dict(experts=1025, rowStride=1025), dict(topK=0),
    dict(topK=17), dict(experts=64, rowStride=64, topK=33), dict(rowStride=15), dict(dtype=3),
    dict(tokens=1 << 31), dict(tokens=1 << 62), dict(rowStride=1 << 62), dict(logits=None),
    dict(logits=[A, 0]), dict(dlogits=[0, A]), dict(loss=0), dict(counts=0), dict(workspace=0),
    dict(workspaceBytes=16), dict(workspace=A + 8 * STEP + 4), dict(loss=A + 2 * STEP + 2),
    dict(logits=[A + 2, A + STEP]), dict(chosen=[A + 4 * STEP + 2, 0]),
    dict(dlogits=[A + 6 * STEP, A + 6 * STEP + 64]),       # two ranks' gradients overlap
    dict(dlogits=[A + STEP, A + 7 * STEP]),                # over another rank's logits
    dict(dlogits=[A + 16, A + 7 * STEP]),                  # partly over its own
    dict(loss=A + 8 * STEP), dict(counts=A + 64),
])
def test_balance_refusals(bad):
    assert code(vr.vr_balance_loss, *balance_args(**bad)) == INV


def test_balance_workspace():
    assert code(vr.vr_balance_loss_workspace_bytes, 0, 1, 1) == INV
    assert code(vr.vr_balance_loss_workspace_bytes, 1, 1, 1025) == INV
    small = vr.vr_balance_loss_workspace_bytes(1, 1, 8)
    assert 0 < small <= vr.vr_balance_loss_workspace_bytes(8, 1 << 20, 1024)


def xent_args(**kw):
    a = dict(hidden=A, hiddenStride=64, weight=A + STEP, weightStride=64, targets=A + 2 * STEP,
             tokens=100, dim=64, vocab=500, dtype=vr.VR_BFLOAT16, ignoreIndex=-100, mean=True,
             gradScale=1.0, losses=A + 3 * STEP, lse=A + 4 * STEP, loss=A + 5 * STEP,
             dHidden=A + 6 * STEP, dWeight=A + 7 * STEP, workspace=A + 8 * STEP,
             workspaceBytes=8 << 20)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad", [
    dict(dtype=vr.VR_FLOAT32), dict(dtype=9), dict(dim=0), dict(vocab=0), dict(tokens=1 << 31),
    dict(tokens=1 << 62), dict(vocab=1 << 31), dict(dim=1 << 25, hiddenStride=1 << 25,
                                                    weightStride=1 << 25),
    dict(hiddenStride=63), dict(weightStride=63), dict(hiddenStride=1 << 40), dict(hidden=0),
    dict(weight=0), dict(targets=0), dict(losses=0), dict(lse=0), dict(loss=0), dict(workspace=0),
    dict(workspaceBytes=1 << 16), dict(workspace=A + 8 * STEP + 8), dict(targets=A + 2 * STEP + 4),
    dict(losses=A + 3 * STEP + 2), dict(hidden=A + 1), dict(dWeight=A + 7 * STEP + 1),
    dict(dHidden=A), dict(dWeight=A + STEP), dict(lse=A + 3 * STEP + 4), dict(loss=A + 2 * STEP),
    dict(workspace=A + 7 * STEP + 256),
])
def test_linear_xent_refusals(bad):
    assert code(vr.vr_linear_xent, *xent_args(**bad)) == INV


def test_linear_xent_workspace():
    size = vr.vr_linear_xent_workspace_bytes
    B = vr.VR_BFLOAT16
    assert code(size, A, 64, A, 64, 10, 64, 0, B, 1) == INV
    loss, grads = (size(A, 64, A, 64, 1000, 64, 5000, B, g) for g in (0, 1))
    assert 0 < loss < grads
    # rows that are no 16-byte units need a copy
    assert size(A, 65, A, 64, 1000, 64, 5000, B, 0) > loss
    assert size(A + 2, 64, A, 64, 1000, 64, 5000, B, 0) > loss
    assert code(size, A, 64, A, 64, 10, 64, 100, B, 3) == INV
    # many tokens, or the least workspace: the gradient factors are taken in
    # pieces, tokens x vocab of them are not held
    assert size(A, 64, A, 64, 1 << 16, 64, 1 << 17, B, 1) < (1 << 33)
    kept, least = (size(A, 4096, A, 4096, 4096, 4096, 1 << 17, B, g) for g in (1, 2))
    assert kept > 2 << 29 and least < 1 << 29


def ortho_args(**kw):
    a = dict(src=[A, A + STEP], dst=[A + 2 * STEP, A + 3 * STEP], count=2, rows=40, cols=60,
             dtype=vr.VR_BFLOAT16, steps=2, coefs=None, eps=1e-7, scale=1.0,
             workspace=A + 4 * STEP, workspaceBytes=4 << 20)
    a.update(kw)
    return list(a.values())


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("bad", [
    dict(count=0), dict(rows=0), dict(cols=0), dict(rows=1 << 25), dict(cols=1 << 62),
    dict(dtype=5), dict(steps=0), dict(steps=33), dict(eps=-1.0), dict(eps=NAN), dict(scale=INF),
    dict(coefs=[1.5, NAN, 0.0] * 2), dict(coefs=[1.0] * 5), dict(src=None), dict(dst=None),
    dict(src=[A, 0]), dict(dst=[0, A]), dict(src=[A + 1, A + STEP]), dict(workspace=0),
    dict(workspace=A + 4 * STEP + 8), dict(workspaceBytes=1000),
    dict(dst=[A + 2 * STEP, A + 2 * STEP + 64]), dict(dst=[A + STEP, A + 3 * STEP]),
    dict(dst=[A + 16, A + 3 * STEP]), dict(workspace=A + 1024),
])
def test_orthogonalize_refusals(bad):
    assert code(vr.vr_orthogonalize, *ortho_args(**bad)) == INV


def test_orthogonalize_refuses_coefficients_that_leave_the_range():
    assert code(vr.vr_orthogonalize, *ortho_args(coefs=[20.0, 0.0, 0.0] * 2)) == UNS
    assert code(vr.vr_orthogonalize, *ortho_args(steps=3, coefs=[3.0, 0.0, 0.0] * 3)) == UNS
    assert code(vr.vr_orthogonalize, *ortho_args(coefs=[1.0, -16.0, 0.0] * 2)) == UNS


def test_orthogonalize_workspace():
    size = vr.vr_orthogonalize_workspace_bytes
    assert code(size, 0, 8, 8, vr.VR_FLOAT32) == INV
    assert size(1, 64, 32, vr.VR_FLOAT32) == size(1, 32, 64, vr.VR_FLOAT32)
    # launches take at most 64 matrices, one after the other
    assert size(200, 64, 64, vr.VR_BFLOAT16) == size(64, 64, 64, vr.VR_BFLOAT16)
