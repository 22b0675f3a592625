"""The training operators stay within the buffers they are given: workspaces
and outputs lie between guard bytes, and the results are compared as well."""

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import double_binary_tree_gb300 as vr  # noqa: E402
from tests import operator_refs as refs  # noqa: E402
from tests.test_gpu_linear_xent import DT, IGNORE, compare, make  # noqa: E402

GUARD = 1 << 20
FILL = 0xA5


class Arena:
    """One allocation from which guarded buffers are cut."""

    def __init__(self):
        self.kept = []

    def cut(self, nbytes, offset=0):
        """nbytes bytes that begin `offset` bytes after a 256-byte boundary,
        255 at the start (NaN), between guards."""
        base = torch.full((2 * GUARD + nbytes + offset,), FILL, device="cuda", dtype=torch.uint8)
        part = base[GUARD + offset:GUARD + offset + nbytes]
        part.fill_(255)
        assert part.data_ptr() % 256 == offset % 256
        self.kept.append((base, GUARD + offset, GUARD + offset + nbytes))
        return part

    def like(self, shape, dtype, offset=0):
        n = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
        return self.cut(n, offset).view(dtype).view(shape)

    def intact(self):
        return all(bool((b[:lo] == FILL).all()) and bool((b[hi:] == FILL).all())
                   for b, lo, hi in self.kept)


def xent(arena, h, w, y, code, scale, grads, offset=0):
    (T, D), V = h.shape, w.shape[0]
    n = vr.vr_linear_xent_workspace_bytes(h, D, w, D, T, D, V, code, grads)
    work = arena.cut(n, offset)
    losses, lse = (arena.like((T,), torch.float32) for _ in range(2))
    loss = arena.like((1,), torch.float32)
    dh, dw = arena.like((T, D), h.dtype), arena.like((V, D), h.dtype)
    vr.vr_linear_xent(h, D, w, D, y, T, D, V, code, IGNORE, True, scale, losses, lse, loss, dh, dw,
                      work, n, torch.cuda.current_stream())
    return losses, lse, loss, dh, dw


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,D,V", [(300, 64, 380000), (2600, 128, 60000), (4100, 64, 40000)])
def test_pieces_of_the_vocabulary_with_ragged_tokens(T, D, V, dtype):
    """More tokens than dim and over 256 MB of numerators: the vocabulary in
    pieces.  The last tile of 256 tokens holds 44, 40 and 4 of them: its other
    rows are no part of the call."""
    code, ty = DT[dtype]
    scale = 64.0 * T if dtype == "fp16" else 1.0
    h, w, y = make(T, D, V, ty, T)
    arena = Arena()
    got = xent(arena, h, w, y, code, scale, 1)
    assert vr.vr_stream_status() == 0
    assert arena.intact()
    compare(got, refs.xent(h, w, y, IGNORE, True, scale), ty)


# A workspace needs 16-byte alignment, whatever the width of the accesses that
# the kernels make into it: the same bits from every such place.
OFFSETS = [16, 32, 112, 240]


@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,D,V,least", [
    (70, 64, 300, False), (300, 136, 1000, False), (130, 65, 1000, False),  # padded weight
    (300, 64, 380000, False),                                                # in pieces
    (600, 640, 240000, True)])                                               # by the workspace
def test_xent_workspace_alignment(T, D, V, least, dtype, offset):
    code, ty = DT[dtype]
    scale = 64.0 * T if dtype == "fp16" else 1.0
    h, w, y = make(T, D, V, ty, 5, ignored=0.1)
    want = xent(Arena(), h, w, y, code, scale, 2 if least else 1)
    arena = Arena()
    got = xent(arena, h, w, y, code, scale, 2 if least else 1, offset)
    assert vr.vr_stream_status() == 0
    assert arena.intact()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def ortho(arena, ms, code, offset=0):
    rows, cols = ms[0].shape
    n = vr.vr_orthogonalize_workspace_bytes(len(ms), rows, cols, code)
    work = arena.cut(n, offset)
    out = [arena.like((rows, cols), ms[0].dtype) for _ in ms]
    vr.vr_orthogonalize(ms, out, len(ms), rows, cols, code, 5, None, 1e-7, 1.0, work, n,
                        torch.cuda.current_stream())
    return out


@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("count,rows,cols", [(2, 100, 60), (3, 200, 333), (1, 333, 200),
                                             (1, 1500, 1030)])
def test_orthogonalize_workspace_alignment(count, rows, cols, dtype, offset):
    code, ty = dict(DT, fp32=(vr.VR_FLOAT32, torch.float32))[dtype]
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    ms = [torch.randn(rows, cols, generator=g, device="cuda").to(ty) for _ in range(count)]
    want = ortho(Arena(), ms, code)
    arena = Arena()
    got = ortho(arena, ms, code, offset)
    assert vr.vr_stream_status() == 0
    assert arena.intact()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("R,T,E", [(2, 7, 30), (4, 500, 64), (2, 3000, 257)])
def test_balance_workspace_alignment(R, T, E, offset):
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    logits = [torch.randn(T, E, generator=g, device="cuda") for _ in range(R)]

    def run(arena, at):
        n = vr.vr_balance_loss_workspace_bytes(R, T, E)
        work = arena.cut(n, at)
        loss, counts = arena.like((1,), torch.float32), arena.like((E,), torch.int32)
        picks = [arena.like((T, 3), torch.int32) for _ in range(R)]
        out = [arena.like((T, E), torch.float32) for _ in range(R)]
        vr.vr_balance_loss(logits, E, None, R, T, E, 3, vr.VR_FLOAT32, 0.01, 1.0, loss, counts,
                           picks, out, work, n, torch.cuda.current_stream())
        return [loss, counts] + picks + out

    want = run(Arena(), 0)
    arena = Arena()
    got = run(arena, offset)
    assert vr.vr_stream_status() == 0
    assert arena.intact()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
