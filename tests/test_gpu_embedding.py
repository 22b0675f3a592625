"""vr_embedding and vr_embedding_grad against their definitions in 64 bits
(more_refs.py)."""

import math

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
IGNORE = -100


def rand(shape, ty, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(ty)


def words(T, V, seed, ignored=0.0):
    """Words by frequency, some ignored."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    u = torch.rand(T, generator=g, device="cuda")
    ids = (torch.exp(u * math.log(V + 1)) - 1).long().clamp(0, V - 1)
    ids[torch.rand(T, generator=g, device="cuda") < ignored] = IGNORE
    return ids


def lookup(w, ids, code, scale, arena=None, stride=None, offset=0, stream=None):
    V, D = w.shape
    T = len(ids)
    arena = arena or Arena()
    stride = stride or D
    out = arena.like((max(T, 1) * stride,), w.dtype, offset)
    vr.vr_embedding(w, max(w.stride(0), D), ids, T, D, V, code, IGNORE, scale, out, stride,
                    stream or torch.cuda.current_stream())
    assert vr.vr_stream_status(stream) in (0, vr.VR_ERR_INVALID_ARGUMENT)
    assert arena.intact()
    return out.view(-1, stride)[:T]


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,D,V", [
    (1, 1, 1), (1, 1024, 500), (7, 33, 50), (300, 136, 1000), (64, 4099, 77), (5000, 64, 20000),
    (3, 4102, 9), (2, 20000, 3)])
def test_lookup(T, D, V, dtype):
    code, ty = DT[dtype]
    w, ids = rand((V, D), ty, T + D), words(T, V, D, 0.2)
    got = lookup(w, ids, code, 0.37)
    want, bound = more_refs.embedding(w, ids, float(torch.tensor(0.37)))
    refs.assert_close(got, want, bound, ty)


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,D,V", [
    (1, 1, 1), (1, 1000, 5000), (40, 33, 7), (777, 136, 1000), (300, 1030, 2000), (31, 64, 600),
    (64, 4099, 40), (8192, 24, 5000), (8193, 24, 5000), (30011, 72, 70001)])
@pytest.mark.parametrize("add", [False, True])
def test_gradient(T, D, V, dtype, add):
    code, ty = DT[dtype]
    check_grad(rand((T, D), ty, T + D), words(T, V, D, 0.1), V, dtype, 0.5, add)


def grad(dout, ids, V, code, scale, old, arena=None, offset=0, stream=None, stride=None):
    T, D = dout.shape
    arena = arena or Arena()
    n = vr.vr_embedding_grad_workspace_bytes(T, D, V, code)
    work, dw = arena.cut(n, offset), arena.like((V, D), dout.dtype)
    if old is not None:
        dw.copy_(old)
    vr.vr_embedding_grad(dout, stride or max(dout.stride(0), D), ids, T, D, V, code, IGNORE, scale,
                         old is not None, dw, work, n, stream or torch.cuda.current_stream())
    return dw


def check_grad(dout, ids, V, dtype, scale, add, status=0, **kw):
    code, ty = DT[dtype]
    D = dout.shape[1]
    old = rand((V, D), ty, 9) if add else None
    arena = Arena()
    got = grad(dout, ids, V, code, scale, old, arena, **kw)
    assert vr.vr_stream_status() == status
    assert arena.intact()
    want, bound = more_refs.embedding_grad(dout, ids, V, scale, old)
    refs.assert_close(got, want, bound, ty)
    if add:  # words that do not occur: bit for bit what was there
        there = torch.zeros(V, dtype=torch.bool, device="cuda")
        there[ids[(ids >= 0) & (ids < V)]] = True
        assert torch.equal(got[~there], old[~there])
    # the same bits again, from workspaces at other places
    for offset in (16, 240):
        assert torch.equal(got, grad(dout, ids, V, code, scale, old, offset=offset))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [31, 32, 33, 64, 65, 1000, 8192, 20000])
def test_gradient_of_one_word(T, dtype):
    """Every token the same: one sum over all chunks.  And two words that meet
    in the middle of a chunk, and at its end."""
    ty = DT[dtype][1]
    dout = rand((T, 40), ty, T)
    same = torch.full((T,), 5, device="cuda")
    check_grad(dout, same, 7, dtype, 1.0, False)
    for at in (1, T // 2, T - 1, min(32, T - 1)):
        two = same.clone()
        two[at:] = 6
        check_grad(dout, two.flip(0), 7, dtype, 1.0, True)


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,D", [(1, 600), (33, 520), (1023, 41), (1024, 1032), (1025, 1032),
                                 (1024, 262), (900, 3), (3001, 40), (1024, 4096), (1024, 4100),
                                 (20, 1), (8200, 33)])
@pytest.mark.parametrize("add", [False, True])
def test_gradient_of_frequent_words(T, D, dtype, add):
    """Words of 32 and 33 tokens, of a third of all and of one, a table of a few
    thousand rows, for each way of summing."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T + D)
    ids = torch.randint(0, 9000, (T,), generator=g, device="cuda")
    ids[:T // 3], ids[T // 3:][:32], ids[T // 3 + 32:][:33] = 77, 8999, 0
    ids = ids[torch.randperm(T, generator=g, device="cuda")]
    ids[T - 1:] = IGNORE if T % 2 else 8999
    check_grad(rand((T, D), DT[dtype][1], T), ids, 9000, dtype, 0.7, add)


def test_more_units_than_the_grid_has_warps():
    """Few tokens of many columns: several rounds, frequent words in each."""
    ids = torch.arange(700, device="cuda") % 11
    check_grad(rand((700, 4000), torch.bfloat16, 1), ids, 12, "bf16", 1.0, False)
    check_grad(rand((900, 4001), torch.bfloat16, 2), torch.arange(900, device="cuda") % 23, 23,
               "bf16", 1.0, True)


@pytest.mark.parametrize("T,D,V", [(16384, 512, 200000), (16384, 40, 300), (12000, 33, 70000),
                                   (6000, 1024, 90000)])
@pytest.mark.parametrize("add", [False, True])
def test_gradient_by_either_sort(T, D, V, add):
    """Thousands of tokens, of a table that takes longer to zero than they take
    one CTA to sort, and of others."""
    ids = words(T, V, T + D, 0.05)
    ids[::20] = 3
    check_grad(rand((T, D), torch.float32, T), ids, V, "fp32", 1.0, add)


def test_words_of_many_bits():
    V = (1 << 20) + 3  # three passes
    ids = torch.randint(0, V, (9001,), device="cuda")
    ids[:9] = torch.tensor([V - 1, 0, V - 1, V, 1 << 40, -5, 511, 512, V - 2], device="cuda")
    check_grad(rand((9001, 2), torch.float32, 3), ids, V, "fp32", 1.0, False,
               status=vr.VR_ERR_INVALID_ARGUMENT)
    check_grad(rand((50, 2), torch.float32, 3), ids[:50], V, "fp32", 1.0, True,
               status=vr.VR_ERR_INVALID_ARGUMENT)


def test_words_outside_the_table_are_reported():
    w = rand((10, 16), torch.float32, 1)
    ids = torch.tensor([3, 10, -1, IGNORE, 9], device="cuda")
    out = torch.full((5, 16), math.nan, device="cuda")
    vr.vr_embedding(w, 16, ids, 5, 16, 10, vr.VR_FLOAT32, IGNORE, 1.0, out, 16,
                    torch.cuda.current_stream())
    assert vr.vr_stream_status() == vr.VR_ERR_INVALID_ARGUMENT
    assert torch.equal(out[[0, 4]], w[[3, 9]]) and not out[1:4].any()
    ids[1:3] = IGNORE
    vr.vr_embedding(w, 16, ids, 5, 16, 10, vr.VR_FLOAT32, IGNORE, 1.0, out, 16,
                    torch.cuda.current_stream())
    assert vr.vr_stream_status() == 0


def test_an_ignored_index_inside_the_table():
    """ignoreIndex may be a word (padding): its row is neither read nor
    counted."""
    w = rand((10, 16), torch.float32, 1)
    w[4] = math.nan
    ids = torch.tensor([4, 3, 4], device="cuda")
    out = torch.empty(3, 16, device="cuda")
    vr.vr_embedding(w, 16, ids, 3, 16, 10, vr.VR_FLOAT32, 4, 2.0, out, 16,
                    torch.cuda.current_stream())
    assert not out[[0, 2]].any() and torch.equal(out[1], 2 * w[3])


@pytest.mark.parametrize("ignored", [0.0, 0.5, 1.0])
def test_ignored_rows_may_hold_anything(ignored):
    ids = words(300, 50, 2, ignored)
    dout = rand((300, 24), torch.bfloat16, 4)
    dout[ids < 0] = math.nan
    check_grad(dout, ids, 50, "bf16", 1.0, False)
    check_grad(dout, ids, 50, "bf16", 1.0, True)


def test_a_nan_stays_in_its_row():
    ids = torch.arange(70, device="cuda") % 35
    dout = rand((70, 8), torch.float32, 4)
    dout[40, 3] = math.nan
    got = grad(dout, ids, 40, vr.VR_FLOAT32, 1.0, None)
    assert torch.isnan(got).sum() == 1 and math.isnan(float(got[5, 3]))
    assert not got[35:].any()


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("D,pad,offset", [(64, 8, 0), (64, 2, 0), (64, 1, 0), (64, 0, 2),
                                          (65, 3, 4), (1, 6, 2)])
def test_strides_and_alignment(D, pad, offset, dtype):
    code, ty = DT[dtype]
    size = torch.empty(0, dtype=ty).element_size()
    offset = -(-offset // size) * size
    wide, ids = rand((90, D + pad), ty, 5), words(200, 90, 6, 0.1)
    w = wide[:, :D]
    got = lookup(w, ids, code, 1.0, stride=D + pad, offset=offset)
    want, bound = more_refs.embedding(w, ids, 1.0)
    refs.assert_close(got[:, :D], want, bound, ty)
    raw = got[:, D:].contiguous().view(torch.uint8)
    assert bool((raw == 255).all())  # between the rows: as it was
    dwide = rand((200, D + pad), ty, 7)
    check_grad(dwide[:, :D], ids, 90, dtype, 1.0, True, stride=D + pad)


def test_no_tokens():
    w, none = rand((10, 16), torch.float32, 1), torch.empty(0, dtype=torch.long, device="cuda")
    vr.vr_embedding(w, 16, none, 0, 16, 10, vr.VR_FLOAT32, IGNORE, 1.0, None, 16,
                    torch.cuda.current_stream())
    for add in (False, True):
        old = w.clone()
        n = vr.vr_embedding_grad_workspace_bytes(0, 16, 10, vr.VR_FLOAT32)
        work = torch.empty(n, dtype=torch.uint8, device="cuda")
        vr.vr_embedding_grad(None, 16, none, 0, 16, 10, vr.VR_FLOAT32, IGNORE, 1.0, add, old, work,
                             n, torch.cuda.current_stream())
        assert torch.equal(old, w if add else torch.zeros_like(w))


@pytest.mark.parametrize("T", [500, 9000])
def test_streams_and_graphs(T):
    """On another stream, and two captured calls with a workspace each, replayed
    on new inputs in place."""
    V, D = 3000, 48
    dout, ids = rand((T, D), torch.bfloat16, 1), words(T, V, 2)
    want = grad(dout, ids, V, vr.VR_BFLOAT16, 1.0, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = grad(dout, ids, V, vr.VR_BFLOAT16, 1.0, None, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    n = vr.vr_embedding_grad_workspace_bytes(T, D, V, vr.VR_BFLOAT16)
    graphs = []
    for k in range(2):
        work = torch.empty(n, dtype=torch.uint8, device="cuda")
        dw = torch.empty(V, D, device="cuda", dtype=torch.bfloat16)
        mine = ids.clone()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            vr.vr_embedding_grad(dout, D, mine, T, D, V, vr.VR_BFLOAT16, IGNORE, 1.0, False, dw,
                                 work, n, torch.cuda.current_stream())
        graphs.append((graph, mine, dw, work))
    new = words(T, V, 77)
    graphs[1][1].copy_(new)
    for _ in range(2):
        for graph, *_ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][2], want)
    assert torch.equal(graphs[1][2], grad(dout, new, V, vr.VR_BFLOAT16, 1.0, None))


def test_gradient_against_differences():
    """The lookup is linear: its change along a direction is the gradient's
    product with the direction."""
    w, ids = rand((30, 16), torch.float32, 1).double(), words(50, 30, 3, 0.1)
    dout, d = rand((50, 16), torch.float32, 2), rand((30, 16), torch.float32, 3)
    out = [lookup((w + s * d.double()).float(), ids, vr.VR_FLOAT32, 1.5) for s in (-1.0, 1.0)]
    change = float(((out[1] - out[0]).double() * dout.double()).sum()) / 2
    got = grad(dout, ids, 30, vr.VR_FLOAT32, 1.5, None)
    size = float(((out[1].abs() + out[0].abs()).double() * dout.abs().double()).sum())
    assert abs(change - float((got.double() * d.double()).sum())) <= 8 * 2.0 ** -24 * size
