"""vr_grouped_linear and vr_grouped_linear_grad against their definitions in 64
bits (more_refs.py)."""

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import double_binary_tree_gb300 as vr  # noqa: E402
from tests import more_refs, operator_refs as refs  # noqa: E402
from tests.test_gpu_operator_memory import Arena  # noqa: E402

DT = {"fp16": (vr.VR_FLOAT16, torch.float16), "bf16": (vr.VR_BFLOAT16, torch.bfloat16)}


class Case:
    def __init__(self, counts, K, N, dtype, spare=0, seed=0, pad=0, offset=0):
        self.counts, self.K, self.N = counts, K, N
        self.code, self.ty = DT[dtype]
        self.rows, self.used, self.E = sum(counts) + spare, sum(counts), len(counts)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def make(rows, cols, scale=1.0):
            wide = (torch.randn(rows, cols + pad, generator=g, device="cuda") * scale).to(self.ty)
            flat = torch.empty(wide.numel() + offset, device="cuda", dtype=self.ty)[offset:]
            out = flat.view(wide.shape)
            out.copy_(wide)
            return out[:, :cols]

        self.x, self.dy = make(self.rows, K), make(self.rows, N)
        w = torch.randn(self.E * N * K + offset, generator=g, device="cuda") / math.sqrt(K)
        self.w = w.to(self.ty)[offset:].view(self.E, N, K)
        self.device_counts = torch.tensor(counts, device="cuda", dtype=torch.int32)
        self.pad = pad

    def linear(self, offset=0, out_pad=0, arena=None, stream=None, out_offset=0):
        arena = arena or Arena()
        xs, os = self.K + self.pad, self.N + out_pad
        n = vr.vr_grouped_linear_workspace_bytes(self.x, xs, self.w, self.rows, self.K, self.N,
                                                 self.E, self.code)
        work = arena.cut(n, offset)
        out = arena.like((max(self.rows, 1) * os,), self.ty, out_offset)
        vr.vr_grouped_linear(self.x, xs, self.w, self.device_counts, self.rows, self.K, self.N,
                             self.E, self.code, out, os, work, n,
                             stream or torch.cuda.current_stream())
        return out.view(-1, os)

    def grad(self, offset=0, arena=None, dx=True, dw=True, stream=None, out_offset=0):
        arena = arena or Arena()
        xs, ys = self.K + self.pad, self.N + self.pad
        n = vr.vr_grouped_linear_grad_workspace_bytes(self.dy, ys, self.x, xs, self.w, self.rows,
                                                      self.K, self.N, self.E, self.code)
        work = arena.cut(n, offset)
        gx = arena.like((self.rows, self.K), self.ty, out_offset) if dx else None
        gw = arena.like((self.E, self.N, self.K), self.ty, out_offset) if dw else None
        vr.vr_grouped_linear_grad(self.dy, ys, self.x, xs, self.w, self.device_counts, self.rows,
                                  self.K, self.N, self.E, self.code, gx, gw, work, n,
                                  stream or torch.cuda.current_stream())
        return gx, gw


def untouched(t):
    return bool((t.contiguous().view(torch.uint8) == 255).all())


def check(case, forward=True, backward=True, status=0, **kw):
    if forward:
        arena = Arena()
        got = case.linear(arena=arena, **kw)
        assert vr.vr_stream_status() == status and arena.intact()
        want, bound = more_refs.grouped(case.x, case.w, case.counts)
        refs.assert_close(got[:case.used, :case.N], want[:case.used], bound[:case.used], case.ty,
                          "out")
        assert untouched(got[case.used:]) and untouched(got[:case.used, case.N:])
    if backward:
        arena = Arena()
        gx, gw = case.grad(arena=arena)
        assert vr.vr_stream_status() == status and arena.intact()
        dx, bx, dw, bw = more_refs.grouped_grad(case.dy, case.x, case.w, case.counts)
        refs.assert_close(gx[:case.used], dx[:case.used], bx[:case.used], case.ty, "dX")
        assert untouched(gx[case.used:])
        refs.assert_close(gw, dw, bw, case.ty, "dWeight")


# few rows a group, some, many: the three kinds of tiles
COUNTS = [
    [1], [8], [33], [0, 1, 0], [1, 0, 2, 31, 32, 33, 0, 7], [0, 5, 0, 40, 64, 65, 127, 128, 129, 0],
    [300, 0, 257, 1], [700, 600, 0, 900, 513, 600], [1500], [1] * 200,
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("K,N", [(64, 64), (200, 136), (72, 520), (520, 264), (8, 8)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "%dx%d" % (len(c), sum(c)))
def test_matches_the_definition(counts, K, N, dtype):
    check(Case(counts, K, N, dtype, seed=K + N + sum(counts)))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("K,N", [(65, 64), (64, 65), (33, 7), (1, 1), (1001, 130), (130, 1001)])
@pytest.mark.parametrize("counts", [[3, 0, 40], [100, 1, 200], [600, 530]],
                         ids=lambda c: "%dx%d" % (len(c), sum(c)))
def test_odd_sizes(counts, K, N, dtype):
    check(Case(counts, K, N, dtype, seed=K + N))


@pytest.mark.parametrize("K,N,pad,offset,out_pad,out_offset", [
    (64, 64, 8, 0, 8, 0), (64, 64, 3, 0, 5, 0), (64, 64, 0, 1, 0, 2), (64, 96, 0, 8, 16, 16),
    (72, 40, 16, 4, 1, 6)])
@pytest.mark.parametrize("counts", [[3, 0, 40], [100, 1, 200]],
                         ids=lambda c: "%dx%d" % (len(c), sum(c)))
def test_strides_and_alignment(counts, K, N, pad, offset, out_pad, out_offset):
    case = Case(counts, K, N, "bf16", pad=pad, offset=offset)
    check(case, out_pad=out_pad, out_offset=out_offset)
    # workspaces at other places, and each gradient by itself: the same bits
    whole = case.grad()
    first = case.linear(out_pad=out_pad)
    for at in (16, 240):
        again = case.linear(offset=at, out_pad=out_pad)
        assert torch.equal(first[:, :N], again[:, :N])  # (NaN between the rows)
        again = case.grad(offset=at, dw=False)[0], case.grad(offset=at, dx=False)[1]
        assert all(torch.equal(a, b) for a, b in zip(whole, again))


@pytest.mark.parametrize("counts", [[5, 0, 17, 30], [100, 3, 0, 200], [555, 600]],
                         ids=lambda c: "%dx%d" % (len(c), sum(c)))
def test_rows_behind_the_last_group(counts):
    """They may hold anything, and stay as they were."""
    case = Case(counts, 96, 160, "bf16", spare=70)
    case.x[case.used:] = math.nan
    case.dy[case.used:] = math.inf
    check(case)


@pytest.mark.parametrize("counts", [[5, 17, 0, 30], [100, 3, 0, 200], [555, 600, 700]],
                         ids=lambda c: "%dx%d" % (len(c), sum(c)))
def test_a_group_does_not_see_its_neighbours(counts):
    case = Case(counts, 96, 160, "bf16")
    clean = [case.linear()] + list(case.grad())
    lo = counts[0]
    hi = lo + counts[1]
    for t in (case.x, case.dy):
        t[lo:hi] = math.nan
    got = [case.linear()] + list(case.grad())
    for a, b in zip(clean[:2], got[:2]):  # rows
        assert torch.equal(a[:lo], b[:lo]) and torch.equal(a[hi:], b[hi:])
        assert bool(torch.isnan(b[lo:hi]).all())
    keep = [e for e in range(len(counts)) if e != 1]
    assert torch.equal(clean[2][keep], got[2][keep]) and bool(torch.isnan(got[2][1]).all())


@pytest.mark.parametrize("bad,held", [([5, -3, 10], [5, 0, 10]), ([5, 30, 10], [5, 15, 0]),
                                      ([2 ** 31 - 1, 2 ** 31 - 1, 7], [20, 0, 0])])
def test_bad_counts_are_cut_off_and_reported(bad, held):
    case = Case(held, 64, 64, "bf16", spare=20 - sum(held))
    case.device_counts.copy_(torch.tensor(bad, dtype=torch.int32))
    check(case, backward=False, status=vr.VR_ERR_INVALID_ARGUMENT)
    check(case, forward=False, status=vr.VR_ERR_INVALID_ARGUMENT)


def test_no_rows():
    case = Case([0, 0], 64, 72, "fp16")
    case.linear()
    _, gw = case.grad()
    assert vr.vr_stream_status() == 0 and not gw.any()
    spare = Case([0, 0], 64, 72, "fp16", spare=9)
    check(spare)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_long_sums(dtype):
    """Sums that are taken in chunks: the truncation of a plain accumulator
    would show in fp16."""
    n = 33000 if dtype == "fp16" else 263000
    check(Case([7, 3], n, 16, dtype), backward=False)
    check(Case([40, 66], n, 8, dtype), backward=False)
    check(Case([600], n, 8, dtype), backward=False)
    check(Case([7, 3], 16, n, dtype), forward=False)
    case = Case([n, 77], 24, 32, dtype)
    check(case, forward=False)
    _, gw = case.grad()
    _, _, dw, _ = more_refs.grouped_grad(case.dy, case.x, case.w, case.counts)
    assert refs.norm_error(gw, dw) <= refs.U_T[case.ty]


def test_many_groups():
    g = torch.Generator()
    g.manual_seed(1)
    counts = torch.randint(0, 6, (1024,), generator=g).tolist()
    check(Case(counts, 64, 40, "bf16", spare=3))
    check(Case([0] * 1023 + [300], 64, 40, "bf16"))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("mean,K,N", [(9, 264, 520), (9, 72, 1040), (50, 64, 1600), (50, 520, 100),
                                      (700, 1032, 2056)])
def test_many_tiles(mean, K, N, dtype):
    """Several tiles for every CTA; groups of very different sizes."""
    g = torch.Generator()
    g.manual_seed(mean)
    n = 16 if mean == 700 else 300
    counts = (torch.exp(torch.randn(n, generator=g)) * mean * 0.6).long().clamp(max=40 * mean)
    counts[::7] = 0
    case = Case(counts.tolist(), K, N, dtype, spare=5)
    check(case)
    again = [case.linear()[:case.used]] + list(case.grad())
    got = [case.linear()[:case.used]] + list(case.grad())
    assert torch.equal(again[0], got[0]) and torch.equal(again[2], got[2])
    assert torch.equal(again[1][:case.used], got[1][:case.used])


@pytest.mark.parametrize("counts", [[5, 0, 17], [100, 3, 200], [555, 600]],
                         ids=lambda c: "%dx%d" % (len(c), sum(c)))
def test_streams_and_graphs(counts):
    """On another stream, and two captured calls with a workspace each; a
    replay takes the counts that are there then."""
    case, other = Case(counts, 96, 160, "bf16"), Case(counts, 100, 161, "bf16", seed=5)
    want = [[c.linear()] + list(c.grad()) for c in (case, other)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [case.linear(stream=side)] + list(case.grad(stream=side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    graphs = []
    for c in (case, other):
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        arena = Arena()
        with torch.cuda.graph(graph):
            out = [c.linear(arena=arena)] + list(c.grad(arena=arena))
        graphs.append((graph, out, arena))
    for _ in range(2):
        for graph, *_ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for (_, out, _), w in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(out, w))
    new = counts[1:] + counts[:1]
    case.counts = new
    case.device_counts.copy_(torch.tensor(new, dtype=torch.int32))
    graphs[0][0].replay()
    assert vr.vr_stream_status() == 0
    again = [case.linear()] + list(case.grad())
    assert all(torch.equal(a, b) for a, b in zip(graphs[0][1], again))
    check(case)


def test_gradients_against_differences():
    """The product is linear in each argument: its change along a direction is
    the gradient's product with the direction (bf16 results: within their
    roundings)."""
    case = Case([9, 0, 30], 48, 56, "bf16")
    gx, gw = case.grad()
    y0 = case.linear().double()
    dy = case.dy.double()
    for t, got in ((case.x, gx), (case.w, gw)):
        saved = t.clone()
        t.add_(torch.randn_like(t))
        d = (t.double() - saved.double())  # as it was rounded
        y1 = case.linear().double()
        t.copy_(saved)
        change = float(((y1 - y0) * dy).sum())
        slack = 2.0 ** -8 * float(((y1.abs() + y0.abs()) * dy.abs()).sum())
        slack += 2.0 ** -8 * float((got.double().abs() * d.abs()).sum())
        assert abs(change - float((got.double() * d).sum())) <= slack
