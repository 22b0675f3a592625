"""Embedding, AdamW and grouped products with tables, weights and tensors of
more than 2^31 elements: what lies behind them is checked."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import double_binary_tree_gb300 as vr  # noqa: E402
from tests import more_refs, operator_refs as refs  # noqa: E402

B16, BF = torch.bfloat16, vr.VR_BFLOAT16


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:  # pragma: no cover
        pytest.skip("needs 60 GB of free memory")
    yield
    torch.cuda.empty_cache()


def test_embedding():
    V, D, T = 40000, 65536, 300
    w = torch.empty(V, D, device="cuda", dtype=B16)
    ids = torch.randint(V - 3000, V, (T,), device="cuda")
    ids[:3] = torch.tensor([0, V - 1, V - 1], device="cuda")
    w[ids] = torch.randn(T, D, device="cuda").to(B16)
    out = torch.empty(T, D, device="cuda", dtype=B16)
    vr.vr_embedding(w, D, ids, T, D, V, BF, -100, 1.0, out, D, torch.cuda.current_stream())
    assert vr.vr_stream_status() == 0
    assert torch.equal(out, w[ids])
    # the gradient into the same buffer: every other row becomes zero
    n = vr.vr_embedding_grad_workspace_bytes(T, D, V, BF)
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    vr.vr_embedding_grad(out, D, ids, T, D, V, BF, -100, 1.0, False, w, work, n,
                         torch.cuda.current_stream())
    assert vr.vr_stream_status() == 0
    words = torch.unique(ids)
    part = torch.searchsorted(words, ids)
    want, bound = more_refs.embedding_grad(out, part, len(words), 1.0)
    refs.assert_close(w[words], want, bound, B16)
    w[words] = 0
    assert all(not bool(w[lo:lo + 4000].any()) for lo in range(0, V, 4000))


def test_grouped():
    """The last of 40 groups lies behind 2^31 elements of the weight."""
    E, N, K = 40, 8192, 8192
    counts = [0] * E
    counts[0], counts[-1] = 9, 70
    rows = sum(counts)
    w = torch.zeros(E, N, K, device="cuda", dtype=B16)
    for e in (0, E - 1):
        w[e] = (torch.randn(N, K, device="cuda") / 90).to(B16)
    x, dy = (torch.randn(rows, n, device="cuda").to(B16) for n in (K, N))
    c = torch.tensor(counts, device="cuda", dtype=torch.int32)
    out, dx = torch.empty_like(dy), torch.empty_like(x)
    n = vr.vr_grouped_linear_workspace_bytes(x, K, w, rows, K, N, E, BF)
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    vr.vr_grouped_linear(x, K, w, c, rows, K, N, E, BF, out, N, work, n,
                         torch.cuda.current_stream())
    n = vr.vr_grouped_linear_grad_workspace_bytes(dy, N, x, K, w, rows, K, N, E, BF)
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    vr.vr_grouped_linear_grad(dy, N, x, K, w, c, rows, K, N, E, BF, dx, None, work, n,
                              torch.cuda.current_stream())
    few, few_counts = w[[0, E - 1]], [9, 70]
    want, bound = more_refs.grouped(x, few, few_counts)
    refs.assert_close(out, want, bound, B16, "out")
    want, bound, dw, bw = more_refs.grouped_grad(dy, x, few, few_counts)
    refs.assert_close(dx, want, bound, B16, "dX")
    # dW into the same buffer
    vr.vr_grouped_linear_grad(dy, N, x, K, w, c, rows, K, N, E, BF, None, w, work, n,
                              torch.cuda.current_stream())
    assert vr.vr_stream_status() == 0
    refs.assert_close(w[[0, E - 1]], dw, bw, B16, "dWeight")
    assert not any(bool(w[e].any()) for e in range(1, E - 1))


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw(bits):
    n = (1 << 31) + 4999
    p, g = (torch.zeros(n, device="cuda", dtype=B16) for _ in range(2))
    ty = torch.uint8 if bits == 8 else torch.float32
    m, v = (torch.zeros(n, device="cuda", dtype=ty) for _ in range(2))
    s = [torch.zeros(-(-n // 256), device="cuda") for _ in range(2)] if bits == 8 else None
    places = [slice(0, 2816), slice((1 << 31) - 768, (1 << 31) + 1024),
              slice((n - 2000) // 256 * 256, n)]  # whole blocks, but for the last
    for at in places:
        k = len(range(*at.indices(n)))
        p[at] = (0.1 * torch.randn(k, device="cuda")).to(B16)
        g[at] = torch.randn(k, device="cuda").to(B16)
    before = [(p[at].float().cpu().numpy(), g[at].float().cpu().numpy()) for at in places]
    vr.vr_adamw([p], [g], [m], [v], s and [s[0]], s and [s[1]], None, [n], 1, BF, BF, bits, 1e-2,
                0.9, 0.99, 1e-8, 0.1, 1, 1.0, 3, None, torch.cuda.current_stream())
    assert vr.vr_stream_status() == 0
    for at, (p0, g0) in zip(places, before):
        zero = 0 * p0
        want, bound, m1, v1 = more_refs.adamw(p0, g0, zero, zero, 1e-2, 0.9, 0.99, 1e-8, 0.1, 1,
                                              1.0)
        refs.assert_close(p[at].cpu(), torch.from_numpy(want), torch.from_numpy(bound), B16)
        if bits == 32:
            assert torch.equal(m[at].cpu(), torch.from_numpy(m1))
            assert torch.equal(v[at].cpu(), torch.from_numpy(v1))
        else:
            cut = more_refs.random_bits(3, 1, at.start, len(m1))
            codes, scales = more_refs.encode("m", m1, cut & 0xffff)
            assert torch.equal(m[at].cpu(), torch.from_numpy(codes))
            blocks = slice(at.start // 256, -(-at.stop // 256))
            assert torch.equal(s[0][blocks].cpu(), torch.from_numpy(scales))
    # nothing else has moved
    assert not bool(p[5000:1 << 30].any()) and not bool(m[5000:1 << 30].any())
