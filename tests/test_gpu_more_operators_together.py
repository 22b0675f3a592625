"""Embedding, grouped products and AdamW one after the other in a captured
graph, from several threads at once, and on several streams at once: the same
bits as one call after the other."""

import threading

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import double_binary_tree_gb300 as vr  # noqa: E402

B16, BF = torch.bfloat16, vr.VR_BFLOAT16
IGNORE = -100


class Chain:
    """Tokens embedded, times their group's weight, and back: the gradients of
    the weight and of the table, and an AdamW step on both."""

    def __init__(self, seed, T=500, D=96, N=200, E=6, V=700, bits=8):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=g, device="cuda")

        self.sizes = T, D, N, E, V
        self.ids = torch.randint(0, V, (T,), generator=g, device="cuda")
        cuts = torch.randint(0, T - 20, (E - 1,), generator=g, device="cuda").sort().values
        ends = torch.cat([cuts, torch.tensor([T - 20], device="cuda")])
        self.counts = torch.diff(ends, prepend=ends.new_zeros(1)).int()
        self.masters = [0.1 * randn(V, D), 0.1 * randn(E, N, D)]
        self.params = [w.to(B16) for w in self.masters]
        self.h, self.y = torch.zeros(T, D, device="cuda", dtype=B16), torch.zeros(
            T, N, device="cuda", dtype=B16)
        self.dh = torch.zeros_like(self.h)
        self.grads = [torch.zeros_like(w) for w in self.params]
        n = [w.numel() for w in self.params]
        ty = torch.uint8 if bits == 8 else torch.float32
        self.bits, self.n = bits, n
        self.m, self.v = ([torch.zeros(k, device="cuda", dtype=ty) for k in n] for _ in range(2))
        self.ms, self.vs = ([torch.zeros(-(-k // 256), device="cuda") for k in n] if bits == 8
                            else None for _ in range(2))
        self.control = torch.tensor([1e-3, 1.0, 1.0], device="cuda")
        w = self.params[1]
        self.work = [torch.empty(k, dtype=torch.uint8, device="cuda") for k in (
            vr.vr_grouped_linear_workspace_bytes(self.h, D, w, T, D, N, E, BF),
            vr.vr_grouped_linear_grad_workspace_bytes(self.y, N, self.h, D, w, T, D, N, E, BF),
            vr.vr_embedding_grad_workspace_bytes(T, D, V, BF))]

    def run(self, stream=None):
        T, D, N, E, V = self.sizes
        s = stream or torch.cuda.current_stream()
        table, w = self.params
        a, b, c = self.work
        vr.vr_embedding(table, D, self.ids, T, D, V, BF, IGNORE, 2.0, self.h, D, s)
        vr.vr_grouped_linear(self.h, D, w, self.counts, T, D, N, E, BF, self.y, N, a, a.numel(), s)
        # (the loss is half the square of y, whose gradient is y)
        vr.vr_grouped_linear_grad(self.y, N, self.h, D, w, self.counts, T, D, N, E, BF, self.dh,
                                  self.grads[1], b, b.numel(), s)
        vr.vr_embedding_grad(self.dh, D, self.ids, T, D, V, BF, IGNORE, 2.0, False, self.grads[0],
                             c, c.numel(), s)
        vr.vr_adamw(self.params, self.grads, self.m, self.v, self.ms, self.vs, self.masters,
                    self.n, 2, BF, BF, self.bits, 0.0, 0.9, 0.99, 1e-8, 0.1, 1, 1.0, 5,
                    self.control, s)

    def state(self):
        return self.masters + self.params + self.grads + self.m + self.v + [self.h, self.y, self.dh]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a.state(), b.state()))


@pytest.mark.parametrize("bits", [8, 32])
def test_a_captured_chain(bits):
    one, two = Chain(1, bits=bits), Chain(1, bits=bits)
    warm = Chain(1, bits=bits)
    warm.run()  # (the library loads its kernels)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        two.run()
    for step in range(1, 5):
        for c in (one, two):
            c.control.copy_(torch.tensor([1e-3 / step, float(step), 0.5]))
        one.run()
        graph.replay()
        assert vr.vr_stream_status() == 0
        assert same(one, two), step
    assert not torch.equal(one.masters[0], warm.masters[0])


def test_streams_at_once():
    want = [Chain(k, T=300 + 97 * k, D=64 + 8 * k, N=136 + 33 * k) for k in range(4)]
    got = [Chain(k, T=300 + 97 * k, D=64 + 8 * k, N=136 + 33 * k) for k in range(4)]
    streams = [torch.cuda.Stream() for _ in got]
    torch.cuda.synchronize()
    for _ in range(5):
        for c in want:
            c.run()
        for c, s in zip(got, streams):
            c.run(s)
    torch.cuda.synchronize()
    assert vr.vr_stream_status() == 0
    assert all(same(a, b) for a, b in zip(want, got))


def test_threads_at_once():
    want = [Chain(k, T=200 + 111 * k, N=101 + 50 * k) for k in range(4)]
    got = [Chain(k, T=200 + 111 * k, N=101 + 50 * k) for k in range(4)]
    for c in want:
        for _ in range(10):
            c.run()
    torch.cuda.synchronize()
    errors = []

    def work(chain):
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream()
            for _ in range(10):
                chain.run(stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in got]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    assert vr.vr_stream_status() == 0
    assert all(same(a, b) for a, b in zip(want, got))
