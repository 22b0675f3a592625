"""vr_linear_xent's gradients over long sums: the tensor cores truncate where they
add, which pulls a long sum towards zero as a whole."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import double_binary_tree_gb300 as vr  # noqa: E402
from tests.test_gpu_linear_xent import call, make  # noqa: E402


def pull(got, want):
    """How much larger the result is along the exact one."""
    return float((got.double() * want).sum() / (want * want).sum()) - 1.0


FP16, BF16 = torch.float16, torch.bfloat16


@pytest.mark.parametrize("T,D,V,ty", [
    (1024, 4096, 131072, FP16),              # dHidden over the vocabulary
    (300, 1024, 400000, FP16), (100, 512, 400000, FP16),  # shared out over clusters
    (1, 64, 300000, FP16),
    (4100, 64, 70000, FP16),                 # in pieces
    (70000, 64, 500, FP16), (70000, 64, 100, FP16),       # dWeight over the tokens
    (2000, 2048, 300000, BF16), (100, 128, 2200000, BF16),
    (600000, 64, 500, BF16), (600000, 64, 100, BF16)])
def test_long_sums_are_not_pulled_to_zero(T, D, V, ty):
    """At most 2048 k are added up in the tensor cores before a rounded sum, 128
    additions truncated by 2^-23 each at most: 2^-16.  (Sums of up to 32768 in
    fp16 and 262144 in bf16, times the CTAs of a cluster, are taken in one go;
    they are not looked at here.)  The factors are 16-bit numbers; their own
    rounding (that of a target's 1 - p is the same for many tokens) is part of
    the reference.  The rest is independent roundings, u / 2 each."""
    h, w, y = make(T, D, V, ty, 41)
    half = ty == FP16
    scale, up = (64.0 * T, 2.0 ** 14) if half else (1.0, 1.0)
    longest = 32768 if half else 262144
    got = call(h, w, y, vr.VR_FLOAT16 if half else vr.VR_BFLOAT16, scale=scale)
    assert vr.vr_stream_status() == 0
    dh, dw = torch.zeros(T, D, **f64()), torch.zeros(V, D, **f64())
    for lo in range(0, T, 1024):
        hi = min(T, lo + 1024)
        p = torch.softmax(h[lo:hi].double() @ w.double().t(), 1)
        p[torch.arange(hi - lo, device="cuda"), y[lo:hi]] -= 1.0
        p = (p * up).to(ty).double() * (scale / T / up)
        dh[lo:hi] = p @ w.double()
        dw.addmm_(p.t(), h[lo:hi].double())
    for g, want, k in ((got[3], dh, V), (got[4], dw, T)):
        u = 2.0 ** -11 if half else 2.0 ** -8
        limit = 2.0 ** -16 + 4 * u / 2 / want.numel() ** 0.5 + 2.0 ** -18
        assert k <= longest or abs(pull(g, want)) <= limit


def f64():
    return dict(dtype=torch.float64, device="cuda")
