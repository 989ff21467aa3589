"""Long sums of one sign in bf16 and e4m3 layers, whose results are rounded to
bf16: the accumulation's own loss stays well below that rounding."""
import pytest
import torch

import dense_ref as R
from dense_guard import guard
from recsys_sparse_embedding_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
# An accumulator takes at most 1024 K-blocks of four additions, each truncated by less than 2^-23 of
# it; parts are added with a rounding each (32 at most), 8 for the bias and the rest.
LOSS = (4096 + 16 + 8) * R.U


def check(got, ref):
    """Each value is one that some sum within the loss rounds to: between the
    roundings of both ends (rounding keeps the order)."""
    lo, hi = (ref * (1 - LOSS)).to(BF16), (ref * (1 + LOSS)).to(BF16)
    bad = int(((got < lo) | (got > hi)).sum())
    assert bad == 0, "%d of %d, off by %.3g in the mean" % (bad, ref.numel(), float(((got.double() - ref) / ref).mean()))


def positive(g, *shape, a=1.0):
    return torch.rand(*shape, generator=g, device="cuda") * a


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,K", [(40, 24, 65600), (300, 136, 1 << 18), (40, 24, 1 << 20), (2600, 2048, 1 << 18)])
def test_long_inputs(dtype, gated, M, N, K):
    """Sums over up to 2^20 inputs; the last case has more tiles than the chip
    takes at once."""
    g = torch.Generator(device="cuda")
    g.manual_seed(K + M)
    rows = 2 * N if gated else N
    W, x = positive(g, rows, K).to(dtype), positive(g, M, K).to(dtype)
    ws, xs = (torch.full((n,), 4.0 / K if n == rows else 1.0, device="cuda") if dtype == E4M3 else None for n in (rows, M))
    if dtype == BF16:
        W = W * (4.0 / K)
        if gated:
            W[:N] = 0.0  # (the gate comes from its bias; the product of two halves would have two losses)
    elif gated:
        W.view(torch.uint8)[:N] = 0
    b = torch.ones(rows, device="cuda")
    layer = B.DenseLayer(W, b, act=B.DSF_ACT_RELU, scale=ws)
    y = torch.empty(M, N, dtype=BF16, device="cuda")
    work = B.DenseWorkspace(layer, M, gated=gated)
    intact = guard(work)
    (B.ctr_glu_fwd if gated else B.ctr_dense_fwd)(layer, x, y, work, x_scale=xs)
    assert intact()
    cols = slice(N, N + 80) if gated else slice(0, 80)
    check(y[:40, :80], x[:40].double() @ W[cols].double().t() * (4.0 / K if dtype == E4M3 else 1.0) + 1)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("both", [True, False])
@pytest.mark.parametrize("M,K,N", [(40, 64, 1 << 18), (1 << 18, 64, 40), (1 << 18, 2560, 2048), (70000, 264, 72)])
def test_long_gradients(gated, both, M, K, N):
    """dx sums over many outputs, dW over many rows (one of them more than the
    chip has tiles for at once). Positive throughout; a gated layer's gate is 1,
    from its bias, so that du is dy."""
    if gated and (N == 1 << 18 or N == 2048):
        N //= 2
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N)
    rows = 2 * N if gated else N
    x, dy = positive(g, M, K).to(BF16), positive(g, M, N).to(BF16)
    W = positive(g, rows, K).to(BF16)
    if gated:
        W[:N] = 0
    layer = B.DenseLayer(W, torch.ones(rows, device="cuda") if gated else None, act=B.DSF_ACT_RELU if gated else B.DSF_ACT_NONE)
    out = dict(dx=torch.empty_like(x), dW=torch.empty_like(W))
    ws = B.DenseWorkspace(layer, M, gated=gated, backward=True)
    bwd = B.ctr_glu_bwd if gated else B.ctr_dense_bwd
    for names in (("dx", "dW"),) if both else (("dx",), ("dW",)):
        intact = guard(ws)
        bwd(layer, x, dy, ws, **{n: out[n] for n in names})
        assert intact()
    d, some = dy.double(), slice(0, 40)  # (a gated layer's gate rows of W are zero: dx is du Wu)
    rows_m = slice(0, min(M, 2000))
    check(out["dx"][rows_m], d[rows_m] @ (W[N:] if gated else W).double())
    check(out["dW"][N:][some] if gated else out["dW"][some], d[:, some].t() @ x.double())


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N", [(40, 72), (600, 512)])
def test_long_inputs_of_the_gradients(gated, M, N, monkeypatch):
    """dz's sums over more than 65536 inputs, with db and without: z near 2 from
    terms of one sign, each gradient within the bound of sums in runs of at most
    32 additions."""
    K = 70000
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    rows = 2 * N if gated else N
    W, x = (positive(g, rows, K) * (8.0 / K)).to(BF16), positive(g, M, K).to(BF16)
    layer = B.DenseLayer(W, torch.zeros(rows, device="cuda"), act=B.DSF_ACT_SILU)
    dy = positive(g, M, N).to(BF16)

    def pre(x, W, b):
        z = x.double() @ W.double().t() + b.double()  # (its terms have one sign)
        return z, (32 + K / 1024 + 8) * R.U * z + 1e-38
    monkeypatch.setattr(R, "pre", pre)
    ref = R.grads(x, W, layer.bias, "silu", dy, gated)
    ws = B.DenseWorkspace(layer, M, gated=gated, backward=True)
    for names in (("dx", "dW"), ("dx", "dW", "db")):
        out = {"dx": torch.empty_like(x), "dW": torch.empty_like(W), "db": torch.empty(rows, device="cuda")}
        intact = guard(ws)
        (B.ctr_glu_bwd if gated else B.ctr_dense_bwd)(layer, x, dy, ws, **{n: out[n] for n in names})
        assert intact()
        for n in names:
            R.assert_within(out[n], *ref[n], "%s of %s" % (n, names))
