"""The backward of the layers at values of z = x W^T + bias that are known
exactly, and at sums of one sign and of mostly zeros."""
import math

import pytest
import torch

import dense_ref as R
from recsys_sparse_embedding_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32



@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K", [64, 1024, 65536])
def test_an_exact_zero_stays_zero_in_the_backward(dtype, gated, K):
    """z = x W^T + bias is exactly zero (sums of ones, less their count), so
    ReLU's gradient is."""
    M, N = 40, 72
    rows = 2 * N if gated else N
    b = torch.full((rows,), -float(K), device="cuda")
    b[N:] = 1.0  # (a gated layer's up half: no zero there)
    layer = B.DenseLayer(torch.ones(rows, K, dtype=dtype, device="cuda"), b, act=B.DSF_ACT_RELU)
    x = torch.ones(M, K, dtype=dtype, device="cuda")
    y, dy = torch.ones(M, N, dtype=dtype, device="cuda"), torch.ones(M, N, dtype=dtype, device="cuda")
    out = dict(dx=torch.ones_like(x), dW=torch.ones_like(layer.W), db=torch.ones(rows, device="cuda"))
    ws = B.DenseWorkspace(layer, M, gated=gated, backward=True)
    (B.ctr_glu_fwd if gated else B.ctr_dense_fwd)(layer, x, y, ws)
    (B.ctr_glu_bwd if gated else B.ctr_dense_bwd)(layer, x, dy, ws, **out)
    assert not y.any()
    for n, t in out.items():
        assert not t.any(), n


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K", [256, 65536])
def test_db_at_a_z_that_is_exact(dtype, K):
    """z = 1 exactly (K products of 1 / K): db is 64 times SiLU's slope there,
    whose evaluation is off by at most 2^-19; equal values add up exactly."""
    M, N = 64, 48
    layer = B.DenseLayer(torch.full((N, K), 1.0 / K, dtype=dtype, device="cuda"), None, act=B.DSF_ACT_SILU)
    x, dy = torch.ones(M, K, dtype=dtype, device="cuda"), torch.ones(M, N, dtype=dtype, device="cuda")
    db = torch.empty(N, device="cuda")
    B.ctr_dense_bwd(layer, x, dy, B.DenseWorkspace(layer, M, backward=True), db=db)
    p = 1 / (1 + math.exp(-1.0))
    want = M * p * (1 + (1 - p))
    assert float((db.double() - want).abs().max()) <= 2.0 ** -19 * want


def pre_in_runs(x, W, b):
    """z and the bound of its error where no more than 32 additions (8 K-blocks of
    64, 16 terms each) go to an accumulator that truncates, by less than 2^-23
    of it each, and the sums of those runs are rounded, by 2^-24 each; 8 for the
    bias and the rest."""
    x, W = x.double(), W.double()
    z, a = x @ W.t() + b.double(), x.abs() @ W.abs().t() + b.double().abs()
    return z, (32 + x.shape[1] / 1024 + 8) * R.U * a + 1e-38


@pytest.mark.parametrize("kind", ["one sign", "mostly zero"])
@pytest.mark.parametrize("K", [500, 2048, 40000])
@pytest.mark.parametrize("gated", [False, True])
def test_gradients_at_sums_of_one_sign_and_of_mostly_zeros(kind, K, gated, monkeypatch):
    """Non-negative inputs, weights and upstream gradients, and inputs of which
    one in 64 is not zero, at long K: each gradient within its bound, and db,
    which is fp32, within one that does not grow with K as a truncating sum's."""
    g = torch.Generator(device="cuda")
    g.manual_seed(K)
    M, N = 96, 56
    rows = 2 * N if gated else N
    W, x = torch.rand(rows, K, generator=g, device="cuda"), torch.rand(M, K, generator=g, device="cuda")
    if kind == "one sign":
        W = W * (4.0 / K)  # (z near 1)
    else:
        W = W - 0.5
        x = x * (torch.rand(M, K, generator=g, device="cuda") < 1 / 64)
    x, W = x.to(BF16), W.to(BF16)
    layer = B.DenseLayer(W, 0.1 * torch.randn(rows, generator=g, device="cuda"), act=B.DSF_ACT_SILU)
    dy = torch.rand(M, N, generator=g, device="cuda").to(BF16)
    out = dict(dx=torch.empty_like(x), dW=torch.empty_like(W), db=torch.empty(rows, device="cuda"))
    ws = B.DenseWorkspace(layer, M, gated=gated, backward=True)
    (B.ctr_glu_bwd if gated else B.ctr_dense_bwd)(layer, x, dy, ws, **out)
    for n, (ref, tol) in R.grads(x, W, layer.bias, "silu", dy, gated).items():
        R.assert_within(out[n], ref, tol, n)
    monkeypatch.setattr(R, "pre", pre_in_runs)
    ref, tol = R.grads(x, W, layer.bias, "silu", dy, gated)["db"]
    R.assert_within(out["db"], ref, tol, "db")
