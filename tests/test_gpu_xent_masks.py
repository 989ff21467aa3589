"""Catalogues masked by finite values: a bias of the type's lowest value, or of any
other value far below the logits, takes an item out as -inf does; a row none of
whose items is left has lse -inf, loss NaN and no gradient."""
import pytest
import torch

import sequence_ref as R
from recsys_sparse_embedding_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
MASKS = [-1e9, -1e10, -7e15, -1e30, -2.5e38, float(torch.finfo(BF16).min), float(torch.finfo(F32).min)]


def run(dtype, M, K, V, b, target, seed=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(M, K, generator=g, device="cuda").to(dtype)
    W = (torch.randn(V, K, generator=g, device="cuda") * 1.5 * K ** -0.5).to(dtype)
    layer = B.DenseLayer(W, b)
    ws = B.SoftmaxXentWorkspace(layer, M, backward=True)
    o = {"loss": torch.empty(M, device="cuda"), "lse": torch.empty(M, device="cuda")}
    B.ctr_softmax_xent_fwd(layer, x, target, o["loss"], o["lse"], ws)
    o.update(dx=torch.full_like(x, 7.0), dW=torch.full_like(W, 7.0), db=torch.full_like(b, 7.0))
    B.ctr_softmax_xent_bwd(layer, x, target, o["lse"], ws, dx=o["dx"], dW=o["dW"], db=o["db"])
    return o


SIZES = [(BF16, 3, 64, 900), (F32, 4, 32, 900), (BF16, 200, 64, 900), (F32, 200, 48, 900), (BF16, 70, 200, 3001), (BF16, 900, 64, 120000)]


@pytest.mark.parametrize("dtype,M,K,V", SIZES)
def test_some_items_masked(dtype, M, K, V):
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    gone = torch.rand(V, generator=g, device="cuda") < 0.4
    gone[:300] = True  # whole tiles, the first ones
    b = torch.randn(V, generator=g, device="cuda")
    here = torch.nonzero(~gone)[:, 0]
    target = here[torch.randint(0, here.numel(), (M,), generator=g, device="cuda")]
    want = run(dtype, M, K, V, torch.where(gone, torch.full_like(b, -float("inf")), b), target)
    for mask in MASKS:
        got = run(dtype, M, K, V, torch.where(gone, torch.full_like(b, mask), b), target)
        for k in want:
            assert torch.equal(got[k], want[k]), (k, mask)


@pytest.mark.parametrize("dtype,M,K,V", SIZES)
def test_every_item_masked(dtype, M, K, V):
    target = torch.arange(M, device="cuda") % V
    for mask in MASKS:
        o = run(dtype, M, K, V, torch.full((V,), mask, device="cuda"), target)
        assert (o["lse"] == -float("inf")).all() and torch.isnan(o["loss"]).all(), mask
        for k in ("dx", "dW", "db"):
            assert (o[k] == 0).all(), (k, mask)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_logits_as_far_as_they_may_be(dtype):
    """All of one value, -6e8 to 6e8: lse is that and log V, rounded (a logit's
    step there is 64, the bound of sequence_ref counts it)."""
    M, K, V = 130, 64, 1000
    target = torch.arange(M, device="cuda") % V
    for b in (-6e8, -1e6, 1e6, 6e8):
        x = torch.zeros(M, K, device="cuda", dtype=dtype)
        W = torch.zeros(V, K, device="cuda", dtype=dtype)
        bias = torch.full((V,), b, device="cuda")
        layer = B.DenseLayer(W, bias)
        loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        B.ctr_softmax_xent_fwd(layer, x, target, loss, lse, B.SoftmaxXentWorkspace(layer, M))
        R.assert_within(lse, R.xent(x, W, bias, target)["lse"], b)
