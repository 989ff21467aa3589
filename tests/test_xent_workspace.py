"""The cross entropy's workspace holds the pairs of every lane, by the bytes
asked for (CPU), and on the GPU nothing changes behind a workspace of exactly
the stated size."""
import ctypes

import pytest
import torch

import sequence_ref as R
from dense_guard import guard
from recsys_sparse_embedding_gb300 import binding as B
from recsys_sparse_embedding_gb300 import build as nbuild

BF16, F32 = torch.bfloat16, torch.float32
SMS = 152


def group_of(mt, clusters):
    """M tiles that are worked on together: 4, or fewer where those would leave
    more clusters (by 3 of 100) without work than the last choice does."""
    best, most = 1, 0.0
    for gm in (4, 2, 1):
        if gm > clusters:
            continue
        e = mt / (-(-mt // gm) * gm) * (clusters // gm * gm) / clusters
        if e > most + 0.03:
            best, most = gm, e
    return best


def slots(mt, nt, rows):
    """Clusters that have pairs of one row: those that share out its N tiles."""
    clusters = min(mt * nt, SMS * 128 // rows)
    return min(nt, clusters // group_of(mt, clusters))


@pytest.fixture(scope="module")
def L():
    nbuild.build()
    return B.lib()


@pytest.mark.parametrize("rows", [128, 256])
def test_the_workspace_holds_every_lanes_pairs(L, rows):
    # (bf16 and K = 256: neither x nor W is laid out, no bias kept; so pairs and the targets' logits)
    layer = B.CDense(4096, None, None, 256, 1000, 256, B.DSF_BF16, B.DSF_ACT_NONE)
    for mt in list(range(1, 600)) + [1000, 2047, 4096]:
        for nt in (1, 2, 3, 4, 7, 8, 38, 40, 51, 76, 101, 152, 4000):
            n = slots(mt, nt, rows)
            for M in ((mt - 1) * rows + 1, mt * rows - 31, mt * rows):
                need = n * 4 * M * 8 + 4 * M
                got = L.dsf_softmax_xent_workspace_bytes(ctypes.byref(layer), M, 0)
                assert got >= need, (mt, nt, M, got, need)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,K", [(BF16, 176), (BF16, 256), (F32, 48)])
@pytest.mark.parametrize("M,V", [(11300, 13000), (11392, 13000), (11800, 13000), (11904, 13001), (15400, 98), (16768, 128),
                                 (23808, 700), (5, 3000), (300, 20001), (700, 5)])
def test_nothing_is_written_behind_the_forwards_workspace(dtype, K, M, V):
    g = torch.Generator(device="cuda")
    g.manual_seed(M + K)
    x = torch.randn(M, K, generator=g, device="cuda").to(dtype)
    W = (torch.randn(V, K, generator=g, device="cuda") * 1.5 * K ** -0.5).to(dtype)
    layer = B.DenseLayer(W, torch.randn(V, generator=g, device="cuda"))
    target = torch.randint(-1, V, (M,), generator=g, device="cuda")
    loss, lse = torch.full((M,), float("nan"), device="cuda"), torch.full((M,), float("nan"), device="cuda")
    ws = B.SoftmaxXentWorkspace(layer, M)
    intact = guard(ws)
    B.ctr_softmax_xent_fwd(layer, x, target, loss, lse, ws)
    assert intact()
    for r in range(0, M, 2000):
        rows = slice(r, r + 2000)
        ref = R.xent(x[rows], W, layer.bias, target[rows])
        R.assert_within(loss[rows], ref["loss"], "loss")
        there = target[rows] >= 0  # (a row left out has its own x, which the reference drops)
        R.assert_within(lse[rows][there], (ref["lse"][0][there], ref["lse"][1][there]), "lse")


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,V", [(1, 64, 100001), (4, 256, 3000), (120, 8, 840001), (513, 16, 200001), (1024, 64, 98304), (5000, 100, 20011),
                                   (65536, 24, 1600), (20000, 128, 5003)])
def test_nothing_is_written_behind_a_narrow_forwards_workspace(M, K, V):
    """few rows, or the sums in one pass"""
    g = torch.Generator(device="cuda")
    g.manual_seed(M + K)
    x = torch.randn(M, K, generator=g, device="cuda").to(BF16)
    W = (torch.randn(V, K, generator=g, device="cuda") * 1.5 * K ** -0.5).to(BF16)
    target = torch.randint(-1, V, (M,), generator=g, device="cuda")
    for bias in (None, torch.randn(V, generator=g, device="cuda")):
        layer = B.DenseLayer(W, bias)
        loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        ws = B.SoftmaxXentWorkspace(layer, M)
        intact = guard(ws)
        B.ctr_softmax_xent_fwd(layer, x, target, loss, lse, ws)
        assert intact()
        assert torch.isfinite(loss).all() and torch.isfinite(lse).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,M,K,V", [(BF16, 5, 64, 3000), (BF16, 700, 64, 70001), (BF16, 700, 72, 5), (F32, 333, 48, 2001),
                                         (BF16, 2000, 136, 12345), (F32, 3000, 20, 16001), (BF16, 70001, 64, 901)])
def test_nothing_is_written_behind_the_backwards_workspace(dtype, M, K, V):
    g = torch.Generator(device="cuda")
    g.manual_seed(M + K)
    x = torch.randn(M, K, generator=g, device="cuda").to(dtype)
    W = (torch.randn(V, K, generator=g, device="cuda") * 1.5 * K ** -0.5).to(dtype)
    layer = B.DenseLayer(W, torch.randn(V, generator=g, device="cuda"))
    target = torch.randint(-1, V, (M,), generator=g, device="cuda")
    loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    ws = B.SoftmaxXentWorkspace(layer, M, backward=True)
    intact = guard(ws)
    B.ctr_softmax_xent_fwd(layer, x, target, loss, lse, ws)
    assert intact()
    out = dict(dx=torch.empty_like(x), dW=torch.empty_like(W), db=torch.empty(V, device="cuda"))
    for names in (("dx", "dW", "db"), ("dx",), ("dW",), ("db",)):
        intact = guard(ws)
        B.ctr_softmax_xent_bwd(layer, x, target, lse, ws, **{n: out[n] for n in names})
        assert intact(), names
