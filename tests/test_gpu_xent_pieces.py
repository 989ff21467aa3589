"""The cross entropy's gradients over a catalogue in pieces, in bf16: where x and W
are wider than the one-pass gradients take, or the rows more, or the catalogue
smaller. dz of all columns passes a piece's 256 MB, and the last piece is short, so
dx is added up over pieces of two sizes (the shorter one with fewer splits), and
bias, targets and db are taken from the piece's first column on."""
import pytest
import torch

import sequence_ref as R
from recsys_sparse_embedding_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
PIECE = 256 << 20


def pieces(M, V):
    """Columns of each piece: whole tiles of 256."""
    p = max(256, PIECE // (2 * M) // 256 * 256)
    return [min(p, V - v) for v in range(0, V, p)]


@pytest.mark.parametrize("M,K,V", [(4097, 136, 40011), (9000, 200, 17003), (70001, 64, 4001), (30000, 128, 8191), (1000, 129, 140001)])
def test_pieces(M, K, V):
    cut = pieces(M, V)
    assert len(cut) > 1 and cut[-1] != cut[0]
    assert K > 128 or M > 65536 or V < 8192
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    x = torch.randn(M, K, generator=g, device="cuda").to(BF16)
    W = (torch.randn(V, K, generator=g, device="cuda") * 1.5 * K ** -0.5).to(BF16)
    b = torch.randn(V, generator=g, device="cuda")
    target = torch.randint(0, V, (M,), generator=g, device="cuda")
    target[torch.rand(M, generator=g, device="cuda") < 0.2] = -1
    target[:8] = torch.tensor([0, cut[0] - 1, cut[0], cut[0] + 1, V - cut[-1] - 1, V - cut[-1], V - 1, -1], device="cuda")
    dloss = 0.5 + torch.rand(M, generator=g, device="cuda")
    layer = B.DenseLayer(W, b)
    ws = B.SoftmaxXentWorkspace(layer, M, backward=True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    B.ctr_softmax_xent_fwd(layer, x, target, loss, lse, ws, status=status)
    ref = R.xent(x, W, b, target, dloss)
    there = target >= 0
    R.assert_within(loss, ref["loss"], "loss")
    R.assert_within(lse[there], (ref["lse"][0][there], ref["lse"][1][there]), "lse")
    all_of_them = None
    for names in (("dx", "dW", "db"), ("dx",), ("dW",), ("db",)):
        ws.buf.fill_(255)
        new = dict(dx=torch.full_like(x, float("nan")), dW=torch.full_like(W, float("nan")), db=torch.full_like(b, float("nan")))
        out = {n: new[n] for n in names}
        B.ctr_softmax_xent_bwd(layer, x, target, lse, ws, dloss=dloss, status=status, **out)
        if all_of_them is None:
            all_of_them = out
            for n in names:
                R.assert_within(out[n], ref[n], n)
        for n in names:
            assert torch.equal(out[n], all_of_them[n]), n
    assert int(status.item()) == 0
