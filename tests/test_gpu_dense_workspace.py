"""Nothing changes behind a layer's workspace of exactly the stated size."""
import pytest
import torch

import dense_ref as R
from dense_guard import guard
from recsys_sparse_embedding_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (9, 64, 300), (33, 45, 77), (300, 1000, 96), (2049, 256, 512), (70, 2100, 1030),
                                   (640, 2048, 264), (4097, 160, 129), (20000, 96, 72), (100, 4096, 4096)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_nothing_is_written_behind_a_layers_workspace(M, K, N, dtype, gated, act):
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    rows = 2 * N if gated else N
    W = (torch.randn(rows, K, generator=g, device="cuda") * K ** -0.5).to(dtype)
    layer = B.DenseLayer(W, torch.randn(rows, generator=g, device="cuda"), act=R.ACTS[act])
    x = torch.randn(M, K, generator=g, device="cuda").to(dtype)
    dy = torch.randn(M, N, generator=g, device="cuda").to(dtype)
    y = torch.empty_like(dy)
    out = dict(dx=torch.empty_like(x), dW=torch.empty_like(W), db=torch.empty(rows, device="cuda"))
    ws = B.DenseWorkspace(layer, M, gated=gated)
    intact = guard(ws)
    (B.ctr_glu_fwd if gated else B.ctr_dense_fwd)(layer, x, y, ws)
    assert intact()
    ws = B.DenseWorkspace(layer, M, gated=gated, backward=True)
    bwd = B.ctr_glu_bwd if gated else B.ctr_dense_bwd
    for names in (("dx", "dW", "db"), ("dx",), ("dW",), ("db",)):
        intact = guard(ws)
        bwd(layer, x, dy, ws, **{n: out[n] for n in names})
        assert intact(), names
