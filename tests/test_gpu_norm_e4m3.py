"""The norm's 8-bit output, byte for byte."""
import pytest
import torch

from recsys_sparse_embedding_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("M,N", [(4000, 1000), (600, 4096), (3000, 33), (70, 16384), (5, 1)])
def test_8_bit_values_are_the_rounded_quotients(xt, M, N, weighted):
    """The e4m3 output against the fp32 output of the same call: scale = max|y|
    / 448, values y / scale, each rounded once (no tolerance)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    x = (torch.randn(M, N, generator=g, device="cuda") * torch.exp(torch.randn(M, 1, generator=g, device="cuda"))).to(xt)
    w = 1 + 0.3 * torch.randn(N, generator=g, device="cuda") if weighted else None
    y, q, scale = torch.empty(M, N, device="cuda"), torch.empty(M, N, dtype=E4M3, device="cuda"), torch.empty(M, device="cuda")
    B.ctr_rms_norm_fwd(x, y, weight=w)
    B.ctr_rms_norm_fwd(x, q, weight=w, y_scale=scale)
    top = y.abs().amax(1)
    assert torch.equal(scale, (top / torch.full_like(top, 448.0)).clamp_min(2.0 ** -126))
    want = (y / scale[:, None]).to(E4M3)
    bad = (q.view(torch.uint8) != want.view(torch.uint8)).sum()
    assert int(bad) == 0, "%d of %d values" % (int(bad), M * N)
