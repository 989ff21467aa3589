"""The gated scan over long sequences with gates that are nearly or fully closed:
what is kept of the state per row, 1 - sigmoid(gate), errs alike in row after row
where the gate is constant, so its roundings add up instead of averaging out.

Bounds. 1 - z, z below 1/2, is one rounding (2^-25, half a step below 1; z itself
errs by (8 + 2 |g|) 2^-23 of its size, tests/sequence_ref.py) and each row's
product another (2^-24 at most): T times their sum of the state. Where z T is
below 2^-25, what is kept is 1 exactly, and the state as it was. It never grows:
a factor of at most 1 gives a product of at most what it multiplies."""
import pytest
import torch

from recsys_sparse_embedding_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def run(gate, lengths, nb, h0, dh_last):
    T, D = gate.shape
    x = torch.zeros_like(gate)
    h, dx, dgate = torch.empty_like(gate), torch.empty_like(gate), torch.empty_like(gate)
    hl, d0 = torch.empty_like(h0), torch.empty_like(h0)
    ws = B.GatedScanWorkspace(T, nb, D)
    B.ctr_gated_scan_fwd(x, gate, h, nb, ws, lengths=lengths, h0=h0, h_last=hl)
    B.ctr_gated_scan_bwd(x, x, gate, h, dx, dgate, nb, ws, lengths=lengths, h0=h0, dh_last=dh_last, dh0=d0)
    return h, hl, d0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lengths,equal", [([131072], False), ([60001, 1, 0, 70000], False), ([65536, 65536], True)])
def test_a_constant_gate(dtype, lengths, equal):
    D, T, nb = 1024, sum(lengths), len(lengths)
    g = torch.linspace(-80, -2, D, device="cuda").to(dtype)
    gate = g.expand(T, D).contiguous()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    h0 = 0.5 + torch.rand(nb, D, generator=gen, device="cuda")
    dl = 0.5 + torch.rand(nb, D, generator=gen, device="cuda")
    n = None if equal else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    h, hl, d0 = run(gate, n, nb, h0, dl)
    closed = g < -30
    assert torch.equal(hl[:, closed], h0[:, closed]) and torch.equal(d0[:, closed], dl[:, closed])
    assert (hl <= h0).all() and (d0 <= dl).all()
    z = torch.sigmoid(g.double())
    keep = torch.sigmoid(-g.double())
    for s, L in enumerate(lengths):
        per_row = 2.0 ** -25 + 2.0 ** -24 + z / keep * (8 + 2 * g.double().abs()) * 2.0 ** -23
        for got, first in ((hl, h0), (d0, dl)):
            want = keep ** L * first[s].double()
            assert ((got[s].double() - want).abs() <= 1.01 * L * per_row * want + 1e-38).all(), s
    assert (h[:lengths[0]].float() <= h0[:1].to(dtype).float()).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_steps_of_serving(dtype):
    """The same state through single steps."""
    D = 256
    g = torch.linspace(-80, -18, D, device="cuda").to(dtype)[None]
    x, h = torch.zeros_like(g), torch.empty_like(g)
    state = torch.linspace(0.5, 1.5, D, device="cuda")[None].contiguous()
    first, ws = state.clone(), B.GatedScanWorkspace(1, 1, D)
    for _ in range(200):
        nxt = torch.empty_like(state)
        B.ctr_gated_scan_fwd(x, g, h, 1, ws, h0=state, h_last=nxt)
        state = nxt
    assert torch.equal(state, first)
