"""The orthogonalised update against a 64-bit evaluation, through the C ABI.

Bounds. The update's 2-norm error: each product of fp32 operands is off by a few
2^-24 of its terms' norms; a step's polynomial has slope at most a = 3.44 on
singular values and on errors, so the errors of five steps add up to at most
3.44 + ... + 3.44^5 < 700 times 8 2^-24 (its three products and roundings) of the
starting norm 1, against an update of norm near sqrt(n) (rank n), or near sqrt(r)
for a gradient of rank r: 700 * 8 * 2^-24 = 3.4e-4 of sqrt(n or r). (For a bf16 W,
X has 17 bits: at most 5e-5 of its norm off where it was measured, so the bound is
kept.) W is then rounded: half a step of its value. Momentum: two roundings."""
import pytest
import torch

import sequence_ref as R
from recsys_sparse_embedding_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def case(seed, wt, gt, r, c, rank=None):
    g = gen(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    grad = rnd(r, c) if rank is None else rnd(r, rank) @ rnd(rank, c)
    return {"W": (rnd(r, c) * 0.05).to(wt), "grad": (1e-3 * grad).to(gt), "momentum": 3e-3 * rnd(r, c)}


def step(c, ws=None, W=None, grad=None, **kw):
    W = c["W"].clone() if W is None else W
    m = c["momentum"].clone()
    ws = ws or B.MuonWorkspace(W)
    ws.buf.fill_(255)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.ctr_muon_update(W, c["grad"] if grad is None else grad, m, ws, status=status, **kw)
    assert int(status.item()) == 0
    return W, m


def check(c, W, m, rank=None, lr=0.02, mu=0.95, weight_decay=0.0, nesterov=True, steps=5):
    w, mr, upd = R.muon(c["W"], c["grad"], c["momentum"], lr, mu, weight_decay, nesterov, steps)
    assert ((m.double() - mr).abs() <= 2 * 2.0 ** -24 * (mr.abs() + c["momentum"].double().abs()) + 1e-38).all()
    half = R.HALF[c["W"].dtype]
    r, n = w.shape
    full = lr * max(1.0, r / n) ** 0.5 * 3.4e-4 * min(r, n, rank or 1 << 30) ** 0.5
    err = float((W.double() - w).norm())
    assert err <= full + float((half * w.abs() + 4 * 2.0 ** -24 * (upd.abs() + c["W"].double().abs())).norm()), err


SHAPES = [(1, 1), (1, 40), (40, 1), (3, 5), (16, 16), (64, 176), (176, 64), (33, 257), (300, 100), (256, 512), (512, 256),
          (1366, 256), (129, 1000), (640, 640), (1024, 2048), (4096, 72), (40, 30000), (70001, 24)]


@pytest.mark.parametrize("r,c", SHAPES)
@pytest.mark.parametrize("wt,gt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
def test_muon(r, c, wt, gt):
    d = case(r + c, wt, gt, r, c)
    W, m = step(d)
    check(d, W, m)


@pytest.mark.parametrize("r,c", [(1024, 1024), (1025, 1101), (1030, 4098), (5000, 1027), (1153, 1409), (2300, 2310), (40001, 1030)])
@pytest.mark.parametrize("wt", [F32, BF16])
def test_symmetric_products_by_half_of_their_tiles(r, c, wt):
    d = case(r * 3 + c, wt, F32, r, c)
    W, m = step(d)
    check(d, W, m)
    V, n = step(d)
    assert torch.equal(W, V) and torch.equal(m, n)


@pytest.mark.parametrize("kw", [dict(nesterov=False), dict(steps=1), dict(steps=9), dict(mu=0.0), dict(lr=0.5, weight_decay=0.1),
                                dict(lr=0.0)], ids=str)
@pytest.mark.parametrize("r,c", [(200, 96), (96, 200)])
def test_arguments(r, c, kw):
    d = case(5, F32, F32, r, c)
    W, m = step(d, **kw)
    if kw.get("steps", 5) <= 5:
        check(d, W, m, **kw)
    if kw.get("lr") == 0.0:
        assert torch.equal(W, d["W"])


def test_the_update_is_near_orthogonal():
    """Five steps send singular values of 0.003 .. 1 (of the norm) to 0.65 .. 1.25."""
    d = case(6, F32, F32, 192, 480)
    d["W"].zero_()
    W, _ = step(d, lr=1.0)
    s = torch.linalg.svdvals(W.double())
    assert float(s.min()) > 0.65 and float(s.max()) < 1.25
    v = case(6, F32, F32, 480, 192)
    v["grad"], v["momentum"], v["W"] = d["grad"].t().contiguous(), d["momentum"].t().contiguous(), d["W"].t().contiguous()
    W2, _ = step(v, lr=1.0)
    assert float((W2.t() - W * (480 / 192) ** 0.5).norm() / W2.norm()) < 1e-4


@pytest.mark.parametrize("rank", [1, 4])
def test_gradients_of_low_rank(rank):
    d = case(7, F32, F32, 256, 300, rank)
    d["momentum"].zero_()
    W, m = step(d)
    check(d, W, m, rank)


def test_zero_and_tiny_and_large_gradients():
    d = case(8, F32, F32, 100, 60)
    d["grad"].zero_()
    d["momentum"].zero_()
    W, m = step(d, weight_decay=0.5)
    assert torch.equal(m, d["momentum"]) and ((W - d["W"] * 0.99).abs() <= 2.0 ** -22 * d["W"].abs()).all()
    for scale in (1e-30, 1e-6, 1e15):
        d = case(9, F32, F32, 100, 60)
        d["grad"] *= scale
        d["momentum"] *= scale
        W, m = step(d)
        check(d, W, m)
    d["grad"][3, 4] = float("nan")
    W, m = step(d)
    assert torch.isnan(W).all() and int(torch.isnan(m).sum()) == 1


def test_strided_matrices():
    d = case(10, F32, BF16, 130, 90)
    W0, m0 = step(d)
    for extra, off in ((6, 0), (7, 3), (30, 1)):
        buf = torch.full((130, 90 + extra + off), 7.0, device="cuda")
        gbuf = torch.full((130, 90 + extra + off), 7.0, device="cuda").to(BF16)
        W, grad = buf[:, off:off + 90], gbuf[:, off:off + 90]
        W.copy_(d["W"])
        grad.copy_(d["grad"])
        _, m = step(d, W=W, grad=grad)
        assert torch.equal(W, W0) and torch.equal(m, m0)
        buf[:, off:off + 90] = 7.0
        assert (buf == 7.0).all()


def test_equal_steps_streams_and_graphs():
    d = case(11, F32, F32, 512, 384)
    W0, m0 = step(d)
    ws = B.MuonWorkspace(d["W"])
    side = torch.cuda.Stream()
    W, m = d["W"].clone(), d["momentum"].clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        B.ctr_muon_update(W, d["grad"], m, ws)
    side.synchronize()
    assert torch.equal(W, W0) and torch.equal(m, m0)
    ms = [(torch.empty_like(W), torch.empty_like(m)) for _ in range(2)]
    graphs = []
    for w, q in ms:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.ctr_muon_update(w, d["grad"], q, ws)
        graphs.append(g)
    for _ in range(2):
        for w, q in ms:
            w.copy_(d["W"])
            q.copy_(d["momentum"])
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for w, q in ms:
            assert torch.equal(w, W0) and torch.equal(q, m0)


def test_refusals():
    d = case(12, F32, F32, 20, 30)
    ws = B.MuonWorkspace(d["W"])
    ok = dict(W=d["W"], grad=d["grad"], momentum=d["momentum"], workspace=ws)
    B.ctr_muon_update(**ok)
    for kw in (dict(W=d["W"].half()), dict(W=d["W"].t()), dict(grad=d["grad"][:19]), dict(grad=d["grad"].double()),
               dict(momentum=d["momentum"].to(BF16)), dict(momentum=d["momentum"].t()), dict(grad=d["grad"].cpu()),
               dict(W=d["W"][0])):
        with pytest.raises(ValueError):
            B.ctr_muon_update(**{**ok, **kw})
    for kw in (dict(mu=1.0), dict(mu=-0.1), dict(lr=float("nan")), dict(weight_decay=-1.0), dict(steps=0), dict(steps=17),
               dict(workspace=B.MuonWorkspace(d["W"][:1]))):
        with pytest.raises(B.DsfError):
            B.ctr_muon_update(**{**ok, **kw})
