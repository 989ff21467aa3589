"""The sequence-tower operators captured, replayed on changed inputs, and run on
another stream, in each of their forms: what a replay gives is what a call on the
same inputs gives, bit by bit."""
import pytest
import torch

from recsys_sparse_embedding_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def rnd(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda") * std


def held(fill, call, outs):
    """fill(seed) puts inputs in place, call() makes outs of them. Eager results of
    two inputs, then the same by a graph of one capture and by another stream."""
    def results(run, seed):
        fill(seed)
        for t in outs:
            t.fill_(7.0)
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        return [t.clone() for t in outs]

    want = [results(call, s) for s in (1, 2)]
    fill(3)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    side = torch.cuda.Stream()

    def on_side():
        with torch.cuda.stream(side):
            call()

    for run in (graph.replay, on_side, graph.replay):
        for s, w in zip((1, 2), want):
            for a, b in zip(results(run, s), w):
                assert torch.equal(a, b)
    assert any(not torch.equal(a, b) for a, b in zip(*want))


def jagged(seed, nb, T):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    cuts = torch.randint(0, T + 1, (nb - 1,), generator=g, device="cuda").sort().values
    ends = torch.cat([cuts, torch.tensor([T], device="cuda")])
    return torch.diff(ends, prepend=ends.new_zeros(1)).to(torch.int32)


# (400,000 rows of 2 sequences: marks cleared by a launch of their own; 70,001 sequences: sums of lengths first)
@pytest.mark.parametrize("nb,T,D,equal", [(2, 400000, 64, False), (70001, 60000, 16, False), (300, 9000, 48, False), (6, 6, 64, True),
                                          (3, 30000, 36, True), (40, 2560, 64, True), (5, 0, 32, False)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan(dtype, nb, T, D, equal):
    new = lambda *s, t=dtype: torch.empty(*s, device="cuda", dtype=t)  # noqa: E731
    xg, dh, h0, dl = new(T, 2 * D), new(T, D), new(nb, D, t=F32), new(nb, D, t=F32)
    lengths = None if equal else torch.zeros(nb, dtype=torch.int32, device="cuda")
    h, dxg, hl, d0 = new(T, D), new(T, 2 * D), new(nb, D, t=F32), new(nb, D, t=F32)
    ws = B.GatedScanWorkspace(T, nb, D)

    def fill(seed):
        for k, t in enumerate((xg, dh, h0, dl)):
            t.copy_(rnd(10 * seed + k, *t.shape))
        if not equal:
            lengths.copy_(jagged(seed, nb, T))

    def call():
        B.ctr_gated_scan_fwd(xg[:, :D], xg[:, D:], h, nb, ws, lengths=lengths, h0=h0, h_last=hl)
        B.ctr_gated_scan_bwd(dh, xg[:, :D], xg[:, D:], h, dxg[:, :D], dxg[:, D:], nb, ws, lengths=lengths, h0=h0, dh_last=dl, dh0=d0)

    held(fill, call, [h, dxg, hl, d0])


@pytest.mark.parametrize("dtype,M,K,V", [(BF16, 1, 64, 9001), (F32, 3, 16, 9001), (BF16, 2, 60, 777), (BF16, 900, 64, 120000), (BF16, 70, 100, 800001),
                                         (BF16, 300, 200, 5000), (F32, 500, 176, 12961), (F32, 3000, 48, 20001), (BF16, 9000, 136, 17003)])
def test_cross_entropy(dtype, M, K, V):
    new = lambda *s, t=dtype: torch.empty(*s, device="cuda", dtype=t)  # noqa: E731
    x, W, b, g = new(M, K), new(V, K), new(V, t=F32), new(M, t=F32)
    target = torch.zeros(M, dtype=torch.int64, device="cuda")
    loss, lse, dx, dW, db = new(M, t=F32), new(M, t=F32), new(M, K), new(V, K), new(V, t=F32)
    layer = B.DenseLayer(W, b)
    ws = B.SoftmaxXentWorkspace(layer, M, backward=True)

    def fill(seed):
        x.copy_(rnd(10 * seed, M, K))
        W.copy_(rnd(10 * seed + 1, V, K, std=1.5 * K ** -0.5))
        b.copy_(rnd(10 * seed + 2, V))
        g.copy_(1 + rnd(10 * seed + 3, M).abs())
        target.copy_((rnd(10 * seed + 4, M).abs() * V).long() % V)

    def call():
        B.ctr_softmax_xent_fwd(layer, x, target, loss, lse, ws)
        B.ctr_softmax_xent_bwd(layer, x, target, lse, ws, dloss=g, dx=dx, dW=dW, db=db)

    held(fill, call, [loss, lse, dx, dW, db])


@pytest.mark.parametrize("r,c", [(1, 1), (64, 64), (1366, 256), (1030, 1300), (300000, 24)])
@pytest.mark.parametrize("wt", [F32, BF16])
def test_update(wt, r, c):
    W0, m0 = rnd(1, r, c, std=0.05).to(wt), rnd(2, r, c, std=1e-3)
    grad, W, m = torch.empty(r, c, device="cuda", dtype=wt), torch.empty_like(W0), torch.empty_like(m0)
    ws = B.MuonWorkspace(W0)

    def call():  # (W and momentum are updated in place)
        W.copy_(W0)
        m.copy_(m0)
        B.ctr_muon_update(W, grad, m, ws, weight_decay=0.1)

    held(lambda seed: grad.copy_(rnd(seed, r, c, std=1e-3)), call, [W, m])


@pytest.mark.parametrize("r,c", [(40, 90), (90, 40), (1030, 1100), (70001, 24)])
@pytest.mark.parametrize("wt", [F32, BF16])
@pytest.mark.parametrize("steps", [1, 5])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_a_gradient_that_is_not_finite_reaches_all_of_the_matrix(r, c, wt, steps, value):
    W, m, grad = rnd(3, r, c).to(wt), rnd(4, r, c), rnd(5, r, c)
    grad[r // 2, c // 3] = value
    before = m.clone()
    B.ctr_muon_update(W, grad, m, B.MuonWorkspace(W), steps=steps)
    assert torch.isnan(W.float()).all()
    there = torch.ones_like(m, dtype=torch.bool)
    there[r // 2, c // 3] = False
    assert torch.isfinite(m[there]).all() and not torch.isfinite(m[~there]).any() and torch.isfinite(before).all()
