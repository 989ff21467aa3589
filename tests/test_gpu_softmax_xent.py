"""The softmax cross entropy against a catalogue and its gradients, against
64-bit evaluations (tests/sequence_ref.py has the bounds), through the C ABI."""
import pytest
import torch

import sequence_ref as R
from recsys_sparse_embedding_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")
# 2-norm errors: two roundings to bf16 (dz and the output), each 2^-8 / sqrt 3 in the mean; fp32:
# the exponents' and logits' roundings, a few 2^-23 of |z| + |lse| (up to 16 here)
NORM = {BF16: 3.4e-3, F32: 1e-5}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def case(seed, dtype, M, K, V, bias=True, out=0.2):
    g = gen(seed)
    c = {"x": rnd(g, M, K).to(dtype), "W": rnd(g, V, K, std=1.5 * K ** -0.5).to(dtype), "b": rnd(g, V) if bias else None}
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    c["target"] = torch.where(torch.rand(M, generator=g, device="cuda") < out, torch.full_like(t, -1), t)
    c["dloss"] = 0.5 + torch.rand(M, generator=g, device="cuda")
    return c


def run(c, want=("dx", "dW", "db"), ws=None, dloss=True, x=None):
    """All outputs of both calls (NaN beforehand; the workspace's bytes 255)."""
    x = c["x"] if x is None else x
    M, K = x.shape
    V = c["W"].shape[0]
    layer = B.DenseLayer(c["W"], c["b"])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = lambda dt, *s: torch.full(s, NAN, device="cuda").to(dt)  # noqa: E731
    o = {"loss": new(F32, M), "lse": new(F32, M)}
    ws = ws or B.SoftmaxXentWorkspace(layer, M, backward=bool(want))
    ws.buf.fill_(255)
    B.ctr_softmax_xent_fwd(layer, x, c["target"], o["loss"], o["lse"], ws, status=status)
    if want:
        g = {"dx": new(x.dtype, M, K), "dW": new(x.dtype, V, K), "db": new(F32, V)}
        g = {k: g[k] for k in want}
        ws.buf.fill_(255)
        B.ctr_softmax_xent_bwd(layer, x, c["target"], o["lse"], ws, dloss=c["dloss"] if dloss else None, status=status, **g)
        o.update(g)
    return o, int(status.item())


def check(c, o, ones=False, norm=True):
    ref = R.xent(c["x"], c["W"], c["b"], c["target"], torch.ones_like(c["dloss"]) if ones else c["dloss"])
    live = torch.isfinite(ref["lse"][0]) & (c["target"] >= 0)
    for k in o:
        v, t = ref[k]
        if k == "lse":  # (a row left out has its own x, which the reference drops)
            R.assert_within(o[k][live], (v[live], t[live]), k)
            continue
        R.assert_within(o[k], ref[k], k)
        if norm and k in ("dx", "dW", "db") and min(o[k].shape) >= 48 and min(c["x"].shape) >= 48:
            n, e = float(v.norm()), float((o[k].double() - v).norm())
            assert e <= NORM[F32 if k == "db" else c["x"].dtype] * n, k


SIZES = [(1, 1, 1), (1, 8, 5), (3, 256, 70000), (4, 16, 9001), (2, 128, 1), (4, 72, 130), (5, 64, 9001), (1, 64, 1000), (2, 16, 2), (3, 48, 5), (8, 176, 300), (9, 64, 129), (40, 16, 257), (64, 1024, 3001),
         (127, 8, 33), (128, 64, 128), (129, 100, 1031), (257, 37, 4099), (300, 256, 2000), (513, 520, 777),
         (1000, 64, 12961), (2049, 48, 513), (100, 2050, 300), (31, 200, 40001)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,K,V", SIZES)
def test_xent(dtype, M, K, V):
    for bias in (True, False):
        c = case(M + V, dtype, M, K, V, bias)
        o, status = run(c)
        assert status == 0
        check(c, o)
    o, _ = run(c, dloss=False)
    check(c, o, ones=True)


@pytest.mark.parametrize("dtype,M,K,V", [(BF16, 8192, 64, 40000), (BF16, 5000, 40, 30011), (BF16, 600, 64, 300001),
                                         (F32, 2000, 32, 40000), (F32, 3001, 100, 17000)])
def test_a_catalogue_in_pieces(dtype, M, K, V):
    c = case(1, dtype, M, K, V)
    o, status = run(c)
    assert status == 0
    check(c, o)


@pytest.mark.parametrize("M,K,V", [(1024, 64, 98304), (513, 16, 200001), (4097, 100, 25011), (120, 8, 840001),
                                   (2000, 33, 60000), (65536, 24, 1600), (9000, 128, 12007)])
def test_narrow_rows_in_one_pass(M, K, V):
    """bf16 of at most 128 columns, 10^8 logits: dx and dW without dz in memory."""
    for bias in (True, False):
        c = case(M + K, BF16, M, K, V, bias)
        o, status = run(c)
        assert status == 0
        check(c, o)
    c["target"].random_(0, 3)  # every target in three columns, and every row's
    o, status = run(c)
    assert status == 0
    check(c, o)
    for want in (("dx",), ("dW",), ("db",)):
        p, _ = run(c, want=want)
        assert torch.equal(p[want[0]], o[want[0]]), want


@pytest.mark.parametrize("K", [48, 128])
def test_rows_left_out_and_items_taken_out_in_one_pass(K):
    c = case(15, BF16, 900, K, 120000, out=0.5)
    gone = torch.rand(120000, generator=gen(16), device="cuda") < 0.3
    gone[:600] = True
    c["b"] = torch.where(gone, torch.full_like(c["b"], -INF), c["b"])
    c["target"] = torch.where(c["target"] < 0, c["target"], torch.nonzero(~gone)[:, 0][c["target"] % int((~gone).sum())])
    o, status = run(c)
    assert status == 0
    check(c, o)
    bad = dict(c, x=c["x"].clone())
    bad["x"][c["target"] < 0] = NAN
    p, _ = run(bad)
    for k in ("loss", "dx", "dW", "db"):
        assert torch.equal(o[k], p[k]), k
    assert (p["dx"][c["target"] < 0] == 0).all() and (p["dW"][gone] == 0).all() and (p["db"][gone] == 0).all()
    bad["x"][5] = NAN
    bad["target"][5] = 8000
    p, _ = run(bad)
    keep = torch.arange(900, device="cuda") != 5
    assert torch.equal(o["dx"][keep], p["dx"][keep]) and torch.isnan(p["dx"][5].float()).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_more_rows_than_a_block_of_them(dtype):
    c = case(2, dtype, 70001, 16, 300)
    o, status = run(c)
    assert status == 0
    check(c, o)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,K,V", [(5, 64, 700), (300, 64, 2000), (260, 33, 517)])
def test_rows_left_out(dtype, M, K, V):
    """Their x may hold anything; all of them may be left out; ids out of range."""
    c = case(3, dtype, M, K, V, out=0.5)
    c["target"][0] = 1
    o, _ = run(c)
    bad = dict(c, x=c["x"].clone())
    bad["x"][c["target"] < 0] = NAN
    bad["x"][-1] = INF
    bad["target"] = c["target"].clone()
    bad["target"][-1] = -1
    c["target"][-1] = -1
    o, _ = run(c)
    p, status = run(bad)
    assert status == 0
    for k in ("loss", "dx", "dW", "db"):
        assert torch.equal(o[k], p[k]), k
    assert (p["loss"][c["target"] < 0] == 0).all() and (p["dx"][c["target"] < 0] == 0).all()
    far = dict(bad, target=torch.where(c["target"] < 0, torch.full_like(c["target"], V), c["target"]))
    p, status = run(far)
    assert status == B.FLAG_ID_RANGE
    for k in ("loss", "dx", "dW", "db"):
        assert torch.equal(o[k], p[k]), k
    for none in (-1, -7, V + 5, 2 ** 40, -2 ** 62):
        p, status = run(dict(bad, target=torch.full_like(c["target"], none)))
        assert status == (0 if none == -1 else B.FLAG_ID_RANGE)
        for k in ("loss", "dx", "dW", "db"):
            assert (p[k] == 0).all(), k


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [4, 200])
def test_items_taken_out(dtype, M):
    c = case(4, dtype, M, 64, 900, out=0.0)
    gone = torch.rand(900, generator=gen(5), device="cuda") < 0.5
    gone[:300] = True  # whole tiles
    c["b"] = torch.where(gone, torch.full_like(c["b"], -INF), c["b"])
    c["target"] = torch.nonzero(~gone)[:, 0][c["target"] % int((~gone).sum())]
    o, _ = run(c)
    check(c, o)
    assert (o["db"][gone] == 0).all() and (o["dW"][gone] == 0).all()
    hit = dict(c, target=c["target"].clone())
    hit["target"][0] = 7  # a target that is not possible
    p, _ = run(hit)
    assert float(p["loss"][0]) == INF and torch.isfinite(p["loss"][1:]).all() and torch.isfinite(p["dW"].float()).all()
    none = dict(c, b=torch.full_like(c["b"], -INF))
    p, _ = run(none)
    assert (p["lse"] == -INF).all() and torch.isnan(p["loss"]).all()
    for k in ("dx", "dW", "db"):
        assert (p[k] == 0).all(), k


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_and_non_finite_logits(dtype):
    """Logits far from zero and of one value; NaN and infinities in one row.
    (Near 5000 a logit's own rounding is 2^-24 5000 = 3e-4 of each exponential,
    and at -20000 that of lse, an fp32 number, is 1.2e-3: the elementwise bounds count it, the norms are those of |z| + |lse| up to 16.)"""
    c = case(6, dtype, 150, 64, 1000, out=0.0)
    c["b"] = c["b"] * 1e-3 + 5000.0
    o, _ = run(c)
    check(c, o, norm=False)
    c["b"] = torch.full_like(c["b"], -20000.0)
    c["x"].zero_()
    o, _ = run(c)
    check(c, o, norm=False)
    c = case(7, dtype, 150, 64, 1000, out=0.0)
    o, _ = run(c)
    bad = dict(c, x=c["x"].clone())
    bad["x"][3] = NAN
    p, _ = run(bad)
    keep = torch.arange(150, device="cuda") != 3
    for k in ("loss", "lse", "dx"):
        assert torch.equal(o[k][keep], p[k][keep]) and torch.isnan(p[k][3].float()).all(), k
    up = dict(c, b=c["b"].clone())
    up["b"][500] = INF
    p, _ = run(up, want=())
    assert (p["lse"] == INF).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_each_gradient_alone_and_strided_rows(dtype):
    c = case(8, dtype, 333, 72, 1500)
    o, _ = run(c)
    for want in (("dx",), ("dW",), ("db",), ("dx", "db")):
        p, _ = run(c, want=want)
        ref = R.xent(c["x"], c["W"], c["b"], c["target"], c["dloss"])
        for k in want:
            R.assert_within(p[k], ref[k], k)
    for extra in (8, 24):
        buf = torch.full((333, 72 + extra), NAN, device="cuda").to(dtype)
        buf[:, :72] = c["x"]
        p, _ = run(c, x=buf[:, :72])
        for k in o:
            assert torch.equal(o[k], p[k]), k
    dxw = torch.full((333, 80), NAN, device="cuda").to(dtype)
    layer = B.DenseLayer(c["W"], c["b"])
    ws = B.SoftmaxXentWorkspace(layer, 333, backward=True)
    B.ctr_softmax_xent_bwd(layer, c["x"], c["target"], o["lse"], ws, dloss=c["dloss"], dx=dxw[:, :72])
    R.assert_within(dxw[:, :72], R.xent(c["x"], c["W"], c["b"], c["target"], c["dloss"])["dx"], "dx in wider rows")
    assert torch.isnan(dxw[:, 72:].float()).all()


def test_the_catalogue_as_columns_of_a_wider_table():
    g = gen(9)
    table = torch.full((700, 96), NAN, device="cuda").to(BF16)
    table[:, :64] = rnd(g, 700, 64, std=0.2).to(BF16)
    c = case(9, BF16, 140, 64, 700)
    near = dict(c, W=table[:, :64].contiguous())
    o, _ = run(near)
    p, _ = run(dict(c, W=table[:, :64]))
    for k in o:
        assert torch.equal(o[k], p[k]), k


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_rows(dtype):
    c = case(10, dtype, 0, 64, 100)
    o, status = run(c)
    assert status == 0 and (o["dW"] == 0).all() and (o["db"] == 0).all()


@pytest.mark.parametrize("dtype,M,V", [(BF16, 700, 3000), (F32, 2000, 30000)])
def test_equal_calls_a_larger_workspace_streams_and_graphs(dtype, M, V):
    c = case(11, dtype, M, 64, V)
    o, _ = run(c)
    layer = B.DenseLayer(c["W"], c["b"])
    ws = B.SoftmaxXentWorkspace(layer, 2 * M + 1, backward=True)
    p, _ = run(c, ws=ws)
    for k in o:
        assert torch.equal(o[k], p[k]), k
    outs = [{k: torch.full_like(t, NAN) for k, t in o.items()} for _ in range(2)]

    def both(p):
        B.ctr_softmax_xent_fwd(layer, c["x"], c["target"], p["loss"], p["lse"], ws)
        B.ctr_softmax_xent_bwd(layer, c["x"], c["target"], p["lse"], ws, dloss=c["dloss"], dx=p["dx"], dW=p["dW"], db=p["db"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(outs[0])
    side.synchronize()
    for k in o:
        assert torch.equal(o[k], outs[0][k]), k
    graphs = []
    for p in outs:
        gph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gph):
            both(p)
        graphs.append(gph)
    for _ in range(2):
        for p in outs:
            for t in p.values():
                t.fill_(NAN)
        for gph in graphs:
            gph.replay()
        torch.cuda.synchronize()
        for p in outs:
            for k in o:
                assert torch.equal(o[k], p[k]), k


def test_gradients_against_differences():
    """(f(v + d) - f(v - d)) / 2 along random directions, f = <loss, dloss> in 64
    bits from the kernel's fp32 losses. With n directions' signs a logit moves by
    at most s = step * sum of |W| or |x| over K; the third derivative of a loss
    along it is at most (s / step)^3, so the quotient is off by step^2 / 6 of
    that per row; each loss is rounded by 2^-21 of |lse| + |z| (below 16)."""
    c = case(12, F32, 60, 24, 150)
    o, _ = run(c)
    step, g = 2.0 ** -7, gen(13)

    def f(w):
        p, _ = run(w, want=())
        return float((p["loss"].double() * c["dloss"].double()).sum())

    for name, grad in (("x", "dx"), ("W", "dW"), ("b", "db")):
        d = torch.sign(rnd(g, *c[name].shape))
        # (directions of size 1 / K keep a logit's move near its own size)
        d = d / 8
        slope = (f(dict(c, **{name: c[name] + step * d})) - f(dict(c, **{name: c[name] - step * d}))) / (2 * step)
        want = float((o[grad].double() * d.double()).sum())
        move = 1.0 / 8 if name == "b" else float((c["W"] if name == "x" else c["x"]).abs().sum(1).max()) / 8
        bound = 60 * 1.5 * (step ** 2 / 6 * move ** 3 * 6 + 2.0 ** -21 * 16 / step)
        assert abs(slope - want) <= bound, name


def test_refusals():
    c = case(14, F32, 12, 8, 40)
    layer = B.DenseLayer(c["W"], c["b"])
    ws = B.SoftmaxXentWorkspace(layer, 12, backward=True)
    loss, lse = torch.empty(12, device="cuda"), torch.empty(12, device="cuda")
    ok = dict(layer=layer, x=c["x"], target=c["target"], loss=loss, lse=lse, workspace=ws)
    B.ctr_softmax_xent_fwd(**ok)
    for kw in (dict(x=c["x"].to(BF16)), dict(x=c["x"][:, :7]), dict(target=c["target"].int()), dict(target=c["target"][:11]),
               dict(loss=loss[:11]), dict(lse=lse.double()), dict(target=c["target"].cpu())):
        with pytest.raises(ValueError):
            B.ctr_softmax_xent_fwd(**{**ok, **kw})
    for kw in (dict(dx=c["x"].to(BF16)), dict(dW=c["W"][:39]), dict(db=loss), dict(dloss=loss.double()),
               dict(dW=torch.empty(40, 16, device="cuda")[:, :8])):
        with pytest.raises(ValueError):
            B.ctr_softmax_xent_bwd(layer, c["x"], c["target"], lse, ws, **kw)
    with pytest.raises(B.DsfError):
        B.ctr_softmax_xent_fwd(**{**ok, "workspace": B.SoftmaxXentWorkspace(B.DenseLayer(c["W"][:1]), 1)})
    with pytest.raises(B.DsfError):
        B.SoftmaxXentWorkspace(B.DenseLayer(c["W"], act=B.DSF_ACT_SILU), 4)
