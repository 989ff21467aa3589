"""The dense layer, the gated layer and the RMS norm against 64-bit
evaluations (tests/dense_ref.py has the bounds), through the C ABI."""
import math

import pytest
import torch

import dense_ref as R
from recsys_sparse_embedding_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
# 2-norm errors: one rounding to bf16 is off by at most 2^-8, 2^-8 / sqrt 3 = 2.3e-3 in the mean
# over a binade; a gradient has two of them. fp32: sums of random sign, far below (K + 8) 2^-23.
NORM_FWD = {BF16: 2.4e-3, F32: 3e-6}
NORM_BWD = {BF16: 3.4e-3, F32: 3e-6}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def strided(t, extra, offset=0):
    """t's values in rows `extra` elements longer, `offset` elements into the
    buffer; NaN around them (e4m3: 0x7f bytes, its NaN)."""
    rows, cols = t.shape
    buf = torch.full((rows * (cols + extra) + offset + 64,), float("nan"), device=t.device).to(t.dtype)
    v = buf[offset:offset + rows * (cols + extra)].view(rows, cols + extra)[:, :cols]
    v.copy_(t)
    return v, buf


def is_nan(t):
    return torch.isnan(t.float())


def quantise(t):
    s = (t.abs().amax(1) / 448).clamp_min(2.0 ** -126)
    return (t / s[:, None]).to(E4M3), s


def layer_of(g, dtype, rows, K, act, bias=True):
    W = rnd(g, rows, K, std=(2.0 / (K + rows)) ** 0.5 * 2)
    b = rnd(g, rows, std=0.3) if bias else None
    ws = None
    if dtype == E4M3:
        W, ws = quantise(W)
    return B.DenseLayer(W.to(dtype), b, act=R.ACTS[act], scale=ws)


def x_of(g, dtype, M, K):
    x = rnd(g, M, K)
    return quantise(x) if dtype == E4M3 else (x.to(dtype), None)


SIZES = [(1, 1, 1), (1, 256, 512), (2, 16, 8), (3, 37, 5), (8, 1024, 96), (9, 64, 300), (17, 176, 64), (64, 640, 33),
         (127, 64, 129), (128, 128, 128), (129, 200, 257), (256, 512, 256), (300, 1000, 96), (513, 48, 1040),
         (1000, 513, 300), (2049, 256, 512), (385, 2100, 700),
         # past the sizes that a few CUDA cores do: whole, ragged and odd tiles of each configuration
         (129, 520, 600), (257, 1000, 333), (70, 2100, 1030), (2000, 96, 200), (4097, 160, 129), (640, 2048, 264)]
ACT_OF = ["none", "relu", "silu", "gelu"]


@pytest.mark.parametrize("dtype", [BF16, F32, E4M3])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_dense_fwd(dtype, i):
    M, K, N = SIZES[i]
    g = gen(i)
    for act in ACT_OF if M <= 130 else [ACT_OF[i % 4]]:
        for with_res, bias in ((False, True), (True, False)):
            layer = layer_of(g, dtype, N, K, act, bias)
            x, xs = x_of(g, dtype, M, K)
            res = rnd(g, M, N).to(layer.out_dtype) if with_res else None
            ws = B.DenseWorkspace(layer, M)
            y, buf = strided(torch.zeros(M, N, device="cuda").to(layer.out_dtype), 0)
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            B.ctr_dense_fwd(layer, x, y, ws, residual=res, x_scale=xs, status=st)
            ref, tol = R.dense(x, layer.W, layer.bias, act, res, layer.out_dtype, xs, layer.scale)
            assert int(st.item()) == 0
            R.assert_within(y, ref, tol, "y %s" % act)
            R.assert_norm(y, ref, NORM_FWD[layer.out_dtype], "y %s" % act, M, K, N)
            assert is_nan(buf[M * N:]).all(), "written past the end"


@pytest.mark.parametrize("dtype", [BF16, F32, E4M3])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_glu_fwd(dtype, i):
    M, K, F = SIZES[i]
    g = gen(100 + i)
    for act in ACT_OF if M <= 130 else [ACT_OF[i % 4]]:
        layer = layer_of(g, dtype, 2 * F, K, act, act != "relu")
        x, xs = x_of(g, dtype, M, K)
        ws = B.DenseWorkspace(layer, M, gated=True)
        h, buf = strided(torch.zeros(M, F, device="cuda").to(layer.out_dtype), 0)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        B.ctr_glu_fwd(layer, x, h, ws, x_scale=xs, status=st)
        ref, tol = R.glu(x, layer.W, layer.bias, act, layer.out_dtype, xs, layer.scale)
        assert int(st.item()) == 0
        R.assert_within(h, ref, tol, "h %s" % act)
        R.assert_norm(h, ref, NORM_FWD[layer.out_dtype], "h %s" % act, M, K, F)
        assert is_nan(buf[M * F:]).all(), "written past the end"


def run_bwd(layer, x, dy, gated, **out):
    ws = B.DenseWorkspace(layer, x.shape[0], gated=gated, backward=True)
    ws.buf.fill_(0xff)  # (NaN in every type: nothing may be read before it is written)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    (B.ctr_glu_bwd if gated else B.ctr_dense_bwd)(layer, x, dy, ws, status=st, **out)
    assert int(st.item()) == 0
    return out


def check_bwd(layer, x, dy, act, gated, out):
    ref = R.grads(x, layer.W, layer.bias, act, dy, gated)
    for name, t in out.items():
        v, tol = ref[name]
        R.assert_within(t, v, tol, "%s %s" % (name, act))
        if act != "relu":  # (a ReLU's slope may go either way at z near 0)
            R.assert_norm(t, v, 3e-6 if name == "db" else NORM_BWD[x.dtype], "%s %s" % (name, act),
                          *x.shape, dy.shape[1])


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_layer_bwd(dtype, gated, i):
    M, K, N = SIZES[i]
    g = gen(200 + i)
    for act in ACT_OF if M <= 130 else [ACT_OF[i % 4], ACT_OF[(i + 2) % 4]]:
        layer = layer_of(g, dtype, 2 * N if gated else N, K, act, act != "gelu")
        x, _ = x_of(g, dtype, M, K)
        dy = rnd(g, M, N).to(dtype)
        out = run_bwd(layer, x, dy, gated, dx=torch.empty_like(x), dW=torch.empty(layer.R, K, dtype=dtype, device="cuda"),
                      db=torch.empty(layer.R, device="cuda"))
        check_bwd(layer, x, dy, act, gated, out)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layer_bwd_takes_any_of_its_outputs(dtype, gated):
    g = gen(7)
    M, K, N = 200, 96, 136
    layer = layer_of(g, dtype, 2 * N if gated else N, K, "silu")
    x, _ = x_of(g, dtype, M, K)
    dy = rnd(g, M, N).to(dtype)
    new = {"dx": lambda: torch.empty_like(x), "dW": lambda: torch.empty_like(layer.W),
           "db": lambda: torch.empty(layer.R, device="cuda")}
    for names in (("dx",), ("dW",), ("db",), ("dx", "db"), ()):
        out = run_bwd(layer, x, dy, gated, **{n: new[n]() for n in names})
        check_bwd(layer, x, dy, "silu", gated, out)


@pytest.mark.parametrize("dtype", [BF16, F32, E4M3])
@pytest.mark.parametrize("extra,offset", [(16, 0), (16, 16), (3, 1), (1, 0)])
def test_strided_rows(dtype, extra, offset):
    """Rows longer than their matrix, buffers that start off a boundary (where
    the row's own length allows it: K = 45 here), an in-place residual."""
    g = gen(extra * 7 + offset)
    whole = extra % 16 == 0
    M, K, N = 150, 48 if whole else 45, 80 if whole else 77
    layer = layer_of(g, dtype, N, K, "silu")
    x, xs = x_of(g, dtype, M, K)
    x, _ = strided(x, extra, offset)
    res = rnd(g, M, N).to(layer.out_dtype)
    y, buf = strided(res, extra, offset)
    ws = B.DenseWorkspace(layer, M)
    keep = is_nan(buf)
    B.ctr_dense_fwd(layer, x, y, ws, residual=y, x_scale=xs)
    ref, tol = R.dense(x, layer.W, layer.bias, "silu", res, layer.out_dtype, xs, layer.scale)
    R.assert_within(y, ref, tol, "y")
    assert is_nan(buf)[keep].all(), "written between the rows"
    if dtype != E4M3:
        dy, _ = strided(rnd(g, M, N).to(dtype), extra, offset)
        dx, buf = strided(torch.zeros(M, K, device="cuda").to(dtype), extra, offset)
        keep = is_nan(buf)
        out = run_bwd(layer, x, dy, False, dx=dx, dW=torch.empty(N, K, dtype=dtype, device="cuda"),
                      db=torch.empty(N, device="cuda"))
        check_bwd(layer, x, dy, "silu", False, out)
        assert is_nan(buf)[keep].all(), "written between the rows"


def test_weights_with_a_row_stride():
    g = gen(5)
    for dtype in (BF16, F32):
        W, _ = strided(rnd(g, 96, 64, std=0.1).to(dtype), 32)
        layer = B.DenseLayer(W, None, act=B.DSF_ACT_GELU)
        x, _ = x_of(g, dtype, 140, 64)
        dy = rnd(g, 140, 96).to(dtype)
        y = torch.empty(140, 96, dtype=dtype, device="cuda")
        B.ctr_dense_fwd(layer, x, y, B.DenseWorkspace(layer, 140))
        ref, tol = R.dense(x, W, None, "gelu", None, dtype)
        R.assert_within(y, ref, tol, "y")
        out = run_bwd(layer, x, dy, False, dx=torch.empty_like(x), dW=torch.empty(96, 64, dtype=dtype, device="cuda"),
                      db=torch.empty(96, device="cuda"))
        check_bwd(layer, x, dy, "gelu", False, out)


@pytest.mark.parametrize("M", [1, 5, 200])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_non_finite_rows_stay_apart(dtype, bad, M):
    """A row of x with a non-finite value gives non-finite results in its own
    row only; other rows keep their bits."""
    g = gen(M)
    K, N = 192, 130
    layer = layer_of(g, dtype, N, K, "silu")
    x, _ = x_of(g, dtype, M, K)
    ws = B.DenseWorkspace(layer, M)
    clean, dirty = (torch.empty(M, N, dtype=dtype, device="cuda") for _ in range(2))
    B.ctr_dense_fwd(layer, x, clean, ws)
    row = M // 2
    x[row, 100] = bad
    B.ctr_dense_fwd(layer, x, dirty, ws)
    others = torch.arange(M, device="cuda") != row
    assert torch.equal(clean[others], dirty[others])
    d = dirty[row].float()
    if bad != bad:
        assert torch.isnan(d).all()
    elif dtype == F32:  # (an infinite operand's terms may cancel to NaN)
        assert not torch.isfinite(d).any()
    else:  # +-inf by the weight's sign, through SiLU: inf, or -inf / inf
        w = layer.W[:, 100].float() * bad
        assert torch.isposinf(d[w > 0]).all() and torch.isnan(d[w < 0]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_zero_rows(dtype):
    g = gen(1)
    layer = layer_of(g, dtype, 24, 40, "silu")
    x = torch.empty(0, 40, dtype=dtype, device="cuda")
    y = torch.empty(0, 24, dtype=dtype, device="cuda")
    ws = B.DenseWorkspace(layer, 0, backward=True)
    B.ctr_dense_fwd(layer, x, y, ws)
    dW, db = torch.ones(24, 40, dtype=dtype, device="cuda"), torch.ones(24, device="cuda")
    B.ctr_dense_bwd(layer, x, y, ws, dx=torch.empty_like(x), dW=dW, db=db)
    assert not dW.any() and not db.any()


def test_extreme_fp32_values():
    """Operands at fp32's ends: the largest finite value, its products with
    small weights, and denormals."""
    K = 48
    x = torch.zeros(130, K, device="cuda")
    top = torch.finfo(F32).max
    x[0, 0], x[1, 1], x[2, 2], x[3, 3] = top, -top, 1e-40, 3.39e38
    W = torch.full((40, K), 0.25, device="cuda")
    layer = B.DenseLayer(W)
    y = torch.empty(130, 40, device="cuda")
    B.ctr_dense_fwd(layer, x, y, B.DenseWorkspace(layer, 130))
    ref = x.double() @ W.double().t()
    assert torch.isfinite(y).all()
    R.assert_within(y, ref, 56 * R.U * ref.abs() + 1e-38, "y")
    assert not y[4:].any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_rows_of_a_tiny_layer(dtype):
    """More rows than a grid's second dimension counts, one weight."""
    M, g = 600001, gen(6)
    layer = layer_of(g, dtype, 1, 1, "gelu")
    x = rnd(g, M, 1).to(dtype)
    y = torch.empty(M, 1, dtype=dtype, device="cuda")
    B.ctr_dense_fwd(layer, x, y, B.DenseWorkspace(layer, M))
    ref, tol = R.dense(x, layer.W, layer.bias, "gelu", None, dtype)
    R.assert_within(y, ref, tol, "y")
    out = run_bwd(layer, x, y, False, dx=torch.empty_like(x), dW=torch.empty_like(layer.W),
                  db=torch.empty(1, device="cuda"))
    check_bwd(layer, x, y, "gelu", False, out)


@pytest.mark.parametrize("M", [1, 40])
def test_widest_layers(M):
    """A layer of 2^20 outputs and one of 2^20 inputs (the largest there are)."""
    g = gen(8)
    for N, K in ((1 << 20, 8), (24, 1 << 20)):
        layer = layer_of(g, BF16, N, K, "relu")
        x = rnd(g, M, K).to(BF16)
        y = torch.empty(M, N, dtype=BF16, device="cuda")
        B.ctr_dense_fwd(layer, x, y, B.DenseWorkspace(layer, M))
        ref, tol = R.dense(x, layer.W, layer.bias, "relu", None, BF16)
        R.assert_within(y, ref, tol, "y")


def test_offsets_past_32_bits():
    """An output of more than 2^31 elements; the rows around that offset and
    the last ones are checked."""
    N, K, g = 1032, 16, gen(3)
    M = 2 ** 31 // N + 300
    layer = layer_of(g, BF16, N, K, "relu")
    x = torch.randn(M, K, generator=g, device="cuda", dtype=BF16)
    y = torch.empty(M, N, dtype=BF16, device="cuda")
    B.ctr_dense_fwd(layer, x, y, B.DenseWorkspace(layer, M))
    for a in (0, 2 ** 31 // N - 130, M - 257):
        s = slice(a, min(M, a + 257))
        ref, tol = R.dense(x[s], layer.W, layer.bias, "relu", None, BF16)
        R.assert_within(y[s], ref, tol, "rows from %d" % a)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_equal_inputs_give_equal_bits(dtype):
    g = gen(9)
    M, K, N = 3000, 264, 392
    layer = layer_of(g, dtype, 2 * N, K, "silu")
    x, _ = x_of(g, dtype, M, K)
    dy = rnd(g, M, N).to(dtype)
    runs = []
    for _ in range(3):
        o = run_bwd(layer, x, dy, True, dx=torch.empty_like(x), dW=torch.empty_like(layer.W),
                    db=torch.empty(layer.R, device="cuda"))
        runs.append([t.clone() for t in o.values()])
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [3, 700])
def test_captured_and_replayed(dtype, M):
    """Forward and backward captured into one graph: replays on new inputs in
    the same buffers give what eager calls give, while an eager call runs on
    another stream in its own workspace."""
    g = gen(11)
    K, N = 200, 168
    layer = layer_of(g, dtype, 2 * N, K, "gelu")
    x, _ = x_of(g, dtype, M, K)
    dy = rnd(g, M, N).to(dtype)

    def buffers():
        return (torch.empty(M, N, dtype=dtype, device="cuda"), torch.empty_like(x), torch.empty_like(layer.W),
                torch.empty(layer.R, device="cuda"), B.DenseWorkspace(layer, M, gated=True, backward=True))

    def call(b, x, dy, stream=None):
        B.ctr_glu_fwd(layer, x, b[0], b[4], stream=stream)
        B.ctr_glu_bwd(layer, x, dy, b[4], dx=b[1], dW=b[2], db=b[3], stream=stream)

    eager, graphed = buffers(), buffers()
    call(eager, x, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(graphed, x, dy)
    other = torch.cuda.Stream()
    for k in range(3):
        x.copy_(rnd(g, M, K).to(dtype))
        dy.copy_(rnd(g, M, N).to(dtype))
        torch.cuda.synchronize()
        graph.replay()
        call(eager, x, dy, stream=other)
        torch.cuda.synchronize()
        for a, b in zip(eager[:4], graphed[:4]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("gated", [False, True])
def test_a_larger_workspace_serves_fewer_rows(gated):
    """One workspace for up to 3000 rows, dirty, used for calls of fewer rows."""
    g = gen(21)
    K, N = 136, 120
    layer = layer_of(g, BF16, 2 * N if gated else N, K, "silu")
    ws = B.DenseWorkspace(layer, 3000, gated=gated, backward=True)
    ws.buf.fill_(0xff)
    for M in (3000, 1, 257, 2000, 9):
        x, dy = rnd(g, M, K).to(BF16), rnd(g, M, N).to(BF16)
        y = torch.empty(M, N, dtype=BF16, device="cuda")
        out = dict(dx=torch.empty_like(x), dW=torch.empty_like(layer.W), db=torch.empty(layer.R, device="cuda"))
        if gated:
            B.ctr_glu_fwd(layer, x, y, ws)
            B.ctr_glu_bwd(layer, x, dy, ws, **out)
            ref, tol = R.glu(x, layer.W, layer.bias, "silu", BF16)
        else:
            B.ctr_dense_fwd(layer, x, y, ws)
            B.ctr_dense_bwd(layer, x, dy, ws, **out)
            ref, tol = R.dense(x, layer.W, layer.bias, "silu", None, BF16)
        R.assert_within(y, ref, tol, "y, M = %d" % M)
        check_bwd(layer, x, dy, "silu", gated, out)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("gated", [False, True])
def test_gradients_against_differences(gated, act):
    """The change of a weighted sum of the outputs along a random direction of
    (x, W, b), by central differences of the forward call in fp32. The
    difference's own error: h^2 / 6 times a third derivative, estimated as
    four thirds of what halving h changes in 64 bits (twice that is allowed),
    and the outputs' roundings over h. Those are sums of their own, each of
    which stays within its bound and, rounded to nearest, falls to either side
    alike: their weighted sum has a standard deviation of at most the root of
    the squared bounds' sum, and six of it are allowed."""
    g = gen(31)
    M, K, N, h = 40, 48, 32, 2.0 ** -6
    rows = 2 * N if gated else N
    x, W, b = rnd(g, M, K), rnd(g, rows, K, std=0.2), rnd(g, rows, std=0.3)
    vx, vW, vb, c = rnd(g, M, K), rnd(g, rows, K, std=0.2), rnd(g, rows), rnd(g, M, N)
    layer = B.DenseLayer(W, b, act=R.ACTS[act])
    out = run_bwd(layer, x, c, gated, dx=torch.empty_like(x), dW=torch.empty_like(W), db=torch.empty_like(b))
    slope = sum(float((out[n].double() * v.double()).sum()) for n, v in (("dx", vx), ("dW", vW), ("db", vb)))
    noise = 0.0

    def at(t, exact):
        nonlocal noise
        xt, Wt, bt = x + t * vx, W + t * vW, b + t * vb
        ref, tol = R.glu(xt, Wt, bt, act, F32) if gated else R.dense(xt, Wt, bt, act, None, F32)
        if exact:
            return float((ref * c.double()).sum())
        noise = math.hypot(noise, 6 * float((tol * c.double()).norm()) / (2 * h))
        y = torch.empty(M, N, device="cuda")
        at_t = B.DenseLayer(Wt, bt, act=R.ACTS[act])
        (B.ctr_glu_fwd if gated else B.ctr_dense_fwd)(at_t, xt, y, B.DenseWorkspace(at_t, M, gated=gated))
        return float((y.double() * c.double()).sum())

    def diff(h, exact):
        return (at(h, exact) - at(-h, exact)) / (2 * h)

    got, d1, d2 = diff(h, False), diff(h, True), diff(h / 2, True)
    assert abs(got - slope) <= 2 * 4 / 3 * abs(d1 - d2) + noise, (got, slope, d1, d2, noise)
    # (the comparison says something: a slope along a random direction is of this size)
    size = math.sqrt(sum(float((out[n].double() * v.double()).square().sum())
                         for n, v in (("dx", vx), ("dW", vW), ("db", vb))))
    assert noise < 0.1 * size, (noise, size)


@pytest.mark.parametrize("wl", ["taobao", "long_multihot"])
def test_a_tower_block_trained_after_the_sparse_path(wl):
    """The operators as they are used: din_sparse_fwd's pooled rows normed,
    through a gated layer and a dense layer back with the residual, normed to 8
    bits into an e4m3 layer for serving; and for training a dense layer to the
    logit, with every gradient back to the pooled rows, which din_sparse_bwd
    takes. Each call against 64 bits on its own inputs; dpooled against 64-bit
    autograd of the whole tower. There about ten values on the way are rounded
    to bf16, each within 2^-8 / sqrt 3 in the mean: sqrt(10) of that is 7e-3,
    and 2e-2 is allowed."""
    from helpers import DeviceRun
    from recsys_sparse_embedding_gb300 import synth
    batch = synth.generate(wl, seed=4, B=600, nonzero_bias=True)
    run = DeviceRun(batch)
    db = run.db
    mlp = db.mlp(B.DSF_MODE_BF16_TC)
    run.ws.prepare(mlp)
    M, D, F = batch.B, 256, 688
    pooled, din = torch.empty(M, D, device="cuda"), torch.empty(M, 48, device="cuda")
    B.din_sparse_fwd(db.tables, db.values, db.lengths, db.seq_values, db.seq_lengths, db.max_len, db.q_feat,
                     db.seq_table, M, mlp, pooled, din, run.ws, status=run.status)
    g = gen(77)
    w = 1 + 0.2 * rnd(g, D)
    up, down = layer_of(g, BF16, 2 * F, D, "silu"), layer_of(g, BF16, D, F, "none")
    head = layer_of(g, BF16, 1, D, "none")
    new = lambda *s, dt=BF16: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    res = pooled.to(BF16)
    n, hid, y, logit = new(M, D), new(M, F), new(M, D), new(M, 1)
    ws = [B.DenseWorkspace(up, M, gated=True, backward=True), B.DenseWorkspace(down, M, backward=True),
          B.DenseWorkspace(head, M, backward=True)]
    B.ctr_rms_norm_fwd(pooled, n, weight=w)
    B.ctr_glu_fwd(up, n, hid, ws[0], status=run.status)
    B.ctr_dense_fwd(down, hid, y, ws[1], residual=res, status=run.status)
    B.ctr_dense_fwd(head, y, logit, ws[2], status=run.status)
    ref, _ = R.norm(pooled, w, 1e-6)
    R.assert_within(n, ref, (D + 8) * R.U * ref.abs() + 2.0 ** -8 * ref.abs() * 1.001 + 1e-38, "norm")
    for got, (want, tol) in ((hid, R.glu(n, up.W, up.bias, "silu", BF16)),
                             (y, R.dense(hid, down.W, down.bias, "none", res, BF16)),
                             (logit, R.dense(y, head.W, head.bias, "none", None, BF16))):
        R.assert_within(got, want, tol, "layer")
    # serving: the sum of two blocks normed into 8 bits, and an e4m3 layer
    q, qs, s = torch.empty(M, D, device="cuda").to(E4M3), new(M, dt=F32), new(M, D)
    B.ctr_rms_norm_fwd(y, q, weight=w, residual=res, sum_out=s, y_scale=qs)
    e8 = layer_of(g, E4M3, 520, D, "gelu")
    z = new(M, 520)
    B.ctr_dense_fwd(e8, q, z, B.DenseWorkspace(e8, M), x_scale=qs, status=run.status)
    want, tol = R.dense(q, e8.W, e8.bias, "gelu", None, BF16, qs, e8.scale)
    R.assert_within(z, want, tol, "e4m3 layer")
    # training: back to the pooled rows
    dlogit = rnd(g, M, 1, std=0.1).to(BF16)
    dy, dhid, dn, dpooled = new(M, D), new(M, F), new(M, D), new(M, D, dt=F32)
    grads = [dict(dW=torch.empty_like(l.W), db=torch.empty_like(l.bias)) for l in (up, down, head)]
    dw = torch.empty_like(w)
    B.ctr_dense_bwd(head, y, dlogit, ws[2], dx=dy, status=run.status, **grads[2])
    B.ctr_dense_bwd(down, hid, dy, ws[1], dx=dhid, status=run.status, **grads[1])
    B.ctr_glu_bwd(up, n, dhid, ws[0], dx=dn, status=run.status, **grads[0])
    B.ctr_rms_norm_bwd(dn, pooled, dpooled, weight=w, dsum=dy.float(), dweight=dw, workspace=B.RmsNormWorkspace(M, D))
    for layer, x, d, gated, got, dx in ((up, n, dhid, True, grads[0], dn), (down, hid, dy, False, grads[1], dhid),
                                        (head, y, dlogit, False, grads[2], dy)):
        check_bwd(layer, x, d, "silu" if gated else "none", gated, dict(got, dx=dx))
    leaf = pooled.double().requires_grad_()
    t = leaf * w.double() / torch.sqrt(leaf.square().mean(1, keepdim=True) + 1e-6)
    zz = t @ up.W.double().t() + up.bias.double()
    t = torch.nn.functional.silu(zz[:, :F]) * zz[:, F:] @ down.W.double().t() + down.bias.double() + leaf
    t = t @ head.W.double().t() + head.bias.double()
    want, = torch.autograd.grad(t, leaf, dlogit.double())
    R.assert_norm(dpooled, want, 2e-2, "dpooled", M)
    state = B.SparseState(db.tables, batch.values.size + 3 * batch.seq_values.shape[1])
    bws = B.BwdWorkspace(M, batch.values.size, batch.seq_values.shape[1], batch.D)
    B.din_sparse_bwd(db.tables, db.values, db.lengths, db.seq_values, db.seq_lengths, db.max_len, db.q_feat,
                     db.seq_table, M, mlp, pooled, dpooled, torch.zeros(M, 48, device="cuda"), B.MlpGrads(batch.D),
                     state, bws, status=run.status)
    torch.cuda.synchronize()
    assert int(run.status.item()) == 0
    # feature 0's rows take their samples' slice of dpooled, summed
    f0 = state.grad[0].double().sum(0)
    lengths = torch.from_numpy(batch.lengths.reshape(batch.F, M)[0].astype("int64")).cuda()
    want = (dpooled[:, :16].double() * lengths[:, None]).sum(0)
    assert ((f0 - want).abs() <= 1e-5 * dpooled[:, :16].double().abs().mul(lengths[:, None]).sum(0) + 1e-6).all()


# ------------------------------------------------------------------ RMS norm
NORM_SIZES = [(1, 1), (1, 256), (3, 7), (5, 33), (64, 256), (9, 1000), (130, 1024), (33, 1032), (257, 48), (7, 2048),
              (12, 3001), (3, 4096), (2, 8192), (3, 9999), (2, 16392), (2, 32768), (5000, 264)]


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("yt", [F32, BF16, E4M3])
@pytest.mark.parametrize("i", range(len(NORM_SIZES)))
def test_norm_fwd(xt, yt, i):
    M, N = NORM_SIZES[i]
    g = gen(i)
    for with_res, with_w, extra in ((True, True, 0), (False, False, 0), (True, True, 3)):
        x, _ = strided((rnd(g, M, N) * torch.exp(rnd(g, M, 1))).to(xt), extra)
        res = rnd(g, M, N).to(xt) if with_res else None
        w = 1 + 0.3 * rnd(g, N) if with_w else None
        y, buf = strided(torch.zeros(M, N, device="cuda").to(yt), extra)
        keep = is_nan(buf)
        s = torch.empty(M, N, dtype=xt, device="cuda") if with_res else None
        ys = torch.empty(M, device="cuda") if yt == E4M3 else None
        B.ctr_rms_norm_fwd(x, y, weight=w, residual=res, sum_out=s, eps=1e-6, y_scale=ys)
        assert is_nan(buf)[keep].all(), "written between the rows"
        if with_res:
            assert torch.equal(s, (x.float() + res.float()).to(xt))
        ref, _ = R.norm(s if with_res else x, w, 1e-6)
        tol = (N + 8) * R.U * ref.abs() + 1e-38  # (the row sum's bound halves in the root)
        if yt == E4M3:
            want = (ref.abs().amax(1) / 448).clamp_min(2.0 ** -126)
            assert ((ys.double() - want).abs() <= (N + 10) * R.U * want).all()
            # half a step of e4m3 (2^-4 of the value; 2^-10 below its smallest normal), as values
            q = y.double() * ys.double()[:, None]
            R.assert_within(q, ref, 2.0 ** -4 * ref.abs() + 2.0 ** -10 * want[:, None] + 3 * tol, "y e4m3")
            assert (y.float().abs().amax(1)[want > 2.0 ** -126] == 448).all()
        else:
            R.assert_within(y, ref, tol + R.HALF[yt] * (ref.abs() + tol), "y")


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("i", range(len(NORM_SIZES)))
def test_norm_bwd(xt, dt, i):
    M, N = NORM_SIZES[i]
    g = gen(300 + i)
    for with_sum, with_w, extra in ((True, True, 0), (False, False, 0), (True, True, 5)):
        s, _ = strided((rnd(g, M, N) * torch.exp(rnd(g, M, 1))).to(xt), extra)
        dy = rnd(g, M, N).to(dt)
        w = 1 + 0.3 * rnd(g, N) if with_w else None
        up = rnd(g, M, N).to(xt) if with_sum else None
        dx, buf = strided(torch.zeros(M, N, device="cuda").to(xt), extra)
        keep = is_nan(buf)
        dw = torch.empty(N, device="cuda") if with_w else None
        B.ctr_rms_norm_bwd(dy, s, dx, weight=w, eps=1e-5, dsum=up, dweight=dw,
                           workspace=B.RmsNormWorkspace(M, N) if with_w else None)
        rx, tx, rw, tw = R.norm_grads(dy, s, w, 1e-5, up)
        R.assert_within(dx, rx, tx + R.HALF[xt] * (rx.abs() + tx) + 1e-38, "dx")
        assert is_nan(buf)[keep].all(), "written between the rows"
        if with_w:
            R.assert_within(dw, rw, tw, "dweight")


def test_norm_in_place_and_odd_rows():
    """The sum written over the residual, dx over the upstream gradient; rows
    of zeros (scale 2^-126, values 0), of NaN, and of infinities."""
    g = gen(2)
    x, res = rnd(g, 40, 512).to(BF16), rnd(g, 40, 512).to(BF16)
    x[3], res[3] = 0, 0
    x[5, 9] = float("nan")
    x[7, 11] = float("inf")
    want = (x.float() + res.float()).to(BF16)
    y, ys = torch.empty(40, 512, device="cuda").to(E4M3), torch.empty(40, device="cuda")
    B.ctr_rms_norm_fwd(x, y, residual=res, sum_out=res, y_scale=ys)
    assert torch.equal(res.nan_to_num(7), want.nan_to_num(7))
    assert float(ys[3]) == 2.0 ** -126 and not y[3].float().any()
    assert is_nan(y[5]).all() and is_nan(y[7, 11])
    rest = [i for i in range(40) if i not in (5, 7)]
    assert not is_nan(y[rest]).any()
    s, dy, up = rnd(g, 40, 512).to(BF16), rnd(g, 40, 512).to(BF16), rnd(g, 40, 512).to(BF16)
    rx, tx, _, _ = R.norm_grads(dy, s, None, 1e-6, up)
    B.ctr_rms_norm_bwd(dy, s, up, dsum=up)
    R.assert_within(up, rx, tx + R.HALF[BF16] * (rx.abs() + tx), "dx")


def test_norm_zero_rows():
    dw = torch.ones(16, device="cuda")
    z = torch.empty(0, 16, device="cuda")
    B.ctr_rms_norm_fwd(z, torch.empty_like(z))
    B.ctr_rms_norm_bwd(z, z, torch.empty_like(z), dweight=dw, workspace=B.RmsNormWorkspace(0, 16))
    assert not dw.any()


# ------------------------------------------------------------------ the binding's refusals
def test_binding_refuses_wrong_tensors():
    g = gen(0)
    layer = layer_of(g, BF16, 32, 64, "none")
    x, y = rnd(g, 4, 64).to(BF16), torch.empty(4, 32, dtype=BF16, device="cuda")
    ws = B.DenseWorkspace(layer, 4)
    for args in ((x.float(), y), (x, y.float()), (x[:, :32], y), (x.cpu(), y), (x, y[:, :16]), (x, y.t()),
                 (x.t().contiguous().t(), y)):
        with pytest.raises(ValueError):
            B.ctr_dense_fwd(layer, *args, ws)
    with pytest.raises(ValueError):
        B.ctr_dense_fwd(layer, x, y, ws, x_scale=torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        B.DenseLayer(rnd(g, 8, 8).to(E4M3))
    with pytest.raises(ValueError):
        B.DenseLayer(rnd(g, 8, 8).half())
    with pytest.raises(B.DsfError):  # a workspace without room for the backward
        B.ctr_dense_bwd(layer, x, y, B.DenseWorkspace(layer, 0), dx=torch.empty_like(x))
    with pytest.raises(B.DsfError):  # 16-byte rows at an odd address
        B.ctr_dense_fwd(layer, strided(x, 8, 1)[0], y, ws)
    with pytest.raises(B.DsfError):
        B.ctr_rms_norm_fwd(x, torch.empty_like(x), eps=0.0)
