"""The gated scan and its gradients against 64-bit evaluations
(tests/sequence_ref.py has the bounds), through the C ABI."""
import pytest
import torch

import sequence_ref as R
from recsys_sparse_embedding_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def inputs(seed, dtype, T, D, nb):
    g = gen(seed)
    v = {"x": rnd(g, T, D).to(dtype), "gate": (rnd(g, T, D) * 1.5 - 1 + 2 * rnd(g, D)).to(dtype), "dh": rnd(g, T, D).to(dtype)}
    v["h0"], v["dh_last"] = rnd(g, nb, D), rnd(g, nb, D)
    return v


def run(v, lengths, nb, state=True, equal=False, wide=False, ws=None, backward=True):
    """All outputs of both calls; everything around them is NaN beforehand."""
    T, D = v["x"].shape
    dtype = v["x"].dtype
    n = None if equal else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    ws = ws or B.GatedScanWorkspace(T, nb, D)
    ws.buf.fill_(255)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = lambda *s: torch.full(s, NAN, device="cuda")  # noqa: E731
    if wide:  # the halves of wider rows
        xg = torch.full((T, 2 * D + wide), NAN, device="cuda").to(dtype)
        x, gate = xg[:, :D], xg[:, D:2 * D]
        x.copy_(v["x"]), gate.copy_(v["gate"])
        dxg = torch.full((T, 2 * D + wide), NAN, device="cuda").to(dtype)
        dx, dgate = dxg[:, :D], dxg[:, D:2 * D]
    else:
        x, gate, dx, dgate = v["x"], v["gate"], new(T, D).to(dtype), new(T, D).to(dtype)
    o = {"h": new(T, D).to(dtype), "dx": dx, "dgate": dgate, "h_last": new(nb, D), "dh0": new(nb, D)}
    h0, dl = (v["h0"], v["dh_last"]) if state else (None, None)
    B.ctr_gated_scan_fwd(x, gate, o["h"], nb, ws, lengths=n, h0=h0, h_last=o["h_last"], status=status)
    if backward:
        ws.buf.fill_(255)
        B.ctr_gated_scan_bwd(v["dh"], x, gate, o["h"], dx, dgate, nb, ws, lengths=n, h0=h0, dh_last=dl, dh0=o["dh0"], status=status)
    if wide:
        assert torch.isnan(dxg[:, 2 * D:].float()).all()
    return o, int(status.item())


def check(v, lengths, o, state=True, what=""):
    ref = R.scan(v["x"], v["gate"], lengths, v["h0"] if state else None, v["dh"], v["dh_last"] if state else None)
    T = sum(lengths)
    for k, r in ref.items():
        rows = o[k] if k in ("h_last", "dh0") else o[k][:T]
        R.assert_within(rows, r, what + k)
    for k in ("h", "dx", "dgate"):
        assert torch.isnan(o[k][T:].float()).all(), "rows behind the last sequence were written: " + k


def jagged(seed, nb, mean):
    g = torch.Generator().manual_seed(seed)
    return [int(x) for x in torch.empty(nb).exponential_(1.0 / mean, generator=g).floor()]


SHAPES = [("one", [1]), ("few", [0, 3, 0, 0, 5, 1]), ("ones", [1] * 300), ("two_long", [700, 0, 1500]),
          ("clicks", jagged(1, 400, 5)), ("mixed", jagged(2, 60, 90)), ("ends_empty", [40, 129, 0, 0, 0]),
          ("blocks", [128, 64, 256, 512, 32, 1, 127])]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [1, 4, 16, 37, 48, 64, 130, 200])
@pytest.mark.parametrize("name,lengths", SHAPES, ids=[s[0] for s in SHAPES])
def test_scan(dtype, D, name, lengths):
    T = sum(lengths)
    for state, behind, wide in ((True, 0, 0), (False, 5, 3), (True, 1, 4)):
        v = inputs(len(name) + D, dtype, T + behind, D, len(lengths))
        o, status = run(v, lengths, len(lengths), state=state, wide=wide)
        assert status == 0
        check(v, lengths, o, state)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,lengths", [(64, [20000]), (33, [9000, 3]), (8, [3, 45000]), (128, [4096, 4096, 9001]),
                                       (72, [12001, 1, 0, 5000])], ids=str)
def test_long_sequences_over_many_groups_of_chunks(dtype, D, lengths):
    v = inputs(3, dtype, sum(lengths), D, len(lengths))
    v["gate"] -= 4  # a long memory: states reach over many chunks
    o, status = run(v, lengths, len(lengths))
    assert status == 0
    check(v, lengths, o)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nb,L,D", [(1, 1, 64), (512, 1, 256), (7, 1, 33), (1000, 1, 2), (3, 1, 1001), (3, 64, 64), (5, 100, 48), (2, 5000, 64), (300, 8, 20)])
def test_equal_lengths(dtype, nb, L, D):
    v = inputs(nb + L, dtype, nb * L, D, nb)
    o, status = run(v, None, nb, equal=True)
    assert status == 0
    check(v, [L] * nb, o)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_gates_ends(dtype):
    """Saturated gates: the state kept for ever, and replaced at once."""
    v = inputs(4, dtype, 3000, 48, 2)
    v["gate"][:, :16] = -120.0
    v["gate"][:, 16:32] = 120.0
    v["gate"][:, 32:40] = -30.0
    o, _ = run(v, [1400, 1600], 2)
    check(v, [1400, 1600], o)
    assert torch.equal(o["h_last"][:, :16], v["h0"][:, :16])


def test_no_rows_and_no_sequences():
    v = inputs(5, F32, 0, 32, 3)
    for equal in (True, False):
        o, status = run(v, [0, 0, 0], 3, equal=equal)
        assert status == 0
        assert torch.equal(o["h_last"], v["h0"]) and torch.equal(o["dh0"], v["dh_last"])
        o, _ = run(v, [0, 0, 0], 3, state=False, equal=equal)
        assert (o["h_last"] == 0).all() and (o["dh0"] == 0).all()
    v = inputs(5, F32, 6, 32, 0)
    o, status = run(v, [], 0)
    assert status == 0 and torch.isnan(o["h"]).all() and torch.isnan(o["dx"]).all()


@pytest.mark.parametrize("lengths,T,cut,flag", [
    ([3, -2, 4], 20, [3, 0, 4], B.FLAG_NEG_LENGTH),
    ([300, 500], 600, [300, 300], B.FLAG_COUNT),
    ([2 ** 31 - 1, 2 ** 31 - 1, 5], 700, [700, 0, 0], B.FLAG_COUNT),
    ([-5, 900, 3], 100, [0, 100, 0], B.FLAG_COUNT | B.FLAG_NEG_LENGTH)])
def test_bad_lengths(lengths, T, cut, flag):
    v = inputs(6, F32, T, 40, len(lengths))
    o, status = run(v, lengths, len(lengths))
    assert status == flag
    check(v, cut, o)


@pytest.mark.parametrize("D,lengths", [(4, [140000, 3]), (64, [0, 131073]), (36, [1] * 1500 + [270000])], ids=["4", "64", "36"])
def test_more_rows_than_one_block_marks(D, lengths):
    v = inputs(9, F32, sum(lengths), D, len(lengths))
    o, status = run(v, lengths, len(lengths))
    assert status == 0
    check(v, lengths, o)


@pytest.mark.parametrize("nb,mean", [(65536, 0.8), (65537, 0.8), (200003, 0.6)])
def test_very_many_sequences(nb, mean):
    """Most of them empty; one of a negative length among the last."""
    lengths = jagged(7, nb, mean)
    v = inputs(8, F32, sum(lengths) + 2, 8, nb)
    o, status = run(v, lengths[:-3] + [-4] + lengths[-2:], nb)
    cut = lengths[:-3] + [0] + lengths[-2:]
    assert status == B.FLAG_NEG_LENGTH
    check(v, cut, o)


@pytest.mark.parametrize("D", [48, 33])
def test_non_finite_values_stay_in_their_sequence(D):
    lengths = [5, 300, 1, 700, 40, 1300]
    begin = [sum(lengths[:i]) for i in range(7)]
    v = inputs(7, F32, sum(lengths), D, 6)
    bad = {k: t.clone() for k, t in v.items()}
    bad["x"][begin[1] + 3] = float("inf")
    bad["gate"][begin[3] + 650] = NAN
    bad["dh"][begin[1] + 299] = NAN
    bad["h0"][5] = float("inf")
    bad["dh_last"][3] = NAN
    o, _ = run(v, lengths, 6)
    p, _ = run(bad, lengths, 6)
    for s in (0, 2, 4):
        rows = slice(begin[s], begin[s + 1])
        for k in ("h", "dx", "dgate"):
            assert torch.equal(o[k][rows], p[k][rows]), (k, s)
        for k in ("h_last", "dh0"):
            assert torch.equal(o[k][s], p[k][s]), (k, s)
    assert torch.equal(o["h"][begin[1]:begin[1] + 3], p["h"][begin[1]:begin[1] + 3])
    assert not torch.isfinite(p["h"][begin[1] + 3:begin[2]]).any()
    assert not torch.isfinite(p["h_last"][5]).any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_equal_calls_give_equal_bits(dtype):
    lengths = [9000, 20, 14000]
    v = inputs(8, dtype, sum(lengths), 256, 3)
    v["gate"] -= 3
    o, _ = run(v, lengths, 3)
    for _ in range(5):
        p, _ = run(v, lengths, 3)
        for k in o:
            assert torch.equal(o[k], p[k]), k


def test_a_state_carried_from_call_to_call():
    """A sequence in one call, in two, and row by row as when serving."""
    v = inputs(9, F32, 700, 64, 1)
    whole, _ = run(v, [700], 1)
    ws = B.GatedScanWorkspace(700, 1, 64)
    h, state = torch.empty(700, 64, device="cuda"), v["h0"].clone()
    for a, b in ((0, 400), (400, 700)):
        nxt = torch.empty_like(state)
        B.ctr_gated_scan_fwd(v["x"][a:b], v["gate"][a:b], h[a:b], 1, ws, h0=state, h_last=nxt)
        state = nxt
    ref = R.scan(v["x"], v["gate"], [700], v["h0"])
    R.assert_within(h, ref["h"], "two calls")
    state = v["h0"].clone()
    for t in range(40):
        nxt = torch.empty_like(state)
        B.ctr_gated_scan_fwd(v["x"][t:t + 1], v["gate"][t:t + 1], h[t:t + 1], 1, ws, h0=state, h_last=nxt)
        state = nxt
    R.assert_within(h[:40], (ref["h"][0][:40], ref["h"][1][:40]), "steps")


def test_rows_far_apart():
    """Offsets past 2^31 elements."""
    T, D, ld = 70000, 24, 32000
    buf = torch.empty(T * ld, dtype=BF16, device="cuda")
    x = buf.view(T, ld)[:, :D]
    v = inputs(10, BF16, T, D, 2)
    x.copy_(v["x"])
    h = buf.view(T, ld)[:, 64:64 + D]
    ws = B.GatedScanWorkspace(T, 2, D)
    n = torch.tensor([30000, 40000], dtype=torch.int32, device="cuda")
    B.ctr_gated_scan_fwd(x, v["gate"], h, 2, ws, lengths=n)
    near = torch.empty(T, D, dtype=BF16, device="cuda")
    B.ctr_gated_scan_fwd(v["x"], v["gate"], near, 2, ws, lengths=n)
    assert torch.equal(h, near)


def test_streams_and_graphs():
    lengths = [5000, 12, 3000]
    v = inputs(11, BF16, sum(lengths), 64, 3)
    o, _ = run(v, lengths, 3)
    ws = B.GatedScanWorkspace(sum(lengths), 3, 64)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [{k: torch.zeros_like(t) for k, t in o.items()} for _ in range(2)]

    def both(p):
        B.ctr_gated_scan_fwd(v["x"], v["gate"], p["h"], 3, ws, lengths=n, h0=v["h0"], h_last=p["h_last"])
        B.ctr_gated_scan_bwd(v["dh"], v["x"], v["gate"], p["h"], p["dx"], p["dgate"], 3, ws, lengths=n, h0=v["h0"],
                             dh_last=v["dh_last"], dh0=p["dh0"])

    with torch.cuda.stream(side):
        both(outs[0])
    side.synchronize()
    for k in o:
        assert torch.equal(outs[0][k], o[k]), k
    graphs = []
    for p in outs:  # two graphs on one workspace, replayed one after the other
        gph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gph):
            both(p)
        graphs.append(gph)
    for _ in range(3):
        for p in outs:
            for t in p.values():
                t.fill_(NAN)
        for gph in graphs:
            gph.replay()
        torch.cuda.synchronize()
        for p in outs:
            for k in o:
                assert torch.equal(p[k], o[k]), k


def test_gradients_against_differences():
    """(f(v + d) - f(v - d)) / 2 along random directions, f = <h, dh> +
    <h_last, dh_last> in 64 bits from the kernel's fp32 outputs. The steps are
    2^-7: the third derivatives of f along a direction of norm sqrt(T D) are
    taken as at most 4 T D, so the quotient is off by at most 2^-14 4 T D / 6;
    fp32 roundings of T D outputs (about 2^-22 each, of random sign) add
    2^-22 sqrt(T D) 2^7."""
    lengths, D = [3, 0, 60, 17], 32
    T = sum(lengths)
    v = inputs(12, F32, T, D, 4)
    o, _ = run(v, lengths, 4)

    def f(w):
        p, _ = run(w, lengths, 4, backward=False)
        return float((p["h"].double() * v["dh"].double()).sum() + (p["h_last"].double() * v["dh_last"].double()).sum())

    step, g = 2.0 ** -7, gen(13)
    for name, grad in (("x", "dx"), ("gate", "dgate"), ("h0", "dh0")):
        d = torch.sign(rnd(g, *v[name].shape))
        up, down = dict(v), dict(v)
        up[name], down[name] = v[name] + step * d, v[name] - step * d
        slope = (f(up) - f(down)) / (2 * step)
        want = float((o[grad].double() * d.double()).sum())
        n = d.numel()
        assert abs(slope - want) <= step ** 2 * 4 * n / 6 + 2.0 ** -22 * (T * D) ** 0.5 / step, name


def test_refusals():
    v = inputs(14, F32, 12, 8, 3)
    ws = B.GatedScanWorkspace(12, 3, 8)
    h = torch.empty_like(v["x"])
    n = torch.tensor([4, 4, 4], dtype=torch.int32, device="cuda")
    ok = dict(x=v["x"], gate=v["gate"], h=h, B=3, workspace=ws, lengths=n)
    B.ctr_gated_scan_fwd(**ok)
    for kw in (dict(x=v["x"].half()), dict(x=v["x"].cpu()), dict(gate=v["gate"].to(BF16)), dict(gate=v["gate"][:, :7]),
               dict(h=h[:11]), dict(h=h.t().contiguous().t()), dict(lengths=n.long()), dict(lengths=n[:2]),
               dict(lengths=n.cpu()), dict(lengths=None, B=5), dict(h0=v["h0"][:2]), dict(h0=v["h0"].to(BF16)),
               dict(h_last=v["h0"].t()), dict(lengths=None, B=0)):
        with pytest.raises(ValueError):
            B.ctr_gated_scan_fwd(**{**ok, **kw})
    with pytest.raises(B.DsfError):
        B.ctr_gated_scan_fwd(**{**ok, "workspace": B.GatedScanWorkspace(0, 1, 8)})
    with pytest.raises(B.DsfError):
        B.GatedScanWorkspace(-1, 1, 8)
