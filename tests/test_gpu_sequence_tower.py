"""The sequence-tower operators together, as a training step uses them: item rows
from the catalogue through a dense layer to x and gate, the gated scan over jagged
click sequences, the cross entropy against the catalogue, the gradients back through
all of them, and the update of the layer's matrix."""
import os
import subprocess
import sys

import pytest
import torch

import sequence_ref as R
from recsys_sparse_embedding_gb300 import binding as B

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F32 = torch.bfloat16, torch.float32
# 2-norms: bf16 rounds items, x and gate, h, dz, dh, dx and dgate, and the gradients (nine roundings
# of at most 2^-8, each passed on by operators that grow none of them more than twofold in the
# mean): 18 2^-8 at the worst, a quarter of it where signs are random. fp32: the same count of 2^-23
# times the sums' lengths (up to 64 terms' roots)
REL = {BF16: 18 * 2.0 ** -8 / 4, F32: 18 * 64 * 2.0 ** -23}


def setup(dtype, V=3000, D=48, nb=200):
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    lengths = torch.randint(0, 12, (nb,), generator=g, device="cuda")
    lengths[3], lengths[50] = 300, 0
    T = int(lengths.sum())
    s = {"table": (rnd(V, D) * 0.3).to(dtype), "W": (rnd(2 * D, D) * D ** -0.5).to(dtype), "b": 0.1 * rnd(2 * D),
         "lengths": lengths.to(torch.int32), "T": T, "nb": nb, "D": D, "V": V,
         "items": torch.randint(0, V, (T,), generator=g, device="cuda")}
    ends = lengths.cumsum(0)
    nxt = torch.cat([s["items"][1:], s["items"][:1]])
    nxt[(ends[lengths > 0] - 1)] = -1  # a sequence's last row has no next item
    s["target"] = nxt
    s["momentum"] = torch.zeros(2 * D, D, device="cuda")
    return s


class Step:
    """What a program keeps: handles, workspaces, activations."""

    def __init__(self, s):
        dt, T, D, V = s["table"].dtype, s["T"], s["D"], s["V"]
        new = lambda *sh, t=dt: torch.full(sh, float("nan"), device="cuda").to(t)  # noqa: E731
        self.s = s
        self.layer, self.catalogue = B.DenseLayer(s["W"], s["b"]), B.DenseLayer(s["table"])
        self.ws_d = B.DenseWorkspace(self.layer, T, backward=True)
        self.ws_s = B.GatedScanWorkspace(T, s["nb"], D)
        self.ws_x = B.SoftmaxXentWorkspace(self.catalogue, T, backward=True)
        self.ws_m = B.MuonWorkspace(s["W"])
        self.x, self.xg, self.h, self.dh, self.dxg, self.dx = (new(T, w) for w in (D, 2 * D, D, D, 2 * D, D))
        self.loss, self.lse = new(T, t=F32), new(T, t=F32)
        self.g = (s["target"] >= 0).float() / int((s["target"] >= 0).sum())
        self.dtable, self.dW, self.db = new(V, D), new(2 * D, D), new(2 * D, t=F32)

    def __call__(self):
        s, D = self.s, self.s["D"]
        torch.index_select(s["table"], 0, s["items"], out=self.x)
        B.ctr_dense_fwd(self.layer, self.x, self.xg, self.ws_d)
        B.ctr_gated_scan_fwd(self.xg[:, :D], self.xg[:, D:], self.h, s["nb"], self.ws_s, lengths=s["lengths"])
        B.ctr_softmax_xent_fwd(self.catalogue, self.h, s["target"], self.loss, self.lse, self.ws_x)
        B.ctr_softmax_xent_bwd(self.catalogue, self.h, s["target"], self.lse, self.ws_x, dloss=self.g, dx=self.dh, dW=self.dtable)
        B.ctr_gated_scan_bwd(self.dh, self.xg[:, :D], self.xg[:, D:], self.h, self.dxg[:, :D], self.dxg[:, D:], s["nb"], self.ws_s,
                             lengths=s["lengths"])
        B.ctr_dense_bwd(self.layer, self.x, self.dxg, self.ws_d, dx=self.dx, dW=self.dW, db=self.db)
        B.ctr_muon_update(s["W"], self.dW, s["momentum"], self.ws_m)


def reference(s, g):
    table, W, b = (s[k].double().requires_grad_() for k in ("table", "W", "b"))
    x = table.detach()[s["items"]].requires_grad_()
    xg = x @ W.t() + b
    z = torch.sigmoid(xg[:, s["D"]:])
    rows, p = [], 0
    for n in s["lengths"].tolist():
        h = torch.zeros(s["D"], dtype=torch.float64, device="cuda")
        for t in range(p, p + n):
            h = (1 - z[t]) * h + z[t] * xg[t, :s["D"]]
            rows.append(h)
        p += n
    logits = torch.stack(rows) @ table.t()
    loss = torch.nn.functional.cross_entropy(logits, s["target"], ignore_index=-1, reduction="none")
    grads = torch.autograd.grad((loss * g).sum(), (x, W, b, table))
    return loss.detach(), grads


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_training_step(dtype):
    s = setup(dtype)
    W0 = s["W"].clone()
    step = Step(s)
    step()
    after = s["W"].clone()
    s["W"].copy_(W0)
    loss, grads = reference(s, step.g.double())
    norm = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert norm(step.loss, loss) <= REL[dtype]
    for got, want, name in zip((step.dx, step.dW, step.db, step.dtable), grads, ("dx", "dW", "db", "dtable")):
        assert norm(got, want) <= REL[dtype], name
    w, m, _ = R.muon(W0, step.dW, torch.zeros_like(s["momentum"]), 0.02, 0.95, 0.0, True, 5)
    assert norm(after, w) <= 2 * R.HALF[dtype] + 1e-5 and norm(s["momentum"], m) <= 2.0 ** -22


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_captured_training_step(dtype):
    """Replayed, the step gives what it gives eagerly, step after step."""
    a, b = setup(dtype), setup(dtype)
    eager, kept = Step(a), Step(b)
    eager()
    kept()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept()
    for _ in range(3):
        eager()
        g.replay()
        torch.cuda.synchronize()
        for k in ("loss", "dx", "dtable", "dW", "db"):
            assert torch.equal(getattr(eager, k), getattr(kept, k)), k
        assert torch.equal(a["W"], b["W"]) and torch.equal(a["momentum"], b["momentum"])


def test_two_streams_at_once():
    """Steps side by side, each with its own workspaces."""
    steps = [Step(setup(BF16)) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for st, stream in zip(steps, streams):
        with torch.cuda.stream(stream):
            for _ in range(3):
                st()
    torch.cuda.synchronize()
    for st in steps[1:]:
        for k in ("loss", "dx", "dtable", "dW", "db"):
            assert torch.equal(getattr(st, k), getattr(steps[0], k)), k
        assert torch.equal(st.s["W"], steps[0].s["W"])


def test_long_scans_on_several_streams():
    """Blocks of one call wait for others of the same call while more calls compete
    for the chip."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    T, D = 60000, 256
    x, gate = (torch.randn(T, D, generator=g, device="cuda").to(BF16) for _ in range(2))
    want = torch.empty_like(x)
    B.ctr_gated_scan_fwd(x, gate, want, 1, B.GatedScanWorkspace(T, 1, D))
    outs = [torch.empty_like(x) for _ in range(4)]
    wss = [B.GatedScanWorkspace(T, 1, D) for _ in outs]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    streams = [torch.cuda.Stream() for _ in outs]
    torch.cuda.synchronize()
    for _ in range(10):
        for o, w, s in zip(outs, wss, streams):
            with torch.cuda.stream(s):
                B.ctr_gated_scan_fwd(x, gate, o, 1, w, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for o in outs:
        assert torch.equal(o, want)


REFUSED = """
import torch
from recsys_sparse_embedding_gb300 import binding as B
x = torch.ones(40, 64, device="cuda")
y, m = torch.empty_like(x), torch.zeros_like(x)
n = torch.tensor([30, 10], dtype=torch.int32, device="cuda")
layer = B.DenseLayer(torch.ones(4800, 64, device="cuda"))
few = B.SoftmaxXentWorkspace(layer, 40, backward=True)
t = torch.zeros(40, dtype=torch.int64, device="cuda")
l, lse = torch.empty(40, device="cuda"), torch.zeros(40, device="cuda")
ws, mw = B.GatedScanWorkspace(40, 40, 64), B.MuonWorkspace(x)
calls = {"scan": lambda: B.ctr_gated_scan_fwd(x, x, y, 2, ws, lengths=n), "step": lambda: B.ctr_gated_scan_fwd(x, x, y, 40, ws),
         "loss": lambda: B.ctr_softmax_xent_fwd(layer, x, t, l, lse, few),
         "gradients": lambda: B.ctr_softmax_xent_bwd(layer, x, t, lse, few, dx=y),
         "update": lambda: B.ctr_muon_update(y, x, m, mw)}
for c in calls.values():
    c()
torch.cuda.synchronize()
for name, c in calls.items():
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        g.capture_begin()
        try:
            s.synchronize()  # not allowed while capturing: the capture is void
        except RuntimeError:
            pass
        try:
            c()
            print(name, "was not refused")
        except B.DsfError as e:
            assert e.code == B.DSF_ECUDA
        try:
            g.capture_end()
        except RuntimeError:
            pass
    B.HashTable(64, 16, B.DSF_F32, [0])  # raises if its launch seems to fail
torch.cuda.synchronize()
print("done")
"""


def test_a_refused_launch_does_not_fail_the_next_call():
    r = subprocess.run([sys.executable, "-c", REFUSED], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.stdout.split() == ["done"], r.stdout + r.stderr[-2000:]
