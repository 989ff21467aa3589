"""The dense-tower operators as they are measured: a dense layer (bias, activation and residual in
the product's epilogue), a gated feed-forward layer, and a root-mean-square norm that adds the
residual and can write 8 bits with a scale per row. Layers and norm have their gradients.

Each operator is here in its plain form (elementary torch operations in 32 bits, rounded once at
the end) and as the library's call; ``own`` says which of the two ``run`` takes.

  dense     y = residual + act(x W^T + b)                      W [N, K]
  glu       h = act(x Wg^T + bg) * (x Wu^T + bu)               W [2F, K]: gate rows, then up rows
  rms_norm  s = x + residual in x's type; y = s w / sqrt(mean(s^2) + eps)

Types: bf16, f32, and e4m3 (x with a scale per row, W with a scale per output; y in bf16; forward
only). Gradients have their tensor's type; biases, the norm's weight and their gradients are fp32.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}


def _dense(name, dtype, M, K, N, act, residual, train):
    return {"name": name, "op": "dense", "dtype": dtype, "M": M, "K": K, "N": N, "act": act, "residual": residual,
            "train": train}


def _glu(name, dtype, M, K, F, act, train):
    return {"name": name, "op": "glu", "dtype": dtype, "M": M, "K": K, "F": F, "act": act, "train": train}


def _norm(name, dtype, out, M, N, residual, train):
    return {"name": name, "op": "rms_norm", "dtype": dtype, "out": out, "M": M, "N": N, "residual": residual,
            "train": train}


def listed():
    return [
        # one request scored alone through a tower's first layer (256 -> 512): launch latency
        _dense("dense_one_request", "bf16", 1, 256, 512, "relu", False, False),
        # a few hundred candidates through the final tower's hidden layer (176 -> 64) in fp32
        _dense("dense_candidates_f32", "f32", 500, 176, 64, "relu", False, False),
        # a batch through the deep tower's second layer (512 -> 256)
        _dense("dense_tower_bf16", "bf16", 8192, 512, 256, "relu", False, False),
        # serving in 8 bits: the projection back of a wide tower block, with the residual
        _dense("dense_serve_e4m3", "e4m3", 8192, 4096, 1024, "none", True, False),
        # a training step of a tower layer kept in fp32
        _dense("dense_train_f32", "f32", 8192, 256, 512, "silu", False, True),
        # a training step of the projection back of a wide tower block
        _dense("dense_train_bf16", "bf16", 8192, 4096, 1024, "none", True, True),
        # one request through a wide gated layer: its weights are read once
        _glu("glu_one_request", "bf16", 1, 1024, 4096, "silu", False),
        # a ragged candidate list in 8 bits, an odd hidden width (8/3 of 1024)
        _glu("glu_candidates_e4m3", "e4m3", 777, 1024, 2731, "silu", False),
        # a training step at the pooled row's width (256), hidden width 8/3 of it: odd
        _glu("glu_train_odd", "bf16", 8192, 256, 683, "gelu", True),
        # a training step of a wide gated layer: the largest case
        _glu("glu_train_wide", "bf16", 16384, 1024, 4096, "silu", True),
        # serving: the residual stream normed into 8 bits for the next product
        _norm("norm_serve_e4m3", "bf16", "e4m3", 65536, 1024, True, False),
        # a training step on the pooled rows (fp32, 256 wide) feeding bf16 towers
        _norm("norm_train_pooled", "f32", "bf16", 8192, 256, False, True),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi):  # half of them whole multiples of 16, the others as they come
        n = log_int(lo, hi)
        return max(16, n // 16 * 16) if rng.random() < 0.5 else n

    op = rng.choice(["dense", "dense", "glu", "glu", "rms_norm"])
    while True:
        M = log_int(1, 16384)
        dtype = rng.choice(["bf16", "bf16", "f32", "e4m3"])
        train = dtype != "e4m3" and rng.random() < 0.5
        # (a ReLU's gradient jumps at zero, where two exact sums may round to either side)
        act = rng.choice(["none", "silu", "gelu"] if train else ["none", "relu", "silu", "gelu"])
        if op == "dense":
            c = _dense("", dtype, M, width(32, 4096), width(32, 4096), act, rng.random() < 0.5, train)
        elif op == "glu":
            c = _glu("", dtype, M, width(32, 2048), width(32, 4096), "silu" if act == "none" else act, train)
        else:
            dtype = rng.choice(["bf16", "f32"])
            train = rng.random() < 0.4
            out = rng.choice(["bf16", dtype] if train else ["bf16", "e4m3", "e4m3", dtype])
            c = _norm("", dtype, out, log_int(1, 65536), width(32, 8192), rng.random() < 0.5, train)
        del c["name"]
        w = work(c)
        # (the largest listed case; fp32 products take six times the tensor-core work of bf16 ones)
        if w["flops"] * (6 if dtype == "f32" and op != "rms_norm" else 1) <= 7e11 and w["bytes"] <= 4e8:
            return c


def work(case):
    """Each input read once, each output written once; two operations per multiply and add."""
    M = case["M"]
    if case["op"] == "rms_norm":
        N, ex, ey = case["N"], BYTES[case["dtype"]], BYTES[case["out"]]
        b = M * N * (ex * (3 if case["residual"] else 1) + ey) + 4 * N
        f = 5.0 * M * N
        if case["out"] == "e4m3":
            b += 4 * M
        if case["train"]:  # and: dy read; dx written; dw written (s is at hand, or written above)
            b += M * N * (ey + ex) + 4 * N
            f += 9.0 * M * N
        return {"bytes": float(b), "flops": f}
    K, e = case["K"], BYTES[case["dtype"]]
    eo = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "dense":
        R, O = case["N"], case["N"]
    else:
        R, O = 2 * case["F"], case["F"]
    b = e * (M * K + R * K) + eo * M * O * (2 if case.get("residual") else 1) + 4 * R
    f = 2.0 * M * K * R
    if case["dtype"] == "e4m3":
        b += 4 * (M + R)
    if case["train"]:
        b += eo * M * O + e * (M * K + R * K) + 4 * R
        f *= 3
    return {"bytes": float(b), "flops": f}


def _quantise(t):
    """t [rows, n] -> (e4m3 values, scale per row)."""
    scale = (t.abs().amax(1) / E4M3_MAX).clamp_min(2.0 ** -126)
    return (t / scale[:, None]).to(torch.float8_e4m3fn), scale


def _inputs(case, seed):
    """The case's tensors, on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2 + 1)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    def uniform(*shape, a=1.0):
        return (torch.rand(*shape, generator=g, device="cuda") * 2 - 1) * a

    M, dt = case["M"], TORCH[case["dtype"]]
    st = {"case": dict(case)}
    if case["op"] == "rms_norm":
        N = case["N"]
        # rows of differing size, as a residual stream's
        st["x"] = (normal(M, N) * torch.exp(0.5 * normal(M, 1))).to(dt)
        st["residual"] = normal(M, N).to(dt) if case["residual"] else None
        st["weight"] = 1 + uniform(N, a=0.5)
        if case["train"]:
            st["dy"] = normal(M, N).to(TORCH[case["out"]])
        return st
    K, dense = case["K"], case["op"] == "dense"
    R, O = (case["N"], case["N"]) if dense else (2 * case["F"], case["F"])
    x = normal(M, K)
    W = uniform(R, K, a=math.sqrt(6.0 / (K + O)))
    st["b"] = uniform(R, a=0.1)
    if case["dtype"] == "e4m3":
        st["x"], st["x_scale"] = _quantise(x)
        st["W"], st["w_scale"] = _quantise(W)
        od = torch.bfloat16
    else:
        st["x"], st["W"], od = x.to(dt), W.to(dt), dt
    st["residual"] = normal(M, O).to(od) if case.get("residual") else None
    if case["train"]:
        st["dy"] = normal(M, O).to(od)
    return st


def prepare(case, seed):
    """Inputs, and what a program keeps beside them: the layer's handle, outputs and workspace."""
    st = _inputs(case, seed)
    if not own:
        return st
    from recsys_sparse_embedding_gb300 import binding as B
    M, train = case["M"], case["train"]
    empty = lambda shape, dt: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    if case["op"] == "rms_norm":
        N, x = case["N"], st["x"]
        st["y"] = empty((M, N), TORCH[case["out"]])
        st["y_scale"] = empty((M,), torch.float32) if case["out"] == "e4m3" else None
        st["sum"] = empty((M, N), x.dtype) if case["residual"] else None
        if train:
            st["dx"], st["dweight"] = torch.empty_like(x), torch.empty_like(st["weight"])
            st["ws"] = B.RmsNormWorkspace(M, N)
        return st
    act = {"none": B.DSF_ACT_NONE, "relu": B.DSF_ACT_RELU, "silu": B.DSF_ACT_SILU, "gelu": B.DSF_ACT_GELU}[case["act"]]
    gated = case["op"] == "glu"
    st["layer"] = B.DenseLayer(st["W"], st["b"], act=act, scale=st.get("w_scale"))
    st["ws"] = B.DenseWorkspace(st["layer"], M, gated=gated, backward=train)
    O = case["F"] if gated else case["N"]
    st["y"] = empty((M, O), torch.bfloat16 if case["dtype"] == "e4m3" else st["x"].dtype)
    if train:
        st["dx"], st["dW"], st["db"] = torch.empty_like(st["x"]), torch.empty_like(st["W"]), torch.empty_like(st["b"])
    return st


def run(state):
    if not own:
        return _plain(state)
    from recsys_sparse_embedding_gb300 import binding as B
    st, case = state, state["case"]
    if case["op"] == "rms_norm":
        B.ctr_rms_norm_fwd(st["x"], st["y"], weight=st["weight"], residual=st["residual"], sum_out=st["sum"], eps=EPS,
                           y_scale=st["y_scale"])
        out = {"y": st["y"]}
        if case["residual"]:
            out["sum"] = st["sum"]
        if case["out"] == "e4m3":
            out["y_scale"] = st["y_scale"]
        if case["train"]:
            s = st["sum"] if case["residual"] else st["x"]
            B.ctr_rms_norm_bwd(st["dy"], s, st["dx"], weight=st["weight"], eps=EPS, dweight=st["dweight"], workspace=st["ws"])
            out["dx"], out["dweight"] = st["dx"], st["dweight"]
        return out
    if case["op"] == "dense":
        B.ctr_dense_fwd(st["layer"], st["x"], st["y"], st["ws"], residual=st["residual"], x_scale=st.get("x_scale"))
    else:
        B.ctr_glu_fwd(st["layer"], st["x"], st["y"], st["ws"], x_scale=st.get("x_scale"))
    out = {"y": st["y"]}
    if case["train"]:
        bwd = B.ctr_dense_bwd if case["op"] == "dense" else B.ctr_glu_bwd
        bwd(st["layer"], st["x"], st["dy"], st["ws"], dx=st["dx"], dW=st["dW"], db=st["db"])
        out["dx"], out["dW"], out["db"] = st["dx"], st["dW"], st["db"]
    return out


# ------------------------------------------------------------------ plain forms, 32 bits
def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    return torch.ones_like(z)


def _plain(st):
    case = st["case"]
    return _plain_norm(st, case) if case["op"] == "rms_norm" else _plain_layer(st, case)


def _plain_norm(st, case):
    x, w, od = st["x"], st["weight"], TORCH[case["out"]]
    s = x if st["residual"] is None else (x.float() + st["residual"].float()).to(x.dtype)
    s32 = s.float()
    r = 1 / torch.sqrt((s32 * s32).mean(1, keepdim=True) + EPS)
    y = s32 * r * w
    if case["out"] == "e4m3":
        q, scale = _quantise(y)
        out = {"y": q, "y_scale": scale}
    else:
        out = {"y": y.to(od)}
    if case["residual"]:
        out["sum"] = s
    if case["train"]:
        dy = st["dy"].float()
        g = dy * w
        c = (g * s32).mean(1, keepdim=True)
        out["dx"] = (r * (g - s32 * (r * r * c))).to(x.dtype)
        out["dweight"] = (dy * s32 * r).sum(0)
    return out


def _plain_layer(st, case):
    x, W, b, act = st["x"].float(), st["W"].float(), st["b"], case["act"]
    if case["dtype"] == "e4m3":
        x, W = x * st["x_scale"][:, None], W * st["w_scale"][:, None]
    od = torch.bfloat16 if case["dtype"] == "e4m3" else st["x"].dtype
    z = x @ W.t() + b
    if case["op"] == "dense":
        y = _act(z, act)
        if st["residual"] is not None:
            y = y + st["residual"].float()
    else:
        gate, up = z[:, :case["F"]], z[:, case["F"]:]
        y = _act(gate, act) * up
    out = {"y": y.to(od)}
    if case["train"]:
        dy = st["dy"].float()
        if case["op"] == "dense":
            dz = dy * _act_grad(z, act)
        else:
            dz = torch.cat([dy * up * _act_grad(gate, act), dy * _act(gate, act)], 1)
        out["dx"], out["dW"], out["db"] = (dz @ W).to(od), (dz.t() @ x).to(od), dz.sum(0)
    return out


# ------------------------------------------------------------------ 64 bits, gradients by autograd
def exact(case, seed):
    st = _inputs(case, seed)
    d = {k: v.double() for k, v in st.items() if isinstance(v, torch.Tensor)}
    F = torch.nn.functional
    if case["op"] == "rms_norm":
        s = st["x"]
        if st["residual"] is not None:
            s = (d["x"] + d["residual"]).to(s.dtype)
        leaf, w = s.double().requires_grad_(), d["weight"].requires_grad_()
        y = leaf * w / torch.sqrt(leaf.square().mean(-1, keepdim=True) + EPS)
        out = {}
        if case["residual"]:
            out["sum"] = s.double()
        if case["out"] == "e4m3":
            out["y_scale"] = torch.maximum(y.detach().abs().max(-1).values / E4M3_MAX, torch.tensor(2.0 ** -126).to(y))
            out["y"] = y.detach() / out["y_scale"][:, None]
        else:
            out["y"] = y.detach()
        if case["train"]:
            out["dx"], out["dweight"] = torch.autograd.grad(y, (leaf, w), d["dy"])
        return out
    acts = {"none": lambda t: t, "relu": F.relu, "silu": F.silu, "gelu": F.gelu}
    x, W, b = d["x"], d["W"], d["b"]
    if case["dtype"] == "e4m3":
        x, W = x * d["x_scale"].unsqueeze(1), W * d["w_scale"].unsqueeze(1)
    for t in (x, W, b):
        t.requires_grad_()
    if case["op"] == "dense":
        y = acts[case["act"]](F.linear(x, W, b))
        if st["residual"] is not None:
            y = y + d["residual"]
    else:
        n = case["F"]
        y = acts[case["act"]](F.linear(x, W[:n], b[:n])) * F.linear(x, W[n:], b[n:])
    out = {"y": y.detach()}
    if case["train"]:
        out["dx"], out["dW"], out["db"] = torch.autograd.grad(y, (x, W, b), d["dy"])
    return out
