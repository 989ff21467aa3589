"""What a sequence tower's training adds to the dense-tower operators, as it is measured: the softmax
cross entropy of rows against a catalogue (its next item), a gated linear recurrence over click
sequences, and the orthogonalised update of the towers' matrices.

Each operator is here in its plain form (elementary torch operations in 32 bits, rounded once at
the end) and as the library's call; ``own`` says which of the two ``run`` takes.

  xent   z = x W^T + b, lse = log sum_v exp z_v, loss = lse - z_target (target -1: a row left out);
         gradients for dloss: dz = dloss (exp(z - lse) - [v = target]), dx = dz W, dW = dz^T x, db
  scan   per sequence and channel h_t = (1 - z_t) h_{t-1} + z_t x_t, z = sigmoid(gate), from h0;
         gradients of x, gate and h0 for dh and dh_last
  muon   momentum m = mu m + g, u = g + mu m, O = five Newton-Schulz steps on u / |u|,
         W = W - lr sqrt(max(1, rows / columns)) O

Types: bf16 and f32. Losses, lse, biases, states (h0, h_last) and momenta are fp32 in both;
gradients have their tensor's type.
"""
import math

import torch

own = False

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
NS = (3.4445, -4.7750, 2.0315)  # the Newton-Schulz step's X -> a X + (b A + c A^2) X, A = X X^T
NS_STEPS, NS_EPS, LR, MU = 5, 1e-7, 0.02, 0.95


def _xent(name, dtype, M, K, V, bias, train):
    return {"name": name, "op": "xent", "dtype": dtype, "M": M, "K": K, "V": V, "bias": bias, "train": train}


def _scan(name, dtype, B, T, D, ragged, h0, train):
    return {"name": name, "op": "scan", "dtype": dtype, "B": B, "T": T, "D": D, "ragged": ragged, "h0": h0, "train": train}


def _muon(name, dtype, R, C):
    return {"name": name, "op": "muon", "dtype": dtype, "R": R, "C": C}


def listed():
    return [
        # one user's next ad against the adgroup table (846,812 rows): its rows are read once
        _xent("xent_one_user", "bf16", 1, 64, 846812, False, False),
        # a few hundred samples against the category table, towers kept in fp32 (176 wide)
        _xent("xent_categories_f32", "f32", 500, 176, 12961, True, True),
        # a batch's training step against the adgroup table
        _xent("xent_train_adgroups", "bf16", 8192, 64, 846812, False, True),
        # a training step of a wide tower, with a popularity correction as the bias: the largest case
        _xent("xent_train_wide", "bf16", 16384, 1024, 65536, True, True),
        # serving: one more click for each of a few hundred users
        _scan("scan_step", "bf16", 512, 512, 256, False, True, False),
        # click sequences of a batch, 5 long in the mean, at the sequence embedding's width (48), in fp32
        _scan("scan_clicks_f32", "f32", 8192, 40960, 48, True, False, True),
        # longer click sequences
        _scan("scan_long_clicks", "bf16", 8192, 285000, 256, True, False, True),
        # a few users' whole histories, continued from a state
        _scan("scan_histories", "bf16", 6, 131071, 1024, True, True, True),
        # the deep tower's first layer
        _muon("muon_tower_f32", "f32", 512, 256),
        # a gated layer of hidden width 683
        _muon("muon_odd_bf16", "bf16", 1366, 256),
        # the projection back of a wide tower block
        _muon("muon_projection_f32", "f32", 1024, 4096),
        # a wide gated layer
        _muon("muon_gated_bf16", "bf16", 8192, 1024),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi):  # half of them whole multiples of 16, the others as they come
        n = log_int(lo, hi)
        return max(16, n // 16 * 16) if rng.random() < 0.5 else n

    op = rng.choice(["xent", "xent", "scan", "scan", "muon"])
    while True:
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if op == "xent":
            c = _xent("", dtype, log_int(1, 16384), width(16, 1024), log_int(100, 1000000), rng.random() < 0.5, rng.random() < 0.6)
            # (fp32 products take six times the tensor-core work of bf16 ones)
            fits = c["M"] * c["V"] <= 6.9e9 and 2.0 * c["M"] * c["K"] * c["V"] <= (2.2e12 if dtype == "bf16" else 3.5e11) and c["K"] * c["V"] <= 2.2e8
        elif op == "scan":
            B = log_int(1, 16384)
            ragged = rng.random() < 0.7
            T = B * log_int(1, 262144) if not ragged else log_int(B, 524288)
            c = _scan("", dtype, B, T, width(16, 2048), ragged, rng.random() < 0.5, rng.random() < 0.6)
            fits = T <= 524288 and T // B <= 65536 and T * c["D"] * BYTES[dtype] <= 2.6e8
        else:
            c = _muon("", dtype, width(16, 8192), width(16, 8192))
            fits = min(c["R"], c["C"]) <= 2048 and work(c)["flops"] <= 1.4e11
        del c["name"]
        if fits:
            return c


def work(case):
    """Each input read once, each output written once; two operations per multiply and add."""
    e = BYTES[case["dtype"]]
    if case["op"] == "xent":
        M, K, V = case["M"], case["K"], case["V"]
        b = e * (M * K + V * K) + M * (8 + 4 + 4) + 4 * V * case["bias"]
        f = 2.0 * M * K * V
        if case["train"]:  # and: dloss read; dx, dW, db written
            b += 4 * M + e * (M * K + V * K) + 4 * V * case["bias"]
            f *= 3
        return {"bytes": float(b), "flops": f}
    if case["op"] == "scan":
        B, n = case["B"], case["T"] * case["D"]
        s = 4.0 * B * case["D"]
        b = 3.0 * e * n + s * (2 if case["h0"] else 1) + 4 * B * case["ragged"]
        f = 8.0 * n
        if case["train"]:  # and: dh, dh_last read; dx, dgate, dh0 written
            b += 3.0 * e * n + s * (2 if case["h0"] else 1)
            f += 10.0 * n
        return {"bytes": b, "flops": f}
    R, C = case["R"], case["C"]
    n, m = min(R, C), max(R, C)
    # W, momentum read and written, the gradient read; two of a step's three products are symmetric
    return {"bytes": float(R * C * (3 * e + 8)), "flops": NS_STEPS * (3.0 * n * n * m + float(n) ** 3)}


def _inputs(case, seed):
    """The case's tensors, on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2 + 1)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    def uniform(*shape, a=1.0):
        return (torch.rand(*shape, generator=g, device="cuda") * 2 - 1) * a

    dt = TORCH[case["dtype"]]
    st = {"case": dict(case)}
    if case["op"] == "xent":
        M, K, V = case["M"], case["K"], case["V"]
        st["x"] = normal(M, K).to(dt)
        st["W"] = normal(V, K, std=1.5 / math.sqrt(K)).to(dt)  # logits of a trained model's spread
        # targets: popular items more often; a twentieth of the rows has none
        rank = torch.rand(M, generator=g, device="cuda", dtype=torch.float64)
        target = torch.exp(rank * math.log(V)).long().clamp_(max=V) - 1
        left_out = torch.rand(M, generator=g, device="cuda") < (0.05 if M > 1 else 0.0)
        st["target"] = torch.where(left_out, torch.full_like(target, -1), target)
        st["b"] = uniform(V, a=2.0) if case["bias"] else None
        if case["train"]:
            st["dloss"] = (1 + uniform(M, a=0.5)) / M
        return st
    if case["op"] == "scan":
        B, T, D = case["B"], case["T"], case["D"]
        # x and gate are the halves of one product's rows
        st["xg"] = torch.cat([normal(T, D), normal(T, D) + uniform(D, a=2.5) - 1.5], 1).to(dt)
        st["lengths"] = None
        if case["ragged"]:
            cuts = torch.randint(0, T + 1, (B - 1,), generator=g, device="cuda").sort().values
            ends = torch.cat([cuts, torch.tensor([T], device="cuda")])
            st["lengths"] = torch.diff(ends, prepend=ends.new_zeros(1)).to(torch.int32)
        st["h0"] = normal(B, D) if case["h0"] else None
        if case["train"]:
            st["dh"] = normal(T, D).to(dt)
            st["dh_last"] = normal(B, D)
        return st
    R, C = case["R"], case["C"]
    # gradients: a few directions that every sample pulls at, and the rest
    k = min(R, C, 8)

    def gradient():
        return 1e-3 * (normal(R, k) @ normal(k, C) + normal(R, C))

    st["grad"] = gradient().to(dt)
    st["momentum"] = 4 * gradient()
    st["W"] = uniform(R, C, a=math.sqrt(6.0 / (R + C))).to(dt)
    return st


def prepare(case, seed):
    """Inputs, and what a program keeps beside them: the layer's handle, outputs and workspace."""
    st = _inputs(case, seed)
    if not own:
        return st
    from recsys_sparse_embedding_gb300 import binding as L
    empty = lambda shape, dt=torch.float32: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    if case["op"] == "xent":
        st["layer"] = L.DenseLayer(st["W"], st["b"])
        st["ws"] = L.SoftmaxXentWorkspace(st["layer"], case["M"], backward=case["train"])
        st["loss"], st["lse"] = empty((case["M"],)), empty((case["M"],))
        if case["train"]:
            st["dx"], st["dW"] = torch.empty_like(st["x"]), torch.empty_like(st["W"])
            st["db"] = None if st["b"] is None else torch.empty_like(st["b"])
    elif case["op"] == "scan":
        B, T, D = case["B"], case["T"], case["D"]
        st["ws"] = L.GatedScanWorkspace(T, B, D)
        st["h"], st["h_last"] = empty((T, D), st["xg"].dtype), empty((B, D))
        if case["train"]:
            st["dxg"] = torch.empty_like(st["xg"])
            st["dh0"] = empty((B, D)) if case["h0"] else None
    else:
        st["ws"] = L.MuonWorkspace(st["W"])
    return st


def run(state):
    if not own:
        return _plain(state)
    from recsys_sparse_embedding_gb300 import binding as L
    st, case = state, state["case"]
    if case["op"] == "xent":
        L.ctr_softmax_xent_fwd(st["layer"], st["x"], st["target"], st["loss"], st["lse"], st["ws"])
        out = {"loss": st["loss"], "lse": st["lse"]}
        if case["train"]:
            L.ctr_softmax_xent_bwd(st["layer"], st["x"], st["target"], st["lse"], st["ws"], dloss=st["dloss"],
                                   dx=st["dx"], dW=st["dW"], db=st["db"])
            out["dx"], out["dW"] = st["dx"], st["dW"]
            if case["bias"]:
                out["db"] = st["db"]
        return out
    if case["op"] == "scan":
        B, D = case["B"], case["D"]
        x, gate = st["xg"][:, :D], st["xg"][:, D:]
        L.ctr_gated_scan_fwd(x, gate, st["h"], B, st["ws"], lengths=st["lengths"], h0=st["h0"], h_last=st["h_last"])
        out = {"h": st["h"], "h_last": st["h_last"]}
        if case["train"]:
            L.ctr_gated_scan_bwd(st["dh"], x, gate, st["h"], st["dxg"][:, :D], st["dxg"][:, D:], B, st["ws"],
                                 lengths=st["lengths"], h0=st["h0"], dh_last=st["dh_last"], dh0=st["dh0"])
            out["dxg"] = st["dxg"]
            if case["h0"]:
                out["dh0"] = st["dh0"]
        return out
    L.ctr_muon_update(st["W"], st["grad"], st["momentum"], st["ws"], lr=LR, mu=MU, nesterov=True, steps=NS_STEPS)
    return {"W": st["W"], "momentum": st["momentum"]}


# ------------------------------------------------------------------ plain forms, 32 bits
def _plain(st):
    case = st["case"]
    return {"xent": _plain_xent, "scan": _plain_scan, "muon": _plain_muon}[case["op"]](st, case)


def _plain_xent(st, case):
    x, W, target = st["x"].float(), st["W"].float(), st["target"]
    z = x @ W.t()
    if case["bias"]:
        z += st["b"]
    top = z.amax(1, keepdim=True)
    there = target >= 0
    at = target.clamp_min(0)[:, None]
    zt = z.gather(1, at)[:, 0]
    e = torch.exp(z.sub_(top))
    s = e.sum(1)
    lse = top[:, 0] + torch.log(s)
    out = {"loss": torch.where(there, lse - zt, torch.zeros_like(lse)), "lse": lse}
    if case["train"]:
        d = torch.where(there, st["dloss"], torch.zeros_like(lse))
        dz = e.mul_((d / s)[:, None])
        dz.scatter_add_(1, at, -d[:, None])
        out["dx"], out["dW"] = (dz @ W).to(st["x"].dtype), (dz.t() @ x).to(st["W"].dtype)
        if case["bias"]:
            out["db"] = dz.sum(0)
    return out


def _double(a, b, longest):
    """y_t = a_t y_{t-1} + b_t along the rows, y_{-1} = 0, by doubling: after k rounds a and b stand for 2^k rows."""
    n = 1
    while n < longest:
        b = torch.cat([b[:n], b[n:] + a[n:] * b[:-n]])
        a = torch.cat([torch.zeros_like(a[:n]), a[n:] * a[:-n]])
        n *= 2
    return b


def _plain_scan(st, case):
    B, T, D = case["B"], case["T"], case["D"]
    xg, longest = st["xg"].float(), T if case["ragged"] else T // B
    x, z = xg[:, :D], 1 / (1 + torch.exp(-xg[:, D:]))
    keep = 1 / (1 + torch.exp(xg[:, D:]))
    lengths = st["lengths"].long() if case["ragged"] else torch.full((B,), longest, device=x.device)
    ends = lengths.cumsum(0)
    row = torch.arange(T, device=x.device)
    seq = torch.searchsorted(ends, row, right=True)
    first, last = (row == (ends - lengths)[seq])[:, None], (row == ends[seq] - 1)[:, None]
    some, tail, head = (lengths > 0)[:, None], (ends - 1).clamp_min(0), (ends - lengths).clamp_max(T - 1)
    h0 = st["h0"] if case["h0"] else torch.zeros(B, D, device=x.device)
    # a sequence starts from its own state: nothing is kept from the row above
    a = torch.where(first, torch.zeros_like(keep), keep)
    h = _double(a, z * x + (keep - a) * h0[seq], longest)
    out = {"h": h.to(st["xg"].dtype), "h_last": torch.where(some, h[tail], h0)}
    if case["train"]:
        # g_t = dh_t + keep_{t+1} g_{t+1} up to a sequence's end
        dh = st["dh"].float() + torch.where(last, st["dh_last"][seq], torch.zeros_like(h))
        up = torch.cat([a[1:], torch.zeros_like(a[:1])])
        g = _double(up.flip(0), dh.flip(0), longest).flip(0)
        before = torch.where(first, h0[seq], torch.cat([h[:1], h[:-1]]))
        out["dxg"] = torch.cat([g * z, g * (x - before) * z * keep], 1).to(st["xg"].dtype)
        if case["h0"]:
            out["dh0"] = torch.where(some, keep[head] * g[head], st["dh_last"])
    return out


def _plain_muon(st, case):
    R, C = case["R"], case["C"]
    g = st["grad"].float()
    st["momentum"].mul_(MU).add_(g)
    X = g + MU * st["momentum"]
    X = X / (torch.sqrt(X.square().sum()) + NS_EPS)
    a, b, c = NS
    X = X.t() if R > C else X
    for _ in range(NS_STEPS):
        A = X @ X.t()
        X = a * X + (b * A + c * (A @ A)) @ X
    X = X.t() if R > C else X
    st["W"].copy_(st["W"].float() - LR * math.sqrt(max(1.0, R / C)) * X)
    return {"W": st["W"], "momentum": st["momentum"]}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = _inputs(case, seed)
    d = {k: v.double() for k, v in st.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if case["op"] == "xent":
        return _exact_xent(case, st, d)
    if case["op"] == "scan":
        return _exact_scan(case, st, d)
    G, Mo = d["grad"], MU * d["momentum"] + d["grad"]
    O = torch.nn.functional.normalize((G + MU * Mo).reshape(-1), dim=0, eps=NS_EPS).reshape(G.shape)
    for _ in range(NS_STEPS):  # on the shorter side
        if case["R"] <= case["C"]:
            A = O.matmul(O.mT)
            O = NS[0] * O + NS[1] * A.matmul(O) + NS[2] * A.matmul(A.matmul(O))
        else:
            A = O.mT.matmul(O)
            O = NS[0] * O + NS[1] * O.matmul(A) + NS[2] * O.matmul(A).matmul(A)
    return {"W": d["W"] - LR * max(1.0, case["R"] / case["C"]) ** 0.5 * O, "momentum": Mo}


def _exact_xent(case, st, d):
    M, V = case["M"], case["V"]
    W, loss, lse, dx = d["W"], [], [], []
    b = d["b"] if case["bias"] else torch.zeros(V, dtype=torch.float64, device="cuda")
    dW, db = torch.zeros_like(W), torch.zeros_like(b)
    rows = max(1, min(M, 400_000_000 // V))
    for r in range(0, M, rows):  # rows by rows
        x, t = d["x"][r:r + rows], st["target"][r:r + rows]
        logp = torch.log_softmax(torch.addmm(b, x, W.t()), 1)
        keep = (t >= 0).double()
        one = t.clamp_min(0).unsqueeze(1)
        loss.append(-logp.gather(1, one).squeeze(1) * keep)
        lse.append(torch.addmm(b, x, W.t())[:, 0] - logp[:, 0])
        if case["train"]:
            dz = logp.exp_()
            dz.scatter_(1, one, dz.gather(1, one) - 1)
            dz.mul_((keep * d["dloss"][r:r + rows]).unsqueeze(1))
            dx.append(dz.mm(W))
            dW.addmm_(dz.t(), x)
            db.add_(dz.sum(0))
    out = {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    if case["train"]:
        out["dx"], out["dW"] = torch.cat(dx), dW
        if case["bias"]:
            out["db"] = db
    return out


def _exact_scan(case, st, d):
    """Step by step, the sequences that are long enough side by side."""
    B, T, D = case["B"], case["T"], case["D"]
    lengths = torch.full((B,), T // B, device="cuda") if st["lengths"] is None else st["lengths"].long()
    begin = lengths.cumsum(0) - lengths
    by = torch.argsort(lengths, descending=True)
    sizes = lengths[by].tolist()
    if sizes[0] > 131072:
        return None
    x, z = d["xg"][:, :D], torch.sigmoid(d["xg"][:, D:])
    h = torch.empty(T, D, dtype=torch.float64, device="cuda")
    before = torch.empty_like(h)
    state = (d["h0"] if case["h0"] else torch.zeros(B, D, dtype=torch.float64, device="cuda"))[by]
    start, live, counts = begin[by], B, []
    for t in range(sizes[0]):
        while sizes[live - 1] <= t:
            live -= 1
        counts.append(live)
        at, s = start[:live] + t, state[:live]
        before[at] = s
        s.lerp_(x[at], z[at])
        h[at] = s
    back = torch.argsort(by)
    out = {"h": h, "h_last": state[back]}
    if case["train"]:
        g = d["dh_last"][by]  # what reaches a sequence's state behind the row
        for t in range(sizes[0] - 1, -1, -1):
            live = counts[t]
            at, s = start[:live] + t, g[:live]
            s.add_(d["dh"][at])
            h[at] = s
            s.mul_(1 - z[at])
        g_rows = h
        out["h"] = before.clone()
        out["h"] += z * (x - before)
        out["dxg"] = torch.cat([g_rows * z, g_rows * (x - before) * z * (1 - z)], 1)
        if case["h0"]:
            out["dh0"] = g[back]
    return out
