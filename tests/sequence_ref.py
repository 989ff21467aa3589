"""The sequence-tower operators in 64 bits, and how far a correct fp32
evaluation may be from them, element by element.

Scan. exp is off by at most (2 + 1.5 |g|) 2^-23 of itself (its argument is
rounded), a quotient by 2 2^-23, so z and a by e = (8 + 2 |g|) 2^-23 of
themselves. A state is a sum of products a_t .. a_s z_s x_s; each step adds at
most 3 e of the sum of the terms' absolute values (z, a, the product and the
sum), and composing pairs in blocks and groups adds at most 48 roundings of it.
h is then rounded to its type, half a step: 2^-8 (bf16) or 2^-24 (fp32). The
backward's g is such a sum as well; dgate takes h_{t-1} as it was written.
"""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -23


def recurrence(a, b):
    """y_t = a_t y_{t-1} + b_t down the rows, y_{-1} = 0, by doubling."""
    n = 1
    while n < a.shape[0]:
        b = torch.cat([b[:n], b[n:] + a[n:] * b[:-n]])
        a = torch.cat([torch.zeros_like(a[:n]), a[n:] * a[:-n]])
        n *= 2
    return b


def scan(x, gate, lengths, h0, dh=None, dh_last=None):
    """{name: (value, bound)} of h, h_last and, for dh, dx, dgate, dh0: over
    the rows of the sequences (lengths: a list)."""
    out, dev = x.dtype, x.device
    B, D, T = len(lengths), x.shape[1], sum(lengths)
    n = torch.tensor(lengths, device=dev, dtype=torch.long)
    begin, some = n.cumsum(0) - n, n > 0
    first, last = begin[some], (begin + n - 1)[some]
    X, Gt = x[:T].double(), gate[:T].double()
    Z, Aa = torch.sigmoid(Gt), torch.sigmoid(-Gt)
    e = (8 + 2 * Gt.abs()) * U
    state = torch.zeros(B, D, dtype=torch.float64, device=dev) if h0 is None else h0.double()
    inner = Aa.clone()  # 0 where a sequence begins
    inner[first] = 0

    def add(v, rows, extra):
        v = v.clone()
        v[rows] += extra
        return v

    def before(v, at_first):  # the row above; at a sequence's first row what is given
        v = torch.cat([torch.zeros_like(v[:1]), v[:-1]])[:T]
        v[first] = at_first
        return v

    h = recurrence(inner, add(Z * X, first, Aa[first] * state[some]))
    H = recurrence(inner, add(Z * X.abs(), first, Aa[first] * state[some].abs()))  # of absolute values
    prev, Hprev = before(h, state[some]), before(H, state[some].abs())
    E = recurrence(inner, 3 * e * (Aa * Hprev + Z * X.abs()))
    eh, eprev = E + 48 * U * H, before(E + 48 * U * H, 0)
    tiny = 1e-38

    def states(rows, v, empty):
        r = empty.clone()
        r[some] = v[rows]
        return r

    zero = torch.zeros_like(state)
    ret = {"h": (h, eh + HALF[out] * (h.abs() + eh) + tiny),
           "h_last": (states(last, h, state), states(last, eh, zero) + tiny)}
    if dh is None:
        return ret
    end = zero if dh_last is None else dh_last.double()
    outer = torch.cat([inner[1:], torch.zeros_like(inner[:1])])[:T]  # a_{t+1}; 0 where a sequence ends

    def backwards(b):
        return recurrence(outer.flip(0), b.flip(0)).flip(0)

    d = dh[:T].double()
    g, G = backwards(add(d, last, end[some])), backwards(add(d.abs(), last, end[some].abs()))
    e_next = torch.cat([e[1:], e[:1]])[:T]
    Eg = backwards(U * G + 3 * e_next * (G - add(d.abs(), last, end[some].abs()))) + 48 * U * G
    w = (X - prev) * Z * Aa
    ew = (eprev + HALF[out] * prev.abs()) * Z * Aa + w.abs() * 3 * e + 2 * U * (X.abs() + prev.abs()) * Z * Aa
    if h0 is not None:  # (a sequence's first row takes h0 itself)
        ew[first] -= (HALF[out] * prev.abs() * Z * Aa)[first]

    def rounded(v, t):
        return v, t + HALF[out] * (v.abs() + t) + tiny

    ret["dx"] = rounded(g * Z, Eg * Z + G * Z * 2 * e)
    ret["dgate"] = rounded(g * w, Eg * (w.abs() + ew) + G * ew + 2 * U * G * w.abs())
    ret["dh0"] = (states(first, Aa * g, end), states(first, Aa * (Eg + 3 * e * G), zero) + tiny)
    return ret


def assert_within(got, ref, what):
    v, tol = ref
    err = (got.double() - v).abs()
    bad = ~(err <= tol)
    assert not bad.any(), "%s: %d of %d beyond the bound, worst error/bound %.3g" % (
        what, int(bad.sum()), bad.numel(), float((err / tol).nan_to_num(float("inf")).max()))


def xent(x, W, b, target, dloss=None):
    """{name: (value, bound)} of loss, lse and, with dloss, dx, dW, db, in 64
    bits. A logit is off by at most ez = (K + 8) 2^-23 of the sum of its terms'
    absolute values (as in dense_ref). exp(z - lse) is off by at most ez, what
    lse is off by, 2 2^-23 of |z| + |lse| (the exponent's roundings) and 4 2^-23
    of itself; a sum of V of them by (300 + V / 1024) 2^-23 (256 in a row's lane
    and merge at most, and a 1024th of the columns in a thread's tiles); log by
    2^-22. A bf16 dz is rounded, half a step."""
    out = x.dtype
    there = (target >= 0) & (target < W.shape[0])
    xd, Wd = x.double(), W.double()
    xd = torch.where(there[:, None], xd, torch.zeros_like(xd))
    V, K = W.shape
    z, a = xd @ Wd.t(), xd.abs() @ Wd.abs().t()
    if b is not None:
        z, a = z + b.double(), a + torch.nan_to_num(b.double().abs(), posinf=0.0)
    ez = (K + 8) * U * a
    lse = torch.logsumexp(z, 1)
    p = torch.nan_to_num(torch.exp(z - lse[:, None]))  # (nothing possible: no gradient)
    fin = torch.nan_to_num(z, neginf=0.0).abs()
    ep = ez + 2 * U * (fin + torch.nan_to_num(lse, neginf=0.0).abs()[:, None]) + 4 * U
    elsum = (p * ep).sum(1) + (300 + V / 1024) * U
    el = elsum + 2 * U * torch.nan_to_num(lse, neginf=0.0).abs() + 2 * U
    at = target.clamp(0, V - 1)[:, None]
    zt, et = z.gather(1, at)[:, 0], ez.gather(1, at)[:, 0]
    zero = torch.zeros_like(lse)
    loss = torch.where(there, lse - zt, zero)
    ret = {"lse": (lse, el), "loss": (loss, torch.where(there, el + et + U * loss.abs(), zero) + 1e-38)}
    if dloss is None:
        return ret
    g = torch.where(there & torch.isfinite(lse), dloss.double(), zero)[:, None]
    dz = g * p
    dz.scatter_add_(1, at, -g)
    e = g.abs() * p * (ep + el[:, None]) + 4 * U * dz.abs()
    er = e + (HALF[out] * (dz.abs() + e) if out == torch.bfloat16 else 0)

    def product(q, eq, r, n):
        v = q @ r
        t = eq @ r.abs() + (n + 8) * U * ((q.abs() + eq) @ r.abs())
        return v, t + HALF[out] * (v.abs() + t) + 1e-38

    M = x.shape[0]
    ret["dx"], ret["dW"] = product(dz, er, Wd, V), product(dz.t(), er.t(), xd, M)
    ret["db"] = dz.sum(0), e.sum(0) + (M + 8) * U * (dz.abs() + e).sum(0) + 1e-38
    return ret


NS = (3.4445, -4.7750, 2.0315)


def muon(W, grad, momentum, lr, mu, decay, nesterov, steps):
    """(W, momentum) after a step, in 64 bits."""
    g, m = grad.double(), mu * momentum.double() + grad.double()
    u = g + mu * m if nesterov else m
    X = u / (u.norm() + 1e-7)
    for _ in range(steps):
        if X.shape[0] <= X.shape[1]:
            A = X @ X.t()
            X = NS[0] * X + (NS[1] * A + NS[2] * A @ A) @ X
        else:
            A = X.t() @ X
            X = NS[0] * X + X @ (NS[1] * A + NS[2] * A @ A)
    s = max(1.0, W.shape[0] / W.shape[1]) ** 0.5
    return (1 - lr * decay) * W.double() - lr * s * X, m, lr * s * X
