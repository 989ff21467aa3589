"""The dense-tower operators in 64 bits, and how far a correct fp32-accumulating
evaluation may be from them, element by element.

Bounds. A sum of K products accumulated in fp32, in any order and with each
addition rounded or truncated, is off by at most (K + 8) 2^-23 of the sum of
the terms' absolute values (the 8 covers the operands' own handling: scales,
the bias, and in fp32 the dropped products of bf16 terms, 2^-21 of each
term). An activation's slope is at most 1.13 and its second derivative at most
1 (SiLU: 0.5, GELU: 0.8); its evaluation is off by at most 2^-19 of |z| + 1 (exp
and quotient: 2^-21 each). A rounding to the output's type is off by half a step:
2^-8 (bf16) or 2^-24 (fp32) of the value. In a bf16 backward dz is rounded
once more, half a step of dz. ReLU's derivative may go either way where |z|
lies within z's own bound.
"""
import math

import torch

from recsys_sparse_embedding_gb300 import binding

ACTS = {"none": binding.DSF_ACT_NONE, "relu": binding.DSF_ACT_RELU, "silu": binding.DSF_ACT_SILU,
        "gelu": binding.DSF_ACT_GELU}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -23


def act(z, name):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    return z


def act_grad(z, name):
    if name == "relu":
        return (z > 0).to(z)
    if name == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def pre(x, W, b, xs=None, ws=None):
    """z and the bound of its error; x, W as the layer has them."""
    x, W = x.double(), W.double()
    if xs is not None:
        x, W = x * xs.double()[:, None], W * ws.double()[:, None]
    z, a = x @ W.t(), x.abs() @ W.abs().t()
    if b is not None:
        z, a = z + b.double(), a + b.double().abs()
    return z, (x.shape[1] + 8) * U * a + 1e-38


def dense(x, W, b, name, residual, out, xs=None, ws=None):
    """(y, bound) of the dense layer."""
    z, dz = pre(x, W, b, xs, ws)
    y = act(z, name)
    tol = 1.13 * dz + (0 if name in ("none", "relu") else 2.0 ** -19 * (z.abs() + 1))
    if residual is not None:
        y = y + residual.double()
        tol = tol + U * residual.double().abs()
    return y, tol + HALF[out] * (y.abs() + tol) + 1e-38


def glu(x, W, b, name, out, xs=None, ws=None):
    z, dz = pre(x, W, b, xs, ws)
    F = z.shape[1] // 2
    g, u, eg, eu = z[:, :F], z[:, F:], dz[:, :F], dz[:, F:]
    a = act(g, name)
    ea = 1.13 * eg + 2.0 ** -19 * (g.abs() + 1)
    y = a * u
    tol = ea * u.abs() + a.abs() * eu + ea * eu + 2 * U * y.abs()
    return y, tol + HALF[out] * (y.abs() + tol) + 1e-38


def grads(x, W, b, name, dy, gated):
    """{name: (gradient, bound)} of dx, dW, db."""
    out = x.dtype
    z, ez = pre(x, W, b)
    dy = dy.double()

    def slope(z, ez):  # act' and its bound
        e = ez + 2.0 ** -19 * (z.abs() + 1)
        if name == "none":
            e = torch.zeros_like(z)
        if name == "relu":
            e = (z.abs() <= ez).to(z)
        return act_grad(z, name), e

    if gated:
        F = z.shape[1] // 2
        g, u, eg, eu = z[:, :F], z[:, F:], ez[:, :F], ez[:, F:]
        s, es = slope(g, eg)
        a, ea = act(g, name), 1.13 * eg + 2.0 ** -19 * (g.abs() + 1)
        dz = torch.cat([dy * u * s, dy * a], 1)
        e = torch.cat([dy.abs() * (u.abs() * es + s.abs() * eu + es * eu), dy.abs() * ea], 1)
    else:
        s, es = slope(z, ez)
        dz, e = dy * s, dy.abs() * es
    e = e + 4 * U * dz.abs()
    er = e + (HALF[out] * (dz.abs() + e) if out == torch.bfloat16 else 0)
    xd, Wd = x.double(), W.double()
    M, R = dz.shape

    def product(p, ep, q, n):
        v = p @ q
        t = ep @ q.abs() + (n + 8) * U * ((p.abs() + ep) @ q.abs())
        return v, t + HALF[out] * (v.abs() + t) + 1e-38

    return {"dx": product(dz, er, Wd, R), "dW": product(dz.t(), er.t(), xd, M),
            "db": (dz.sum(0), e.sum(0) + (M + 8) * U * (dz.abs() + e).sum(0) + 1e-38)}


def norm(s, w, eps):
    s = s.double()
    r = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    return s * r * (1 if w is None else w.double()), r


def norm_grads(dy, s, w, eps, dsum):
    s, dy = s.double(), dy.double()
    _, r = norm(s, None, eps)
    g = dy * (1 if w is None else w.double())
    c = (g * s).mean(1, keepdim=True)
    dx = r * (g - s * r * r * c)
    # 2^-23 each: the two row sums (N + 8 terms; r moves by half of its sum's error), r's root and
    # quotient, the products; relative to the terms' sizes
    n = s.shape[1] + 8
    ca = (g * s).abs().mean(1, keepdim=True)
    tol = n * U * (r * g.abs() + 3 * s.abs() * r ** 3 * ca)
    if dsum is not None:
        dx = dx + dsum.double()
        tol = tol + U * dx.abs()
    dw = (dy * s * r).sum(0)
    return dx, tol, dw, (s.shape[0] + n) * U * (dy * s * r).abs().sum(0) + 1e-38


def assert_within(got, ref, tol, what):
    got = got.double()
    err = (got - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), "%s: %d of %d beyond the bound, worst error/bound %.3g" % (
        what, int(bad.sum()), bad.numel(), float((err / tol).nan_to_num(float("inf")).max()))


def assert_norm(got, ref, rel, what, *sizes):
    """2-norm of the error against the reference's: what independent roundings
    leave, far below the elementwise worst case. It is a mean, so it is taken
    only where every size is 48 or more: a lone value's rounding is off by up
    to 2^-8, sqrt 3 times the mean's 2^-8 / sqrt 3, and all of a gradient's
    values share the rounding of dz where a sum has one term."""
    n = float(ref.norm())
    if n and min(sizes) >= 48:
        e = float((got.double() - ref).norm()) / n
        assert e <= rel, "%s: relative 2-norm error %.3g above %.3g" % (what, e, rel)
