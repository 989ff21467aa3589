"""The orthogonalised update itself, element by element: from W = 0 the new W is
the update, so no old weight's rounding covers what the products lose.

Bounds. X is taken as 5e-5 of its norm off where W is bf16 (the header promises
7e-5 for any gradient), and as 1e-5 where W is fp32 (a lost cross term or one bf16
term leaves 1 to 3e-2). Errors spread over
the elements unevenly: in 64-bit replays of the two-term products (operands in two
terms, the product of the second ones dropped; 64 x 64 to 1024 x 1024) the largest
is up to 10 times the root mean square's share, so an element may be 16 times that
off, and half a step of its type. Elements below 1/64 of the root mean square are
rounded by at most 2^-14 of it (uniformly: 3.5e-5 in the mean square), which with
5e-5 is 6.1e-5; twice that is allowed, from 128 rows and columns on (as the
replays' 2 to 4e-5 there)."""
import pytest
import torch

import sequence_ref as R
from recsys_sparse_embedding_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
OFF = {BF16: 5e-5, F32: 1e-5}


def gradient(seed, r, c, kind):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return 1e-3 * (rnd(r, 8) @ rnd(8, c) + rnd(r, c) if kind == "directions" else rnd(r, c))


def update(grad, wt, **kw):
    W, m = torch.zeros(grad.shape, dtype=wt, device="cuda"), torch.zeros_like(grad)
    B.ctr_muon_update(W, grad, m, B.MuonWorkspace(W), lr=1.0, **kw)
    zero = torch.zeros_like(grad)
    return W.double(), R.muon(zero, grad, zero, 1.0, 0.95, 0.0, True, kw.get("steps", 5))[0]


def check(W, ref, wt):
    n = ref.numel()
    rms = float(ref.norm()) / n ** 0.5
    err = W - ref
    beyond = err.abs() - R.HALF[wt] * ref.abs()
    assert float(beyond.max()) <= 16 * OFF[wt] * rms, float(beyond.max()) / rms
    if wt is F32:
        assert float(err.norm()) <= 2 * OFF[wt] * float(ref.norm())
        return
    if min(ref.shape) >= 128:
        small = ref.abs() < rms / 64
        e = float(err[small].norm()) / int(small.sum()) ** 0.5
        assert e <= 2 * 6.1e-5 * rms, e / rms


SHAPES = [(64, 64), (64, 176), (176, 64), (129, 1000), (300, 100), (512, 256), (256, 512), (1366, 256), (640, 640), (1000, 136),
          (8192, 72), (20000, 300), (300, 20000), (1024, 1024), (1025, 1101), (1030, 4098), (5000, 1027), (2300, 2310)]


@pytest.mark.parametrize("kind", ["spread", "directions"])
@pytest.mark.parametrize("wt", [BF16, F32])
@pytest.mark.parametrize("r,c", SHAPES)
def test_the_update_alone(r, c, wt, kind):
    W, ref = update(gradient(r + c, r, c, kind), wt)
    check(W, ref, wt)


def grows_to(s, steps):
    """The Frobenius norm of X's error after `steps`, to first order, from its
    singular values s at the start. A step adds 8 2^-24 of its three terms'
    norms; what was there grows at most by L, the largest of |p'| and p / x over
    the singular values' range: the derivative of an odd function of a matrix
    has divided differences of p (mean values of p') and (p(a) + p(b)) / (a + b)
    as its factors."""
    e = 4 * 2.0 ** -24
    a, b, c = R.NS
    for _ in range(steps):
        x = torch.linspace(float(s.min()), float(s.max()), 4096, dtype=torch.float64, device=s.device)
        grow = max(float((a + 3 * b * x ** 2 + 5 * c * x ** 4).abs().max()), float((a + b * x ** 2 + c * x ** 4).abs().max()))
        e = grow * e + 8 * 2.0 ** -24 * float((a * s - b * s ** 3 + c * s ** 5).norm())
        s = a * s + b * s ** 3 + c * s ** 5
    return e


@pytest.mark.parametrize("steps", [1, 3, 9])
@pytest.mark.parametrize("r,c", [(200, 96), (96, 200), (300, 300)])
def test_other_numbers_of_steps(r, c, steps):
    grad = gradient(3, r, c, "spread")
    W, ref = update(grad, F32, steps=steps)
    bound = max(1.0, r / c) ** 0.5 * grows_to(torch.linalg.svdvals((grad / grad.norm()).double()), steps) + 2.0 ** -24 * float(ref.norm())
    assert bound <= 0.02 * float(ref.norm())  # (far below what a step more or less, or a lost term, does)
    assert float((W - ref).norm()) <= bound


@pytest.mark.parametrize("kind", ["spread", "directions"])
@pytest.mark.parametrize("r,c", [(262144, 32), (262145, 64), (1 << 20, 16), (16, 1 << 20), (1 << 20, 100)])
def test_long_sums_in_two_terms(r, c, kind):
    """A sum of one sign (A's diagonal) is low by what the tensor cores truncate
    in one run, which scales X as a whole: its mean scale is to be 1 within the
    5e-5 that X may be off (a half step of every element, of random sign, leaves
    2^-8 / sqrt(elements) of it at most)."""
    W, ref = update(gradient(r + c, r, c, kind), BF16)
    check(W, ref, BF16)
    scale = float((W * ref).sum() / ref.square().sum())
    assert abs(scale - 1) <= OFF[BF16] + 2.0 ** -8 / ref.numel() ** 0.5, scale - 1
