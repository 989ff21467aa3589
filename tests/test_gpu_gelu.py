"""GELU and SiLU where their values are small, in the dense layer and its
gradient."""
import math

import pytest
import torch

import dense_ref as R
from recsys_sparse_embedding_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def phi_bound(z):
    """Relative bound of Phi(-|z|) as the kernels evaluate it, in units of 2^-24.
    The exponent -z^2 / 2 carries two roundings and its constant's, 2.5 units of
    z^2 / 2, which exp turns into relative ones; exp2 itself 4, the quotient and
    its sum 4 times its weight of at most 2, the polynomial's fit 1 and its
    eight steps' roundings at most 10, two products 2; 32 covers them."""
    return (1.25 * z * z + 32) * 2.0 ** -24


@pytest.mark.parametrize("M,dtype", [(7, F32), (7, BF16), (8192, F32), (8192, BF16)])
def test_gelus_negative_tail(M, dtype):
    """One input reaches each output with weight 1, so z is the input: values
    and slopes of GELU where they are small keep their significant bits."""
    K, N = 64, 136
    z = -torch.linspace(0.01, 12.0, M * K, device="cuda").view(M, K).to(dtype)
    W = torch.zeros(N, K, dtype=dtype, device="cuda")
    W[torch.arange(K), torch.arange(K)] = 1
    layer = B.DenseLayer(W, None, act=B.DSF_ACT_GELU)
    ws = B.DenseWorkspace(layer, M, backward=True)
    y = torch.empty(M, N, dtype=dtype, device="cuda")
    B.ctr_dense_fwd(layer, z, y, ws)
    d = z.double()
    ref = R.act(d, "gelu")
    R.assert_within(y[:, :K], ref, ref.abs() * (phi_bound(d) + R.HALF[dtype]) + 1e-37, "value")
    dx = torch.empty_like(z)
    dy = torch.ones(M, N, dtype=dtype, device="cuda")
    B.ctr_dense_bwd(layer, z, dy, ws, dx=dx)
    # Phi + z phi: two terms of either sign, each with Phi's bound and two roundings more
    cdf, zphi = 0.5 * torch.erfc(-d / math.sqrt(2)), d * torch.exp(-d * d / 2) / math.sqrt(2 * math.pi)
    ref = cdf + zphi
    tol = (cdf + zphi.abs()) * (phi_bound(d) + 2.0 ** -22)
    R.assert_within(dx, ref, tol + (2.02 if dtype == BF16 else 1) * R.HALF[dtype] * (ref.abs() + tol) + 1e-37, "slope")


def sigmoid_bound(z):
    """Relative bound of 1 / (1 + exp(-z)), z < 0, in units of 2^-24: the exponent
    carries a rounding and its constant's, 1.5 units of z; exp2 4, the sum and
    the quotient 4, two products 2; 16 covers them."""
    return (1.5 * z.abs() + 16) * 2.0 ** -24


@pytest.mark.parametrize("M,dtype", [(7, F32), (7, BF16), (8192, F32), (8192, BF16)])
def test_silus_negative_tail(M, dtype):
    K, N = 64, 136
    z = -torch.linspace(0.01, 70.0, M * K, device="cuda").view(M, K).to(dtype)
    W = torch.zeros(N, K, dtype=dtype, device="cuda")
    W[torch.arange(K), torch.arange(K)] = 1
    layer = B.DenseLayer(W, None, act=B.DSF_ACT_SILU)
    ws = B.DenseWorkspace(layer, M, backward=True)
    y = torch.empty(M, N, dtype=dtype, device="cuda")
    B.ctr_dense_fwd(layer, z, y, ws)
    d = z.double()
    ref = R.act(d, "silu")
    R.assert_within(y[:, :K], ref, ref.abs() * (sigmoid_bound(d) + R.HALF[dtype]) + 1e-37, "value")
    dx = torch.empty_like(z)
    dy = torch.ones(M, N, dtype=dtype, device="cuda")
    B.ctr_dense_bwd(layer, z, dy, ws, dx=dx)
    # p + z p (1 - p): two terms of either sign, each with p's bound and three roundings more
    p = torch.sigmoid(d)
    ref = p * (1 + d * (1 - p))
    tol = (p + (d * p).abs()) * (sigmoid_bound(d) + 2.0 ** -22)
    R.assert_within(dx, ref, tol + (2.02 if dtype == BF16 else 1) * R.HALF[dtype] * (ref.abs() + tol) + 1e-37, "slope")
