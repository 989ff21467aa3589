"""Host-side checks of the dense operators' entry points: bad arguments are
refused before any CUDA call (these run without a GPU)."""
import ctypes

import pytest

from recsys_sparse_embedding_gb300 import binding as B
from recsys_sparse_embedding_gb300 import build as nbuild

P = ctypes.byref
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    nbuild.build()
    return B.lib()


def layer(**kw):
    f = dict(W=4096, bias=4096, scale=None, ldw=64, R=32, K=64, dtype=B.DSF_BF16, act=B.DSF_ACT_SILU)
    f.update(kw)
    return B.CDense(*[f[n] for n in ("W", "bias", "scale", "ldw", "R", "K", "dtype", "act")])


BAD_LAYERS = [
    (dict(W=None), B.DSF_EINVAL), (dict(W=4100), B.DSF_EINVAL), (dict(W=4097, K=33, ldw=33), B.DSF_EINVAL),
    (dict(ldw=63), B.DSF_EINVAL), (dict(ldw=65), B.DSF_EINVAL), (dict(bias=4098), B.DSF_EINVAL),
    (dict(scale=4096), B.DSF_EINVAL), (dict(dtype=B.DSF_E4M3), B.DSF_EINVAL), (dict(dtype=3), B.DSF_EUNSUPPORTED),
    (dict(dtype=-1), B.DSF_EUNSUPPORTED), (dict(act=4), B.DSF_EINVAL), (dict(act=-1), B.DSF_EINVAL),
    (dict(R=0), B.DSF_EINVAL), (dict(K=0), B.DSF_EINVAL), (dict(R=(1 << 20) + 1), B.DSF_EINVAL),
    (dict(K=(1 << 20) + 8, ldw=1 << 21), B.DSF_EINVAL)]


@pytest.mark.parametrize("kw,code", BAD_LAYERS)
def test_bad_layers_are_refused(L, kw, code):
    l = layer(**kw)
    assert L.dsf_dense_workspace_bytes(P(l), 4, 0, 0) == 0
    assert L.ctr_dense_fwd(P(l), 4096, 64, None, None, 0, 4, 4096, 32, 4096, BIG, None, None) == code
    assert L.ctr_glu_fwd(P(l), 4096, 64, None, 4, 4096, 32, 4096, BIG, None, None) == code
    assert L.ctr_dense_bwd(P(l), 4096, 64, 4096, 32, 4, 4096, 64, 4096, 4096, 4096, BIG, None, None) == code
    assert L.ctr_glu_bwd(P(l), 4096, 64, 4096, 32, 4, 4096, 64, 4096, 4096, 4096, BIG, None, None) == code


def test_null_layer(L):
    assert L.dsf_dense_workspace_bytes(None, 4, 0, 0) == 0
    assert L.ctr_dense_fwd(None, 4096, 64, None, None, 0, 4, 4096, 32, 4096, BIG, None, None) == B.DSF_EINVAL
    assert L.ctr_glu_bwd(None, 4096, 64, 4096, 32, 4, 4096, 64, 4096, 4096, 4096, BIG, None, None) == B.DSF_EINVAL


def test_workspace_bytes(L):
    l = layer()
    n0, n1 = (L.dsf_dense_workspace_bytes(P(l), 100, 0, b) for b in (0, 1))
    assert 0 < n0 <= n1 and n0 % 256 == 0
    assert L.dsf_dense_workspace_bytes(P(l), 0, 0, 0) > 0
    assert L.dsf_dense_workspace_bytes(P(l), -1, 0, 0) == 0
    assert L.dsf_dense_workspace_bytes(P(l), 1 << 31, 0, 0) == 0
    assert L.dsf_dense_workspace_bytes(P(l), 4, 2, 0) == 0
    assert L.dsf_dense_workspace_bytes(P(layer(R=33)), 4, 1, 0) == 0
    e = layer(dtype=B.DSF_E4M3, scale=4096)
    assert L.dsf_dense_workspace_bytes(P(e), 4, 0, 0) > 0
    assert L.dsf_dense_workspace_bytes(P(e), 4, 0, 1) == 0


def test_fwd_refusals(L):
    def call(l=None, x=4096, ldx=64, xs=None, res=None, ldr=0, M=4, y=4096, ldy=32, ws=4096, nb=BIG):
        return L.ctr_dense_fwd(P(l or layer()), x, ldx, xs, res, ldr, M, y, ldy, ws, nb, None, None)
    assert call(M=0) == B.DSF_OK
    assert call(M=-1) == B.DSF_EINVAL
    assert call(M=1 << 31) == B.DSF_EINVAL
    assert call(x=None) == B.DSF_EINVAL
    assert call(x=4098) == B.DSF_EINVAL
    assert call(ldx=63) == B.DSF_EINVAL
    assert call(ldx=68) == B.DSF_EINVAL  # rows of 128 bytes, not at 16-byte boundaries
    assert call(xs=4096) == B.DSF_EINVAL
    assert call(l=layer(dtype=B.DSF_E4M3, scale=4096)) == B.DSF_EINVAL  # e4m3 without x_scale
    assert call(y=None) == B.DSF_EINVAL
    assert call(y=4097) == B.DSF_EINVAL
    assert call(ldy=31) == B.DSF_EINVAL
    assert call(res=4096, ldr=31) == B.DSF_EINVAL
    assert call(res=4097, ldr=32) == B.DSF_EINVAL
    assert call(ws=None) == B.DSF_EWORKSPACE
    assert call(ws=4096 + 16) == B.DSF_EWORKSPACE
    assert call(nb=0) == B.DSF_EWORKSPACE
    odd = layer(R=33)
    assert L.ctr_glu_fwd(P(odd), 4096, 64, None, 4, 4096, 16, 4096, BIG, None, None) == B.DSF_EINVAL
    assert L.ctr_glu_fwd(P(layer()), 4096, 64, None, 4, 4096, 15, 4096, BIG, None, None) == B.DSF_EINVAL


def test_bwd_refusals(L):
    def call(l=None, x=4096, ldx=64, dy=4096, lddy=32, M=4, dx=4096, lddx=64, dW=4096, db=4096, ws=4096, nb=BIG):
        return L.ctr_dense_bwd(P(l or layer()), x, ldx, dy, lddy, M, dx, lddx, dW, db, ws, nb, None, None)
    assert call(l=layer(dtype=B.DSF_E4M3, scale=4096)) == B.DSF_EUNSUPPORTED
    assert call(M=-1) == B.DSF_EINVAL
    assert call(x=None) == B.DSF_EINVAL
    assert call(dy=None) == B.DSF_EINVAL
    assert call(lddy=31) == B.DSF_EINVAL
    assert call(lddy=36) == B.DSF_EINVAL
    assert call(dx=4097) == B.DSF_EINVAL
    assert call(lddx=63) == B.DSF_EINVAL
    assert call(dW=4097) == B.DSF_EINVAL
    assert call(db=4098) == B.DSF_EINVAL
    assert call(ws=None) == B.DSF_EWORKSPACE
    assert call(nb=L.dsf_dense_workspace_bytes(P(layer()), 4, 0, 1) - 1) == B.DSF_EWORKSPACE


def test_norm_refusals(L):
    def fwd(x=4096, ldx=16, res=None, ldr=0, xd=B.DSF_F32, w=None, M=4, N=16, eps=1e-6, s=None, lds=0, y=4096, ldy=16,
            yd=B.DSF_F32, ys=None):
        return L.ctr_rms_norm_fwd(x, ldx, res, ldr, xd, w, M, N, eps, s, lds, y, ldy, yd, ys, None)
    assert fwd(M=0) == B.DSF_OK
    for kw in (dict(M=-1), dict(M=1 << 31), dict(N=0), dict(eps=0.0), dict(eps=float("nan")), dict(x=None), dict(y=None),
               dict(ldx=15), dict(ldy=15), dict(res=4096, ldr=15), dict(s=4096, lds=15), dict(x=4098), dict(w=4098),
               dict(yd=B.DSF_E4M3), dict(ys=4096)):
        assert fwd(**kw) == B.DSF_EINVAL, kw
    for kw in (dict(N=32769, ldx=1 << 16, ldy=1 << 16), dict(xd=B.DSF_E4M3), dict(yd=3)):
        assert fwd(**kw) == B.DSF_EUNSUPPORTED, kw

    def bwd(dy=4096, lddy=16, dyd=B.DSF_F32, s=4096, lds=16, xd=B.DSF_F32, w=None, M=4, N=16, eps=1e-6, up=None, ldu=0,
            dx=4096, lddx=16, dw=None, ws=None, nb=0):
        return L.ctr_rms_norm_bwd(dy, lddy, dyd, s, lds, xd, w, M, N, eps, up, ldu, dx, lddx, dw, ws, nb, None)
    assert bwd(M=0) == B.DSF_OK
    for kw in (dict(M=-1), dict(N=0), dict(eps=-1.0), dict(dy=None), dict(s=None), dict(dx=None), dict(lddy=15),
               dict(up=4096, ldu=15), dict(dx=4097), dict(dw=4097)):
        assert bwd(**kw) == B.DSF_EINVAL, kw
    assert bwd(dyd=B.DSF_E4M3) == B.DSF_EUNSUPPORTED
    need = L.dsf_rms_norm_workspace_bytes(4, 16)
    assert need > 0 and L.dsf_rms_norm_workspace_bytes(4, 0) == 0 and L.dsf_rms_norm_workspace_bytes(-1, 16) == 0
    assert bwd(dw=4096) == B.DSF_EWORKSPACE
    assert bwd(dw=4096, ws=4096 + 64, nb=need) == B.DSF_EWORKSPACE
    assert bwd(dw=4096, ws=4096, nb=need - 1) == B.DSF_EWORKSPACE


@pytest.mark.parametrize("dtype", [B.DSF_F32, B.DSF_BF16, B.DSF_E4M3])
@pytest.mark.parametrize("gated", [0, 1])
@pytest.mark.parametrize("R,K", [(2, 1), (128, 256), (1366, 256), (300, 45), (8192, 4096)])
def test_workspace_grows_with_the_rows(L, dtype, gated, R, K):
    """A workspace for M rows serves every call of fewer."""
    l = layer(dtype=dtype, R=R, K=K, ldw=K, scale=4096 if dtype == B.DSF_E4M3 else None)
    for back in (0, 1) if dtype != B.DSF_E4M3 else (0,):
        sizes = [L.dsf_dense_workspace_bytes(P(l), M, gated, back) for M in
                 (0, 1, 8, 9, 31, 32, 33, 100, 127, 128, 129, 255, 257, 1000, 4096, 10001, 65536, 1 << 20)]
        assert sizes == sorted(sizes) and sizes[0] > 0
