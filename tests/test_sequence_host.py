"""Host-side checks of the sequence-tower operators' entry points: bad arguments
are refused before any CUDA call (these run without a GPU)."""
import ctypes

import pytest

from recsys_sparse_embedding_gb300 import binding as B
from recsys_sparse_embedding_gb300 import build as nbuild

P = ctypes.byref
BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    nbuild.build()
    return B.lib()


def layer(**kw):
    f = dict(W=4096, bias=4096, scale=None, ldw=64, R=1000, K=64, dtype=B.DSF_BF16, act=B.DSF_ACT_NONE)
    f.update(kw)
    return B.CDense(*[f[n] for n in ("W", "bias", "scale", "ldw", "R", "K", "dtype", "act")])


@pytest.mark.parametrize("kw,code", [
    (dict(W=None), B.DSF_EINVAL), (dict(W=4100), B.DSF_EINVAL), (dict(ldw=63), B.DSF_EINVAL), (dict(ldw=65), B.DSF_EINVAL),
    (dict(bias=4098), B.DSF_EINVAL), (dict(dtype=B.DSF_E4M3, scale=4096), B.DSF_EUNSUPPORTED), (dict(dtype=7), B.DSF_EUNSUPPORTED),
    (dict(act=B.DSF_ACT_RELU), B.DSF_EINVAL), (dict(R=0), B.DSF_EINVAL), (dict(R=(1 << 20) + 1), B.DSF_EINVAL),
    (dict(K=8200, ldw=8200), B.DSF_EUNSUPPORTED)])
def test_catalogue_layers_are_refused(L, kw, code):
    l = layer(**kw)
    assert L.dsf_softmax_xent_workspace_bytes(P(l), 4, 0) == 0
    assert L.ctr_softmax_xent_fwd(P(l), 4096, 64, 4096, 4, 4096, 4096, 4096, BIG, None, None) == code
    assert L.ctr_softmax_xent_bwd(P(l), 4096, 64, 4096, 4096, None, 4, 4096, 64, 4096, 4096, 4096, BIG, None, None) == code


def test_xent_refusals(L):
    l = layer()

    def fwd(x=4096, ldx=64, t=4096, M=4, loss=4096, lse=4096, ws=4096, nb=BIG):
        return L.ctr_softmax_xent_fwd(P(l), x, ldx, t, M, loss, lse, ws, nb, None, None)
    assert fwd(M=0) == B.DSF_OK
    for kw in (dict(M=-1), dict(M=1 << 31), dict(x=None), dict(x=4098), dict(ldx=63), dict(ldx=68), dict(t=None), dict(t=4100),
               dict(loss=None), dict(loss=4097), dict(lse=None), dict(lse=4098)):
        assert fwd(**kw) == B.DSF_EINVAL, kw
    need = L.dsf_softmax_xent_workspace_bytes(P(l), 4, 0)
    for kw in (dict(ws=None), dict(ws=4096 + 64), dict(nb=need - 1)):
        assert fwd(**kw) == B.DSF_EWORKSPACE, kw

    def bwd(x=4096, ldx=64, t=4096, lse=4096, g=None, M=4, dx=4096, lddx=64, dW=4096, db=4096, ws=4096, nb=BIG):
        return L.ctr_softmax_xent_bwd(P(l), x, ldx, t, lse, g, M, dx, lddx, dW, db, ws, nb, None, None)
    assert bwd(dx=None, dW=None, db=None) == B.DSF_OK
    for kw in (dict(M=-1), dict(x=None), dict(t=None), dict(lse=None), dict(g=4098), dict(dx=4097), dict(lddx=63), dict(dW=4097),
               dict(db=4098)):
        assert bwd(**kw) == B.DSF_EINVAL, kw
    need = L.dsf_softmax_xent_workspace_bytes(P(l), 4, 1)
    for kw in (dict(ws=None), dict(ws=4096 + 64), dict(nb=need - 1)):
        assert bwd(**kw) == B.DSF_EWORKSPACE, kw
    assert L.dsf_softmax_xent_workspace_bytes(P(l), -1, 0) == 0
    assert L.dsf_softmax_xent_workspace_bytes(P(l), 4, 2) == 0


@pytest.mark.parametrize("dtype", [B.DSF_F32, B.DSF_BF16])
@pytest.mark.parametrize("R,K", [(1, 1), (300, 45), (12961, 176), (65536, 1024), (846812, 64), (1 << 20, 128)])
def test_xent_workspace_grows_with_the_rows(L, dtype, R, K):
    """A workspace for M rows serves every call of fewer."""
    l = layer(dtype=dtype, R=R, K=K, ldw=K)
    for back in (0, 1):
        sizes = [L.dsf_softmax_xent_workspace_bytes(P(l), M, back) for M in
                 (0, 1, 4, 5, 31, 100, 127, 129, 255, 511, 513, 1000, 4096, 7937, 8192, 10001, 65536, 65537, 1 << 20)]
        assert sizes == sorted(sizes) and sizes[0] > 0


def test_scan_refusals(L):
    def fwd(x=4096, ldx=16, g=4096, ldg=16, dt=B.DSF_F32, n=None, T=12, nb=3, D=16, h0=None, h=4096, ldh=16, hl=None, ws=4096,
            wb=BIG):
        return L.ctr_gated_scan_fwd(x, ldx, g, ldg, dt, n, T, nb, D, h0, h, ldh, hl, ws, wb, None, None)

    def bwd(dh=4096, lddh=16, x=4096, ldx=16, g=4096, ldg=16, h=4096, ldh=16, dt=B.DSF_F32, n=None, T=12, nb=3, D=16, h0=None,
            dl=None, dx=4096, lddx=16, dg=4096, lddg=16, d0=None, ws=4096, wb=BIG):
        return L.ctr_gated_scan_bwd(dh, lddh, x, ldx, g, ldg, h, ldh, dt, n, T, nb, D, h0, dl, dx, lddx, dg, lddg, d0, ws, wb,
                                    None, None)
    both = (dict(dt=B.DSF_E4M3), B.DSF_EUNSUPPORTED), (dict(T=-1), B.DSF_EINVAL), (dict(T=(1 << 30) + 1), B.DSF_EINVAL), \
        (dict(nb=-1), B.DSF_EINVAL), (dict(D=0), B.DSF_EINVAL), (dict(D=(1 << 20) + 1), B.DSF_EINVAL), \
        (dict(T=13), B.DSF_EINVAL), (dict(n=4098), B.DSF_EINVAL), (dict(x=None), B.DSF_EINVAL), (dict(ldx=15), B.DSF_EINVAL), \
        (dict(g=4097), B.DSF_EINVAL), (dict(ldg=15), B.DSF_EINVAL), (dict(h=None), B.DSF_EINVAL), (dict(ldh=15), B.DSF_EINVAL), \
        (dict(h0=4098), B.DSF_EINVAL), (dict(ws=None), B.DSF_EWORKSPACE), (dict(ws=4096 + 8), B.DSF_EWORKSPACE), \
        (dict(wb=16), B.DSF_EWORKSPACE)
    for kw, code in both:
        assert fwd(**kw) == code and bwd(**kw) == code, kw
    assert fwd(hl=4098) == B.DSF_EINVAL
    for kw in (dict(dh=None), dict(lddh=15), dict(dx=None), dict(lddx=15), dict(dg=4097), dict(lddg=15), dict(dl=4098),
               dict(d0=4098)):
        assert bwd(**kw) == B.DSF_EINVAL, kw
    # no sequences, no rows: nothing to do
    assert fwd(nb=0) == B.DSF_OK and bwd(nb=0) == B.DSF_OK and fwd(T=0, nb=0) == B.DSF_OK
    need = L.dsf_gated_scan_workspace_bytes(12, 3, 16)
    assert fwd(wb=need - 1) == B.DSF_EWORKSPACE and bwd(wb=need - 1) == B.DSF_EWORKSPACE
    assert L.dsf_gated_scan_workspace_bytes(-1, 3, 16) == 0 and L.dsf_gated_scan_workspace_bytes(12, 3, 0) == 0


@pytest.mark.parametrize("D", [1, 16, 37, 48, 64, 100, 1024, 2048])
def test_scan_workspace_grows_with_the_rows(L, D):
    sizes = [L.dsf_gated_scan_workspace_bytes(T, 5, D) for T in (0, 1, 31, 32, 33, 500, 513, 8191, 8193, 131072, 1 << 20)]
    assert sizes == sorted(sizes) and sizes[0] > 0


def test_muon_refusals(L):
    def call(W=4096, ldw=30, wd=B.DSF_F32, g=4096, ldg=30, gd=B.DSF_BF16, m=4096, R=20, C=30, lr=0.02, mu=0.95, wdec=0.0, nest=1,
             steps=5, ws=4096, nb=BIG):
        return L.ctr_muon_update(W, ldw, wd, g, ldg, gd, m, R, C, lr, mu, wdec, nest, steps, ws, nb, None, None)
    for kw in (dict(wd=B.DSF_E4M3), dict(gd=9), dict(R=(1 << 15) + 1, C=1 << 16, ldw=1 << 16, ldg=1 << 16)):
        assert call(**kw) == B.DSF_EUNSUPPORTED, kw
    for kw in (dict(W=None), dict(W=4098), dict(ldw=29), dict(g=None), dict(g=4097), dict(ldg=29), dict(m=None), dict(m=4098),
               dict(R=0), dict(C=-1), dict(R=(1 << 20) + 1), dict(lr=NAN), dict(lr=INF), dict(mu=1.0), dict(mu=-0.5), dict(mu=NAN),
               dict(wdec=-0.1), dict(wdec=INF), dict(nest=2), dict(steps=0), dict(steps=17)):
        assert call(**kw) == B.DSF_EINVAL, kw
    need = L.dsf_muon_workspace_bytes(20, 30)
    for kw in (dict(ws=None), dict(ws=4096 + 128), dict(nb=need - 1)):
        assert call(**kw) == B.DSF_EWORKSPACE, kw
    assert L.dsf_muon_workspace_bytes(0, 4) == 0 and L.dsf_muon_workspace_bytes(1 << 16, 1 << 16) == 0


def test_sizes_beyond_the_limits_are_refused(L):
    """More logits than 2^44, more sequences with lengths than 2^26."""
    l = layer(R=1 << 20, K=8, ldw=8)
    for M, code in ((1 << 24, B.DSF_EWORKSPACE), ((1 << 24) + 1, B.DSF_EUNSUPPORTED)):
        assert L.ctr_softmax_xent_fwd(P(l), 4096, 8, 4096, M, 4096, 4096, 4096, 16, None, None) == code
        assert L.ctr_softmax_xent_bwd(P(l), 4096, 8, 4096, 4096, None, M, 4096, 8, 4096, 4096, 4096, 16, None, None) == code
        for back in (0, 1):
            assert (L.dsf_softmax_xent_workspace_bytes(P(l), M, back) == 0) == (code == B.DSF_EUNSUPPORTED)
    for nb, code in ((1 << 26, B.DSF_EWORKSPACE), ((1 << 26) + 1, B.DSF_EUNSUPPORTED)):
        assert L.ctr_gated_scan_fwd(4096, 16, 4096, 16, B.DSF_F32, 4096, 12, nb, 16, None, 4096, 16, None, 4096, 16, None,
                                    None) == code
        assert L.ctr_gated_scan_bwd(4096, 16, 4096, 16, 4096, 16, 4096, 16, B.DSF_F32, 4096, 12, nb, 16, None, None, 4096, 16,
                                    4096, 16, None, 4096, 16, None, None) == code


def test_scan_workspace_grows_with_the_sequences(L):
    sizes = [L.dsf_gated_scan_workspace_bytes(5000, nb, 33) for nb in (0, 1, 1024, 65536, 65537, 70000, 1 << 20, 1 << 26)]
    assert sizes == sorted(sizes) and sizes[0] > 0
