"""The norm's workspace holds all of its partial sums, by the bytes asked for
(CPU), and on the GPU nothing changes behind a workspace of exactly the
stated size."""
import pytest
import torch

import dense_ref as R
from dense_guard import guard
from recsys_sparse_embedding_gb300 import binding as B
from recsys_sparse_embedding_gb300 import build as nbuild

BF16, F32 = torch.bfloat16, torch.float32
SMS = 152
# The norm's backward: threads per row by the row's length (the first border
# that the length does not pass), with an fp32 operand and without.
GROUPS = {True: ((512, 32), (1024, 64), (2048, 128), (4096, 256), (8192, 512), (32768, 1024)),
          False: ((1024, 32), (4096, 128), (8192, 256), (16384, 512), (32768, 1024))}


def partial_rows(M, N, fp32):
    """Rows of N partial sums that the weight gradient's first kernel writes: one
    per block; a block has 256 threads, 8 rows at a time, where a row is a
    warp's, else it is one row's group; as many blocks as 512 threads per SM
    give, or as there are rows."""
    group = next(g for most, g in GROUPS[fp32] if N <= most)
    threads, rows = (256, 8) if group == 32 else (group, 1)
    return max(1, min((M + rows - 1) // rows, SMS * max(1, 512 // threads)))


@pytest.fixture(scope="module")
def L():
    nbuild.build()
    return B.lib()


LENGTHS = sorted({n for t in GROUPS.values() for most, _ in t for n in (most - 1, most, most + 1) if n <= 32768}
                 | {1, 7, 256, 520, 1000})


@pytest.mark.parametrize("N", LENGTHS)
def test_the_norms_workspace_holds_its_partial_sums(L, N):
    last = 0
    for M in list(range(1, 40)) + list(range(40, 1300, 7)) + [303, 304, 305, 608, 609, 1215, 1216, 1217, 2432, 2433, 9999,
                                                              65536, (1 << 31) - 1]:
        need = max(partial_rows(M, N, f) for f in (True, False)) * N * 4
        got = L.dsf_rms_norm_workspace_bytes(M, N)
        assert got >= need, (M, N, got, need)
    for M in (0, 1, 9, 100, 608, 609, 1216, 5000, 1 << 20):
        got = L.dsf_rms_norm_workspace_bytes(M, N)
        assert got >= last  # (a workspace for M rows serves every call of fewer)
        last = got


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(609, 513), (609, 520), (1217, 1000), (8192, 1024), (2000, 1023), (5000, 264), (3000, 512),
                                 (1300, 2048), (1300, 1025), (700, 4096), (700, 8192), (400, 16384), (200, 32768)])
@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_nothing_is_written_behind_the_norms_workspace(M, N, xt, dt):
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N)
    s = torch.randn(M, N, generator=g, device="cuda").to(xt)
    dy = torch.randn(M, N, generator=g, device="cuda").to(dt)
    w = 1 + 0.3 * torch.randn(N, generator=g, device="cuda")
    dx, dw = torch.empty_like(s), torch.empty_like(w)
    ws = B.RmsNormWorkspace(M, N)
    intact = guard(ws)
    B.ctr_rms_norm_bwd(dy, s, dx, weight=w, eps=1e-5, dweight=dw, workspace=ws)
    assert intact()
    rx, tx, rw, tw = R.norm_grads(dy, s, w, 1e-5, None)
    R.assert_within(dx, rx, tx + R.HALF[xt] * (rx.abs() + tx) + 1e-38, "dx")
    R.assert_within(dw, rw, tw, "dweight")
