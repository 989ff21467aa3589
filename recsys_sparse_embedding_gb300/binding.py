"""ctypes binding of libdinsparse.so (include/dinsparse.h).

Argument marshalling only: every step of the forward runs in the library's
CUDA kernels. PyTorch supplies device memory and the stream. There is no CPU
fallback: if the library is not built, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdinsparse.so")

DSF_F32, DSF_BF16, DSF_E4M3 = 0, 1, 2
DSF_ACT_NONE, DSF_ACT_RELU, DSF_ACT_SILU, DSF_ACT_GELU = 0, 1, 2, 3
DSF_MODE_BF16_TC, DSF_MODE_FP32 = 0, 1
DSF_OK, DSF_EINVAL, DSF_EUNSUPPORTED, DSF_ECUDA, DSF_EWORKSPACE = 0, 1, 2, 3, 4
FLAG_ID_RANGE = 0x01
FLAG_NEG_LENGTH = 0x02
FLAG_SEQ_TRUNC = 0x04
FLAG_COUNT = 0x08
FLAG_TIMEOUT = 0x10
FLAG_NOT_PREPARED = 0x20
FLAG_HASH = 0x40
FLAG_HASH_FULL = 0x80
FLAG_GRAD_LIST = 0x100

EXPORTS = ["dsf_workspace_bytes", "dsf_workspace_init", "dsf_prepare_mlp", "emb_bag_pool",
           "din_jagged_attn", "din_sparse_fwd", "dsf_status_string", "dsf_grid_size",
           "emb_bag_pool_noalloc", "dsf_towers_workspace_bytes", "dsf_prepare_towers", "ctr_towers_fwd",
           "dsf_hash_workspace_bytes", "dsf_hash_init", "dsf_hash_insert", "dsf_hash_find",
           "dsf_bwd_workspace_bytes", "din_sparse_bwd", "emb_adagrad_update", "dsf_read_status",
           "dsf_bwd_workspace_offsets",
           "dsf_dense_workspace_bytes", "ctr_dense_fwd", "ctr_dense_bwd", "ctr_glu_fwd", "ctr_glu_bwd",
           "dsf_rms_norm_workspace_bytes", "ctr_rms_norm_fwd", "ctr_rms_norm_bwd",
           "dsf_gated_scan_workspace_bytes", "ctr_gated_scan_fwd", "ctr_gated_scan_bwd",
           "dsf_softmax_xent_workspace_bytes", "ctr_softmax_xent_fwd", "ctr_softmax_xent_bwd",
           "dsf_muon_workspace_bytes", "ctr_muon_update"]

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class CHash(ctypes.Structure):
    _fields_ = [("workspace", _vp), ("ws_bytes", _sz), ("capacity", _i64), ("D", _i32), ("dtype", _i32),
                ("key_space", _vp)]


class CMlpGrads(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("dW1", "db1", "dW2", "db2", "dw3", "db3")]


class CRowGrads(ctypes.Structure):
    _fields_ = [("grad", _vp), ("touched", _vp), ("list", _vp), ("count", _vp), ("list_cap", _i64)]


class CTables(ctypes.Structure):
    _fields_ = [("table_ptrs", _vp), ("table_rows", _vp), ("F", _i32), ("D", _i32), ("dtype", _i32),
                ("pooling", _vp), ("hash", _vp)]


class CKjt(ctypes.Structure):
    _fields_ = [("values_dev", _vp), ("n_values", _i64), ("lengths_dev", _vp)]


class CSeq(ctypes.Structure):
    _fields_ = [("values_dev", _vp), ("n_per_key", _i64), ("lengths_dev", _vp), ("max_len", _i32)]


class CMlp(ctypes.Structure):
    _fields_ = [("W1", _vp), ("b1", _vp), ("W2", _vp), ("b2", _vp), ("w3", _vp), ("b3", _vp),
                ("K1", _i32), ("N1", _i32), ("N2", _i32), ("mode", _i32)]


class CDense(ctypes.Structure):
    _fields_ = [("W", _vp), ("bias", _vp), ("scale", _vp), ("ldw", _i64), ("R", _i32), ("K", _i32), ("dtype", _i32),
                ("act", _i32)]


class DsfError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__("%s failed: %s (%d)" % (where, status_string(code), code))


_lib = None


def lib() -> ctypes.CDLL:
    """Loads libdinsparse.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libdinsparse.so is not built (run recsys_sparse_embedding_gb300"
                               ".build.build()); there is no fallback implementation")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER
        L.dsf_workspace_bytes.argtypes = [_i32, _i32]
        L.dsf_workspace_bytes.restype = _sz
        L.dsf_workspace_init.argtypes = [_vp, _sz, _vp]
        L.dsf_workspace_init.restype = ctypes.c_int
        L.dsf_prepare_mlp.argtypes = [P(CMlp), _i32, _vp, _sz, _vp]
        L.dsf_prepare_mlp.restype = ctypes.c_int
        L.emb_bag_pool.argtypes = [P(CTables), P(CKjt), _i32, _vp, _vp, _sz, _vp, _vp]
        L.emb_bag_pool.restype = ctypes.c_int
        L.din_jagged_attn.argtypes = [P(CTables), P(CKjt), P(CSeq), _vp, _vp, _i32, P(CMlp),
                                      _vp, _vp, _vp, _sz, _vp, _vp]
        L.din_jagged_attn.restype = ctypes.c_int
        L.din_sparse_fwd.argtypes = [P(CTables), P(CKjt), P(CSeq), _vp, _vp, _i32, P(CMlp),
                                     _vp, _vp, _vp, _vp, _sz, _vp, _vp]
        L.din_sparse_fwd.restype = ctypes.c_int
        L.dsf_status_string.argtypes = [ctypes.c_int]
        L.dsf_status_string.restype = ctypes.c_char_p
        L.emb_bag_pool_noalloc.argtypes = [P(CTables), P(CKjt), _i32, _vp, _vp, _vp]
        L.emb_bag_pool_noalloc.restype = ctypes.c_int
        L.dsf_grid_size.argtypes = [_i32, _i32, _i32, _i32]
        L.dsf_grid_size.restype = _i32
        L.dsf_towers_workspace_bytes.argtypes = []
        L.dsf_towers_workspace_bytes.restype = _sz
        L.dsf_prepare_towers.argtypes = [P(CTowers), _vp, _sz, _vp]
        L.dsf_prepare_towers.restype = ctypes.c_int
        L.ctr_towers_fwd.argtypes = [_vp, _vp, _i32, P(CTowers), _vp, _vp, _sz, _vp, _vp]
        L.ctr_towers_fwd.restype = ctypes.c_int
        L.dsf_hash_workspace_bytes.argtypes = [_i64, _i32, _i32]
        L.dsf_hash_workspace_bytes.restype = _sz
        L.dsf_hash_init.argtypes = [P(CHash), _vp]
        L.dsf_hash_init.restype = ctypes.c_int
        L.dsf_hash_insert.argtypes = [P(CHash), _i32, _vp, _vp, _i64, _vp, _vp]
        L.dsf_hash_insert.restype = ctypes.c_int
        L.dsf_hash_find.argtypes = [P(CHash), _i32, _vp, _i64, _vp, _vp, _vp]
        L.dsf_hash_find.restype = ctypes.c_int
        L.dsf_bwd_workspace_bytes.argtypes = [_i32, _i64, _i64, _i32]
        L.dsf_bwd_workspace_bytes.restype = _sz
        L.din_sparse_bwd.argtypes = [P(CTables), P(CKjt), P(CSeq), _vp, _vp, _i32, P(CMlp), _vp, _vp, _vp,
                                     P(CMlpGrads), P(CRowGrads), _vp, _sz, _vp, _vp]
        L.din_sparse_bwd.restype = ctypes.c_int
        L.emb_adagrad_update.argtypes = [P(CTables), _vp, P(CRowGrads), ctypes.c_float, ctypes.c_float, _vp, _vp]
        L.emb_adagrad_update.restype = ctypes.c_int
        L.dsf_read_status.argtypes = [_vp, _vp, _vp]
        L.dsf_read_status.restype = ctypes.c_int
        L.dsf_bwd_workspace_offsets.argtypes = [_i32, _i64, _i64, _i32, _vp]
        L.dsf_bwd_workspace_offsets.restype = ctypes.c_int
        L.dsf_dense_workspace_bytes.argtypes = [P(CDense), _i64, _i32, _i32]
        L.dsf_dense_workspace_bytes.restype = _sz
        L.ctr_dense_fwd.argtypes = [P(CDense), _vp, _i64, _vp, _vp, _i64, _i64, _vp, _i64, _vp, _sz, _vp, _vp]
        L.ctr_glu_fwd.argtypes = [P(CDense), _vp, _i64, _vp, _i64, _vp, _i64, _vp, _sz, _vp, _vp]
        for f in (L.ctr_dense_bwd, L.ctr_glu_bwd):
            f.argtypes = [P(CDense), _vp, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _sz, _vp, _vp]
        L.dsf_rms_norm_workspace_bytes.argtypes = [_i64, _i32]
        L.dsf_rms_norm_workspace_bytes.restype = _sz
        L.ctr_rms_norm_fwd.argtypes = [_vp, _i64, _vp, _i64, _i32, _vp, _i64, _i32, ctypes.c_float, _vp, _i64, _vp, _i64,
                                       _i32, _vp, _vp]
        L.ctr_rms_norm_bwd.argtypes = [_vp, _i64, _i32, _vp, _i64, _i32, _vp, _i64, _i32, ctypes.c_float, _vp, _i64, _vp,
                                       _i64, _vp, _vp, _sz, _vp]
        for f in (L.ctr_dense_fwd, L.ctr_glu_fwd, L.ctr_dense_bwd, L.ctr_glu_bwd, L.ctr_rms_norm_fwd,
                  L.ctr_rms_norm_bwd):
            f.restype = ctypes.c_int
        L.dsf_gated_scan_workspace_bytes.argtypes = [_i64, _i32, _i32]
        L.dsf_gated_scan_workspace_bytes.restype = _sz
        L.ctr_gated_scan_fwd.argtypes = [_vp, _i64, _vp, _i64, _i32, _vp, _i64, _i32, _i32, _vp, _vp, _i64, _vp, _vp, _sz,
                                         _vp, _vp]
        L.ctr_gated_scan_bwd.argtypes = [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _i64, _i32, _i32, _vp, _vp,
                                         _vp, _i64, _vp, _i64, _vp, _vp, _sz, _vp, _vp]
        for f in (L.ctr_gated_scan_fwd, L.ctr_gated_scan_bwd):
            f.restype = ctypes.c_int
        L.dsf_softmax_xent_workspace_bytes.argtypes = [P(CDense), _i64, _i32]
        L.dsf_softmax_xent_workspace_bytes.restype = _sz
        L.ctr_softmax_xent_fwd.argtypes = [P(CDense), _vp, _i64, _vp, _i64, _vp, _vp, _vp, _sz, _vp, _vp]
        L.ctr_softmax_xent_bwd.argtypes = [P(CDense), _vp, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _sz, _vp,
                                           _vp]
        for f in (L.ctr_softmax_xent_fwd, L.ctr_softmax_xent_bwd):
            f.restype = ctypes.c_int
        L.dsf_muon_workspace_bytes.argtypes = [_i32, _i32]
        L.dsf_muon_workspace_bytes.restype = _sz
        L.ctr_muon_update.argtypes = [_vp, _i64, _i32, _vp, _i64, _i32, _vp, _i32, _i32, ctypes.c_float, ctypes.c_float,
                                      ctypes.c_float, _i32, _i32, _vp, _sz, _vp, _vp]
        L.ctr_muon_update.restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().dsf_status_string(int(code)).decode()


def read_status(status, stream=None) -> int:
    """The DSF_FLAG_* bits in a device status word, once the work queued on
    the stream so far has finished (dsf_read_status)."""
    out = ctypes.c_int32(0)
    _check(lib().dsf_read_status(_dptr(status), ctypes.byref(out), _stream_ptr(stream)), "dsf_read_status")
    return int(out.value)


def _check(rc: int, where: str) -> None:
    if rc != DSF_OK:
        raise DsfError(rc, where)


def _stream_ptr(stream) -> Optional[int]:
    if stream is None:  # (the current stream's handle without a Stream object: a third of a small call's time)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


class EmbeddingTables:
    """F device tables [rows_f, D], all fp32 or all bf16. pooling: per table
    DSF_POOL_SUM or DSF_POOL_MEAN (None: all sum)."""

    def __init__(self, tables: Sequence[torch.Tensor], pooling: Optional[Sequence[int]] = None,
                 hash_table: Optional["HashTable"] = None):
        self.tables = list(tables)
        self.hash = hash_table
        F = len(self.tables)
        D = int(self.tables[0].shape[1])
        dt = self.tables[0].dtype
        for t in self.tables:
            if t.dim() != 2 or int(t.shape[1]) != D or t.dtype != dt or not t.is_contiguous():
                raise ValueError("tables must be contiguous [rows, D] with one D and dtype")
        self.F, self.D = F, D
        self.dtype = DSF_BF16 if dt == torch.bfloat16 else DSF_F32
        self._ptrs = (ctypes.c_void_p * F)(*[t.data_ptr() for t in self.tables])
        self._rows = (ctypes.c_int64 * F)(*[int(t.shape[0]) for t in self.tables])
        self.pooling = None if pooling is None else [int(x) for x in pooling]
        if self.pooling is not None and len(self.pooling) != F:
            raise ValueError("pooling needs one mode per table")
        self._pool = None if self.pooling is None else (ctypes.c_int32 * F)(*self.pooling)
        self.c = CTables(ctypes.cast(self._ptrs, _vp), ctypes.cast(self._rows, _vp), F, D, self.dtype,
                         None if self._pool is None else ctypes.cast(self._pool, _vp),
                         None if hash_table is None else ctypes.cast(ctypes.pointer(hash_table.c), _vp))
        if hash_table is not None and len(hash_table.key_space) != F:
            raise ValueError("the hash table needs one key space entry per table")

    @property
    def rows(self):
        return [int(t.shape[0]) for t in self.tables]


class AttnMLP:
    """Device fp32 attention MLP in Linear [out, in] layout."""

    def __init__(self, W1, b1, W2, b2, w3, b3, mode: int = DSF_MODE_BF16_TC):
        self.t = [x.contiguous() for x in (W1, b1, W2, b2, w3.reshape(-1), b3.reshape(-1))]
        W1, b1, W2, b2, w3, b3 = self.t
        self.mode = int(mode)
        self.c = CMlp(W1.data_ptr(), b1.data_ptr(), W2.data_ptr(), b2.data_ptr(), w3.data_ptr(),
                      b3.data_ptr(), int(W1.shape[1]), int(W1.shape[0]), int(W2.shape[0]), self.mode)

    def with_mode(self, mode: int) -> "AttnMLP":
        return AttnMLP(*self.t, mode=mode)


class Workspace:
    """Caller-owned scratch for one stream: grid-barrier state, per-CTA partial
    sums, packed MLP weights and the query buffer."""

    def __init__(self, B: int, D: int, device=None, stream=None):
        n = int(lib().dsf_workspace_bytes(int(B), int(D)))
        if n == 0:
            raise DsfError(DSF_EUNSUPPORTED, "dsf_workspace_bytes")
        self.B, self.D, self.nbytes = int(B), int(D), n
        self.buf = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
        _check(lib().dsf_workspace_init(self.buf.data_ptr(), n, _stream_ptr(stream)),
               "dsf_workspace_init")

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()

    def prepare(self, mlp: AttnMLP, stream=None) -> None:
        _check(lib().dsf_prepare_mlp(ctypes.byref(mlp.c), self.D, self.ptr, self.nbytes,
                                     _stream_ptr(stream)), "dsf_prepare_mlp")


def _kjt(values: torch.Tensor, lengths: torch.Tensor) -> CKjt:
    return CKjt(values.data_ptr(), int(values.numel()), lengths.data_ptr())


def _seq(seq_values: torch.Tensor, seq_lengths: torch.Tensor, max_len: int) -> CSeq:
    n = int(seq_values.shape[-1]) if seq_values.dim() == 2 else int(seq_values.numel()) // 3
    return CSeq(seq_values.data_ptr(), n, seq_lengths.data_ptr(), int(max_len))


def _i3(x) -> ctypes.Array:
    return (ctypes.c_int32 * 3)(*[int(v) for v in x])


def emb_bag_pool(tables: EmbeddingTables, values: torch.Tensor, lengths: torch.Tensor, B: int,
                 pooled: torch.Tensor, workspace: Workspace, status: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    kjt = _kjt(values, lengths)
    _check(lib().emb_bag_pool(ctypes.byref(tables.c), ctypes.byref(kjt), int(B), pooled.data_ptr(),
                              workspace.ptr, workspace.nbytes, _dptr(status), _stream_ptr(stream)),
           "emb_bag_pool")
    return pooled


def emb_bag_pool_noalloc(tables: EmbeddingTables, values: torch.Tensor, lengths: torch.Tensor,
                         B: int, pooled: torch.Tensor, status: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """emb_bag_pool without a workspace, for callers that cannot allocate
    device memory; its scratch is a fixed array inside the library."""
    kjt = _kjt(values, lengths)
    _check(lib().emb_bag_pool_noalloc(ctypes.byref(tables.c), ctypes.byref(kjt), int(B),
                                      pooled.data_ptr(), _dptr(status), _stream_ptr(stream)),
           "emb_bag_pool_noalloc")
    return pooled


def din_jagged_attn(tables: EmbeddingTables, values: torch.Tensor, lengths: torch.Tensor,
                    seq_values: torch.Tensor, seq_lengths: torch.Tensor, max_len: int,
                    q_feat, seq_table, B: int, mlp: AttnMLP, din: torch.Tensor,
                    workspace: Workspace, logits: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    kjt, seq = _kjt(values, lengths), _seq(seq_values, seq_lengths, max_len)
    qf, st = _i3(q_feat), _i3(seq_table)
    _check(lib().din_jagged_attn(ctypes.byref(tables.c), ctypes.byref(kjt), ctypes.byref(seq),
                                 ctypes.cast(qf, _vp), ctypes.cast(st, _vp), int(B),
                                 ctypes.byref(mlp.c), din.data_ptr(), _dptr(logits), workspace.ptr,
                                 workspace.nbytes, _dptr(status), _stream_ptr(stream)),
           "din_jagged_attn")
    return din


def din_sparse_fwd(tables: EmbeddingTables, values: torch.Tensor, lengths: torch.Tensor,
                   seq_values: torch.Tensor, seq_lengths: torch.Tensor, max_len: int,
                   q_feat, seq_table, B: int, mlp: AttnMLP, pooled: torch.Tensor,
                   din: torch.Tensor, workspace: Workspace, logits: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream=None):
    kjt, seq = _kjt(values, lengths), _seq(seq_values, seq_lengths, max_len)
    qf, st = _i3(q_feat), _i3(seq_table)
    _check(lib().din_sparse_fwd(ctypes.byref(tables.c), ctypes.byref(kjt), ctypes.byref(seq),
                                ctypes.cast(qf, _vp), ctypes.cast(st, _vp), int(B),
                                ctypes.byref(mlp.c), pooled.data_ptr(), din.data_ptr(),
                                _dptr(logits), workspace.ptr, workspace.nbytes, _dptr(status),
                                _stream_ptr(stream)),
           "din_sparse_fwd")
    return pooled, din


def grid_size(D: int, dtype: int, mode: int, with_attention: bool) -> int:
    return int(lib().dsf_grid_size(int(D), int(dtype), int(mode), int(bool(with_attention))))


class CTowers(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("Wd1", "bd1", "Wd2", "bd2", "Wd3", "bd3", "Wf1", "bf1", "wo", "bo")]


class Towers:
    """The dense towers' device fp32 weights ([out, in]) and their packed
    workspace. Wd1 [512, 256], bd1 [512], Wd2 [256, 512], bd2 [256],
    Wd3 [128, 256], bd3 [128], Wf1 [64, 176], bf1 [64], wo [64], bo [1]."""

    NAMES = ("Wd1", "bd1", "Wd2", "bd2", "Wd3", "bd3", "Wf1", "bf1", "wo", "bo")

    def __init__(self, weights: Sequence[torch.Tensor], device="cuda"):
        self.w = [torch.as_tensor(t, dtype=torch.float32, device=device).contiguous() for t in weights]
        if len(self.w) != len(self.NAMES):
            raise ValueError("towers need %d weight tensors" % len(self.NAMES))
        self.c = CTowers(*[t.data_ptr() for t in self.w])
        self.nbytes = int(lib().dsf_towers_workspace_bytes())
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)

    def prepare(self, stream=None):
        _check(lib().dsf_prepare_towers(ctypes.byref(self.c), self.buf.data_ptr(), self.nbytes,
                                        _stream_ptr(stream)), "dsf_prepare_towers")


def ctr_towers_fwd(pooled: torch.Tensor, din: torch.Tensor, B: int, towers: Towers,
                   logit: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None):
    _check(lib().ctr_towers_fwd(pooled.data_ptr(), din.data_ptr(), int(B), ctypes.byref(towers.c),
                                logit.data_ptr(), towers.buf.data_ptr(), towers.nbytes,
                                _dptr(status), _stream_ptr(stream)), "ctr_towers_fwd")
    return logit


class HashTable:
    """Hash-table storage (one device workspace) for the tables whose
    key_space[f] >= 0: raw int64 keys in [0, 2^56) map to rows of one fused
    pool; an unseen key reads zero. capacity: the minimum slot count."""

    def __init__(self, capacity: int, D: int, dtype: int, key_space: Sequence[int], device="cuda",
                 stream=None):
        self.key_space = [int(k) for k in key_space]
        self._ks = (ctypes.c_int32 * len(self.key_space))(*self.key_space)
        self.nbytes = int(lib().dsf_hash_workspace_bytes(int(capacity), int(D), int(dtype)))
        if self.nbytes == 0:
            raise DsfError(DSF_EINVAL, "dsf_hash_workspace_bytes")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        self.c = CHash(self.buf.data_ptr(), self.nbytes, int(capacity), int(D), int(dtype),
                       ctypes.cast(self._ks, _vp))
        _check(lib().dsf_hash_init(ctypes.byref(self.c), _stream_ptr(stream)), "dsf_hash_init")

    def insert(self, key_space: int, keys: torch.Tensor, rows: torch.Tensor,
               status: Optional[torch.Tensor] = None, stream=None):
        keys = keys.contiguous()
        rows = rows.contiguous()
        _check(lib().dsf_hash_insert(ctypes.byref(self.c), int(key_space), keys.data_ptr(), rows.data_ptr(),
                                     int(keys.numel()), _dptr(status), _stream_ptr(stream)),
               "dsf_hash_insert")

    def find(self, key_space: int, keys: torch.Tensor, status: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
        keys = keys.contiguous()
        out = torch.empty_like(keys)
        _check(lib().dsf_hash_find(ctypes.byref(self.c), int(key_space), keys.data_ptr(), int(keys.numel()),
                                   out.data_ptr(), _dptr(status), _stream_ptr(stream)), "dsf_hash_find")
        return out


class MlpGrads:
    """Device fp32 gradients of the attention MLP (overwritten by a backward
    call): dW1 [256, 12D], db1 [256], dW2 [64, 256], db2 [64], dw3 [64], db3 [1]."""

    def __init__(self, D: int, device="cuda"):
        K1 = 12 * D
        self.t = dict(dW1=torch.zeros(256, K1, device=device), db1=torch.zeros(256, device=device),
                      dW2=torch.zeros(64, 256, device=device), db2=torch.zeros(64, device=device),
                      dw3=torch.zeros(64, device=device), db3=torch.zeros(1, device=device))
        self.c = CMlpGrads(*[self.t[n].data_ptr() for n in ("dW1", "db1", "dW2", "db2", "dw3", "db3")])

    def __getitem__(self, k):
        return self.t[k]


class SparseState:
    """Per-storage row-gradient buffers, touched flags and AdaGrad
    accumulators for a set of tables: one [rows, D] / [rows] set per plain
    table, and one for the hash pool shared by the hash-table tables; the
    touched-row list holds list_cap entries."""

    def __init__(self, tables: EmbeddingTables, list_cap: int, device="cuda", accum_init: float = 0.0):
        F, D = tables.F, tables.D
        ks = tables.hash.key_space if tables.hash is not None else [-1] * F
        pool_rows = None
        if tables.hash is not None:
            pool_rows = (self._pool_rows(tables.hash))
        first = next((f for f in range(F) if ks[f] >= 0), None)
        self.grad, self.touched, self.accum = [], [], []
        for f in range(F):
            if ks[f] >= 0 and f != first:
                self.grad.append(self.grad[first])
                self.touched.append(self.touched[first])
                self.accum.append(self.accum[first])
                continue
            n = pool_rows if ks[f] >= 0 else int(tables.tables[f].shape[0])
            self.grad.append(torch.zeros(n, D, device=device))
            self.touched.append(torch.zeros(n, dtype=torch.int32, device=device))
            self.accum.append(torch.full((n, D), float(accum_init), device=device))
        self.list = torch.zeros(max(1, int(list_cap)), dtype=torch.int64, device=device)
        self.count = torch.zeros(1, dtype=torch.int32, device=device)
        self._g = (_vp * F)(*[t.data_ptr() for t in self.grad])
        self._t = (_vp * F)(*[t.data_ptr() for t in self.touched])
        self._a = (_vp * F)(*[t.data_ptr() for t in self.accum])
        self.c = CRowGrads(ctypes.cast(self._g, _vp), ctypes.cast(self._t, _vp), self.list.data_ptr(),
                           self.count.data_ptr(), int(list_cap))

    @staticmethod
    def _pool_rows(ht: "HashTable") -> int:
        slots = 8
        while slots < ht.c.capacity:
            slots *= 2
        return slots + 1

    @property
    def accum_ptrs(self):
        return ctypes.cast(self._a, _vp)


class BwdWorkspace:
    def __init__(self, B: int, n_values: int, n_per_key: int, D: int, device="cuda"):
        self.nbytes = int(lib().dsf_bwd_workspace_bytes(int(B), int(n_values), int(n_per_key), int(D)))
        if self.nbytes == 0:
            raise DsfError(DSF_EINVAL, "dsf_bwd_workspace_bytes")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        off = (ctypes.c_int64 * 6)()
        _check(lib().dsf_bwd_workspace_offsets(int(B), int(n_values), int(n_per_key), int(D),
                                               ctypes.cast(off, _vp)), "dsf_bwd_workspace_offsets")
        self.offsets = list(off)
        self.D = int(D)

    def views(self, P: int, bf16: bool):
        """The intermediates the last din_sparse_bwd left in this workspace,
        over the first P positions: x, h1, h2 (h1 W2^T), dh2, g (dh2 W2),
        dh1, as tensors viewing the buffer."""
        K1 = 12 * self.D
        op = torch.bfloat16 if bf16 else torch.float32
        out = {}
        for i, (name, width, dt) in enumerate((("x", K1, op), ("h1", 256, op), ("h2", 64, torch.float32),
                                               ("dh2", 64, op), ("g", 256, torch.float32), ("dh1", 256, op))):
            es = 2 if dt == torch.bfloat16 else 4
            o = self.offsets[i]
            out[name] = self.buf[o:o + P * width * es].view(dt).view(P, width)
        return out


def din_sparse_bwd(tables: EmbeddingTables, values, lengths, seq_values, seq_lengths, max_len: int, q_feat,
                   seq_table, B: int, mlp: AttnMLP, pooled, dpooled, ddin, grads: MlpGrads,
                   state: SparseState, ws: BwdWorkspace, status=None, stream=None):
    kjt = _kjt(values, lengths)
    seq = _seq(seq_values, seq_lengths, max_len)
    qf = (ctypes.c_int32 * 3)(*q_feat)
    st = (ctypes.c_int32 * 3)(*seq_table)
    _check(lib().din_sparse_bwd(ctypes.byref(tables.c), ctypes.byref(kjt), ctypes.byref(seq),
                                ctypes.cast(qf, _vp), ctypes.cast(st, _vp), int(B), ctypes.byref(mlp.c),
                                pooled.data_ptr(), _dptr(dpooled), ddin.data_ptr(), ctypes.byref(grads.c),
                                ctypes.byref(state.c), ws.buf.data_ptr(), ws.nbytes, _dptr(status),
                                _stream_ptr(stream)), "din_sparse_bwd")


def emb_adagrad_update(tables: EmbeddingTables, state: SparseState, lr: float = 1e-3, eps: float = 1e-10,
                       status=None, stream=None):
    _check(lib().emb_adagrad_update(ctypes.byref(tables.c), state.accum_ptrs, ctypes.byref(state.c),
                                    float(lr), float(eps), _dptr(status), _stream_ptr(stream)),
           "emb_adagrad_update")


# ------------------------------------------------------------- dense-tower operators
_DTYPES = {torch.float32: DSF_F32, torch.bfloat16: DSF_BF16, torch.float8_e4m3fn: DSF_E4M3}


def _mat(name: str, t: torch.Tensor, dtype, rows: int, cols: int, dev: int):
    """Pointer and row stride of a [rows, cols] matrix on device dev whose
    columns are contiguous; raises ValueError for anything else."""
    if t.dtype is not dtype or t.shape != (rows, cols) or t.get_device() != dev:
        raise ValueError("%s: %s [%d, %d] on cuda:%d expected, got %s %s on %s" % (
            name, dtype, rows, cols, dev, t.dtype, list(t.shape), t.device))
    ld, one = t.stride()
    if rows <= 1:
        ld = cols
    elif ld < cols:
        raise ValueError("%s: rows overlap" % name)
    if one != 1 and cols > 1 and rows > 0:
        raise ValueError("%s: columns must be contiguous" % name)
    return t.data_ptr(), ld


def _vec(name: str, t: Optional[torch.Tensor], n: int, dev: int) -> Optional[int]:
    """Pointer of a contiguous fp32 [n] vector (None for None)."""
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.shape != (n,) or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("%s: contiguous float32 [%d] on cuda:%d expected" % (name, n, dev))
    return t.data_ptr()


def _dev_of(t: torch.Tensor) -> int:
    """The tensor's CUDA device index, which has to be the current device's:
    the calls launch there."""
    dev = t.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError("a tensor on %s, but the current device is cuda:%d" % (t.device, torch.cuda.current_device()))
    return dev


def _on(dev: int, stream) -> Optional[int]:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream_ptr(stream)


class DenseLayer:
    """Device weights of a dense layer (W [N, K]) or a gated layer (W [2F, K]:
    the gate rows, then the up rows): float32, bfloat16, or float8_e4m3fn with
    scale float32 [rows]. bias: float32 [rows] or None. act: DSF_ACT_*."""

    def __init__(self, W: torch.Tensor, bias: Optional[torch.Tensor] = None, act: int = DSF_ACT_NONE,
                 scale: Optional[torch.Tensor] = None):
        if W.dim() != 2 or W.dtype not in _DTYPES:
            raise ValueError("W: a float32, bfloat16 or float8_e4m3fn matrix expected")
        R, K = int(W.shape[0]), int(W.shape[1])
        self.dtype, self.type = _DTYPES[W.dtype], W.dtype
        self.dev = W.get_device()
        if self.dev < 0:
            raise ValueError("W: a CUDA tensor expected")
        ptr, ldw = _mat("W", W, W.dtype, R, K, self.dev)
        if (scale is not None) != (self.dtype == DSF_E4M3):
            raise ValueError("scale: given for float8_e4m3fn weights, and only for them")
        self.W, self.bias, self.scale, self.R, self.K, self.act = W, bias, scale, R, K, int(act)
        self.out_dtype = torch.bfloat16 if self.dtype == DSF_E4M3 else W.dtype
        self.c = CDense(ptr, _vec("bias", bias, R, self.dev), _vec("scale", scale, R, self.dev), ldw, R, K, self.dtype,
                        self.act)
        self._ref = ctypes.byref(self.c)

    @property
    def device(self):
        return self.W.device


class DenseWorkspace:
    """Scratch of a layer's calls for up to M rows; gated: for ctr_glu_*;
    backward: for the gradients too."""

    def __init__(self, layer: DenseLayer, M: int, gated: bool = False, backward: bool = False):
        self.nbytes = int(lib().dsf_dense_workspace_bytes(layer._ref, int(M), int(bool(gated)), int(bool(backward))))
        if self.nbytes == 0:
            raise DsfError(DSF_EINVAL, "dsf_dense_workspace_bytes")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=layer.device)
        self.ptr, self.dev = self.buf.data_ptr(), layer.dev


def _x_of(layer: DenseLayer, x: torch.Tensor, workspace: DenseWorkspace):
    dev = layer.dev
    if dev != torch.cuda.current_device() or workspace.dev != dev:
        raise ValueError("the layer is on cuda:%d, the workspace on cuda:%d, and the current device is cuda:%d" % (
            dev, workspace.dev, torch.cuda.current_device()))
    M = x.shape[0] if x.dim() == 2 else -1
    return dev, M, _mat("x", x, layer.type, M, layer.K, dev)


def _scale_of(layer: DenseLayer, x_scale, M: int):
    if (x_scale is not None) != (layer.dtype == DSF_E4M3):
        raise ValueError("x_scale: given for float8_e4m3fn layers, and only for them")
    return _vec("x_scale", x_scale, M, layer.dev)


def ctr_dense_fwd(layer: DenseLayer, x: torch.Tensor, y: torch.Tensor, workspace: DenseWorkspace,
                  residual: Optional[torch.Tensor] = None, x_scale: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y [M, N] = residual + act(x W^T + bias); y may be the residual."""
    dev, M, (xp, ldx) = _x_of(layer, x, workspace)
    yp, ldy = _mat("y", y, layer.out_dtype, M, layer.R, dev)
    rp, ldr = (None, 0) if residual is None else _mat("residual", residual, layer.out_dtype, M, layer.R, dev)
    _check(lib().ctr_dense_fwd(layer._ref, xp, ldx, _scale_of(layer, x_scale, M), rp, ldr, M, yp, ldy, workspace.ptr,
                               workspace.nbytes, _dptr(status), _on(dev, stream)), "ctr_dense_fwd")
    return y


def ctr_glu_fwd(layer: DenseLayer, x: torch.Tensor, h: torch.Tensor, workspace: DenseWorkspace,
                x_scale: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """h [M, F] = act(x Wg^T + bg) * (x Wu^T + bu), W = [Wg; Wu]."""
    dev, M, (xp, ldx) = _x_of(layer, x, workspace)
    hp, ldh = _mat("h", h, layer.out_dtype, M, layer.R // 2, dev)
    _check(lib().ctr_glu_fwd(layer._ref, xp, ldx, _scale_of(layer, x_scale, M), M, hp, ldh, workspace.ptr,
                             workspace.nbytes, _dptr(status), _on(dev, stream)), "ctr_glu_fwd")
    return h


def _layer_bwd(name, layer, x, dy, cols, workspace, dx, dW, db, status, stream):
    dev, M, (xp, ldx) = _x_of(layer, x, workspace)
    T = layer.type
    gp, ldg = _mat("the upstream gradient", dy, T, M, cols, dev)
    dxp, lddx = (None, 0) if dx is None else _mat("dx", dx, T, M, layer.K, dev)
    dWp = None
    if dW is not None:
        dWp, _ = _mat("dW", dW, T, layer.R, layer.K, dev)
        if not dW.is_contiguous():
            raise ValueError("dW: contiguous expected")
    _check(getattr(lib(), name)(layer._ref, xp, ldx, gp, ldg, M, dxp, lddx, dWp, _vec("db", db, layer.R, dev),
                                workspace.ptr, workspace.nbytes, _dptr(status), _on(dev, stream)), name)


def ctr_dense_bwd(layer: DenseLayer, x: torch.Tensor, dy: torch.Tensor, workspace: DenseWorkspace,
                  dx: Optional[torch.Tensor] = None, dW: Optional[torch.Tensor] = None,
                  db: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of ctr_dense_fwd for dy [M, N], each overwritten where given
    (the residual's gradient is dy itself)."""
    _layer_bwd("ctr_dense_bwd", layer, x, dy, layer.R, workspace, dx, dW, db, status, stream)


def ctr_glu_bwd(layer: DenseLayer, x: torch.Tensor, dh: torch.Tensor, workspace: DenseWorkspace,
                dx: Optional[torch.Tensor] = None, dW: Optional[torch.Tensor] = None,
                db: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of ctr_glu_fwd for dh [M, F]."""
    _layer_bwd("ctr_glu_bwd", layer, x, dh, layer.R // 2, workspace, dx, dW, db, status, stream)


class RmsNormWorkspace:
    """Scratch of ctr_rms_norm_bwd's weight gradient for up to M rows of N."""

    def __init__(self, M: int, N: int, device="cuda"):
        self.nbytes = int(lib().dsf_rms_norm_workspace_bytes(int(M), int(N)))
        if self.nbytes == 0:
            raise DsfError(DSF_EINVAL, "dsf_rms_norm_workspace_bytes")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        self.ptr, self.dev = self.buf.data_ptr(), self.buf.get_device()


def ctr_rms_norm_fwd(x: torch.Tensor, y: torch.Tensor, weight: Optional[torch.Tensor] = None,
                     residual: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
                     eps: float = 1e-6, y_scale: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """s = x + residual (into sum_out where given), y = s * weight /
    sqrt(mean(s^2) + eps); y float32, bfloat16, or float8_e4m3fn with y_scale."""
    dev, xt, yt = _dev_of(x), x.dtype, y.dtype
    if x.dim() != 2 or xt not in _DTYPES or yt not in _DTYPES:
        raise ValueError("x and y: matrices of a supported type expected")
    M, N = x.shape
    xp, ldx = _mat("x", x, xt, M, N, dev)
    yp, ldy = _mat("y", y, yt, M, N, dev)
    rp, ldr = (None, 0) if residual is None else _mat("residual", residual, xt, M, N, dev)
    sp, lds = (None, 0) if sum_out is None else _mat("sum_out", sum_out, xt, M, N, dev)
    _check(lib().ctr_rms_norm_fwd(xp, ldx, rp, ldr, _DTYPES[xt], _vec("weight", weight, N, dev), M, N, eps, sp, lds, yp,
                                  ldy, _DTYPES[yt], _vec("y_scale", y_scale, M, dev), _on(dev, stream)),
           "ctr_rms_norm_fwd")
    return y


def ctr_rms_norm_bwd(dy: torch.Tensor, s: torch.Tensor, dx: torch.Tensor, weight: Optional[torch.Tensor] = None,
                     eps: float = 1e-6, dsum: Optional[torch.Tensor] = None, dweight: Optional[torch.Tensor] = None,
                     workspace: Optional[RmsNormWorkspace] = None, stream=None) -> None:
    """dx = the norm's gradient at s for dy, plus dsum where given; dweight
    (which needs the workspace) overwritten."""
    dev, st, gt = _dev_of(s), s.dtype, dy.dtype
    if s.dim() != 2 or st not in _DTYPES or gt not in _DTYPES:
        raise ValueError("s and dy: matrices of a supported type expected")
    M, N = s.shape
    gp, ldg = _mat("dy", dy, gt, M, N, dev)
    sp, lds = _mat("s", s, st, M, N, dev)
    dp, ldd = (None, 0) if dsum is None else _mat("dsum", dsum, st, M, N, dev)
    xp, ldx = _mat("dx", dx, st, M, N, dev)
    wp, nb = (None, 0) if workspace is None else (workspace.ptr, workspace.nbytes)
    if workspace is not None and workspace.dev != dev:
        raise ValueError("the workspace is on cuda:%d" % workspace.dev)
    _check(lib().ctr_rms_norm_bwd(gp, ldg, _DTYPES[gt], sp, lds, _DTYPES[st], _vec("weight", weight, N, dev), M, N, eps,
                                  dp, ldd, xp, ldx, _vec("dweight", dweight, N, dev), wp, nb, _on(dev, stream)),
           "ctr_rms_norm_bwd")


# ------------------------------------------------------------- sequence towers and their training
class GatedScanWorkspace:
    """Scratch of the gated scan's calls for up to T rows of D channels in up
    to B sequences."""

    def __init__(self, T: int, B: int, D: int, device="cuda"):
        self.nbytes = int(lib().dsf_gated_scan_workspace_bytes(int(T), int(B), int(D)))
        if self.nbytes == 0:
            raise DsfError(DSF_EINVAL, "dsf_gated_scan_workspace_bytes")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        self.ptr, self.dev = self.buf.data_ptr(), self.buf.get_device()


def _scan_of(x: torch.Tensor, B: int, workspace: GatedScanWorkspace, lengths):
    dev = _dev_of(x)
    if workspace.dev != dev:
        raise ValueError("the workspace is on cuda:%d" % workspace.dev)
    if x.dim() != 2 or x.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("x: a float32 or bfloat16 matrix expected")
    T, D = x.shape
    if lengths is not None and (lengths.dtype is not torch.int32 or lengths.shape != (B,) or lengths.get_device() != dev
                                or not lengths.is_contiguous()):
        raise ValueError("lengths: contiguous int32 [%d] on cuda:%d expected" % (B, dev))
    if lengths is None and (T % B if B > 0 else T):
        raise ValueError("%d rows are not %d sequences of one length" % (T, B))
    return dev, T, D, _dptr(lengths)


def _state(name: str, t: Optional[torch.Tensor], B: int, D: int, dev: int) -> Optional[int]:
    """Pointer of a contiguous fp32 [B, D] matrix (None for None)."""
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.shape != (B, D) or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("%s: contiguous float32 [%d, %d] on cuda:%d expected" % (name, B, D, dev))
    return t.data_ptr()


def ctr_gated_scan_fwd(x: torch.Tensor, gate: torch.Tensor, h: torch.Tensor, B: int, workspace: GatedScanWorkspace,
                       lengths: Optional[torch.Tensor] = None, h0: Optional[torch.Tensor] = None,
                       h_last: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """h_t = (1 - z_t) h_{t-1} + z_t x_t with z = sigmoid(gate) along each of B
    sequences of rows (lengths int32 [B]; None: of equal length), from h0
    [B, D] (None: zeros); the last states into h_last where given."""
    dev, T, D, lp = _scan_of(x, B, workspace, lengths)
    xp, ldx = _mat("x", x, x.dtype, T, D, dev)
    gp, ldg = _mat("gate", gate, x.dtype, T, D, dev)
    hp, ldh = _mat("h", h, x.dtype, T, D, dev)
    _check(lib().ctr_gated_scan_fwd(xp, ldx, gp, ldg, _DTYPES[x.dtype], lp, T, B, D, _state("h0", h0, B, D, dev), hp, ldh,
                                    _state("h_last", h_last, B, D, dev), workspace.ptr, workspace.nbytes, _dptr(status),
                                    _on(dev, stream)), "ctr_gated_scan_fwd")
    return h


def ctr_gated_scan_bwd(dh: torch.Tensor, x: torch.Tensor, gate: torch.Tensor, h: torch.Tensor, dx: torch.Tensor,
                       dgate: torch.Tensor, B: int, workspace: GatedScanWorkspace,
                       lengths: Optional[torch.Tensor] = None, h0: Optional[torch.Tensor] = None,
                       dh_last: Optional[torch.Tensor] = None, dh0: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of ctr_gated_scan_fwd (h: its output) for dh and dh_last
    (None: zeros): dx, dgate, and dh0 where given, each overwritten."""
    dev, T, D, lp = _scan_of(x, B, workspace, lengths)
    m = [_mat(n, t, x.dtype, T, D, dev) for n, t in (("dh", dh), ("x", x), ("gate", gate), ("h", h), ("dx", dx),
                                                     ("dgate", dgate))]
    _check(lib().ctr_gated_scan_bwd(*m[0], *m[1], *m[2], *m[3], _DTYPES[x.dtype], lp, T, B, D, _state("h0", h0, B, D, dev),
                                    _state("dh_last", dh_last, B, D, dev), *m[4], *m[5], _state("dh0", dh0, B, D, dev),
                                    workspace.ptr, workspace.nbytes, _dptr(status), _on(dev, stream)), "ctr_gated_scan_bwd")


class SoftmaxXentWorkspace:
    """Scratch of the cross entropy of up to M rows against a catalogue layer;
    backward: for the gradients too."""

    def __init__(self, layer: DenseLayer, M: int, backward: bool = False):
        self.nbytes = int(lib().dsf_softmax_xent_workspace_bytes(layer._ref, int(M), int(bool(backward))))
        if self.nbytes == 0:
            raise DsfError(DSF_EINVAL, "dsf_softmax_xent_workspace_bytes")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=layer.device)
        self.ptr, self.dev = self.buf.data_ptr(), layer.dev


def _target_of(target: torch.Tensor, M: int, dev: int) -> int:
    if target.dtype is not torch.int64 or target.shape != (M,) or target.get_device() != dev or not target.is_contiguous():
        raise ValueError("target: contiguous int64 [%d] on cuda:%d expected" % (M, dev))
    return target.data_ptr()


def ctr_softmax_xent_fwd(layer: DenseLayer, x: torch.Tensor, target: torch.Tensor, loss: torch.Tensor, lse: torch.Tensor,
                         workspace: SoftmaxXentWorkspace, status: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """loss [M] = lse - z_target, lse [M] = log sum exp of z = x W^T + bias over
    the catalogue's V rows W (layer, without an activation); target int64 [M],
    -1: the row is left out (loss 0). The logits are not kept."""
    dev, M, (xp, ldx) = _x_of(layer, x, workspace)
    _check(lib().ctr_softmax_xent_fwd(layer._ref, xp, ldx, _target_of(target, M, dev), M, _vec("loss", loss, M, dev),
                                      _vec("lse", lse, M, dev), workspace.ptr, workspace.nbytes, _dptr(status),
                                      _on(dev, stream)), "ctr_softmax_xent_fwd")
    return loss


def ctr_softmax_xent_bwd(layer: DenseLayer, x: torch.Tensor, target: torch.Tensor, lse: torch.Tensor,
                         workspace: SoftmaxXentWorkspace, dloss: Optional[torch.Tensor] = None,
                         dx: Optional[torch.Tensor] = None, dW: Optional[torch.Tensor] = None,
                         db: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of ctr_softmax_xent_fwd (lse: its output) for dloss [M] (None:
    ones), each overwritten where given."""
    dev, M, (xp, ldx) = _x_of(layer, x, workspace)
    dxp, lddx = (None, 0) if dx is None else _mat("dx", dx, layer.type, M, layer.K, dev)
    dWp = None
    if dW is not None:
        dWp, _ = _mat("dW", dW, layer.type, layer.R, layer.K, dev)
        if not dW.is_contiguous():
            raise ValueError("dW: contiguous expected")
    _check(lib().ctr_softmax_xent_bwd(layer._ref, xp, ldx, _target_of(target, M, dev), _vec("lse", lse, M, dev),
                                      _vec("dloss", dloss, M, dev), M, dxp, lddx, dWp, _vec("db", db, layer.R, dev),
                                      workspace.ptr, workspace.nbytes, _dptr(status), _on(dev, stream)),
           "ctr_softmax_xent_bwd")


class MuonWorkspace:
    """Scratch of ctr_muon_update for matrices of W's shape."""

    def __init__(self, W: torch.Tensor):
        if W.dim() != 2:
            raise ValueError("W: a matrix expected")
        self.R, self.C = (int(n) for n in W.shape)
        self.nbytes = int(lib().dsf_muon_workspace_bytes(self.R, self.C))
        if self.nbytes == 0:
            raise DsfError(DSF_EINVAL, "dsf_muon_workspace_bytes")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=W.device)
        self.ptr, self.dev = self.buf.data_ptr(), self.buf.get_device()


def ctr_muon_update(W: torch.Tensor, grad: torch.Tensor, momentum: torch.Tensor, workspace: MuonWorkspace,
                    lr: float = 0.02, mu: float = 0.95, weight_decay: float = 0.0, nesterov: bool = True, steps: int = 5,
                    status: Optional[torch.Tensor] = None, stream=None) -> None:
    """One optimiser step on a dense matrix: momentum = mu momentum + grad, the
    update grad + mu momentum (nesterov) or momentum orthogonalised by `steps`
    Newton-Schulz steps, W = W - lr (weight_decay W + sqrt(max(1, rows /
    columns)) update). W and grad float32 or bfloat16, momentum float32."""
    dev = _dev_of(W)
    if workspace.dev != dev:
        raise ValueError("the workspace is on cuda:%d" % workspace.dev)
    if W.dim() != 2 or W.dtype not in (torch.float32, torch.bfloat16) or grad.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("W and grad: float32 or bfloat16 matrices expected")
    R, C = W.shape
    wp, ldw = _mat("W", W, W.dtype, R, C, dev)
    gp, ldg = _mat("grad", grad, grad.dtype, R, C, dev)
    if momentum.dtype is not torch.float32 or momentum.shape != (R, C) or momentum.get_device() != dev \
            or not momentum.is_contiguous():
        raise ValueError("momentum: contiguous float32 [%d, %d] on cuda:%d expected" % (R, C, dev))
    _check(lib().ctr_muon_update(wp, ldw, _DTYPES[W.dtype], gp, ldg, _DTYPES[grad.dtype], momentum.data_ptr(), R, C, lr, mu,
                                 weight_decay, int(bool(nesterov)), int(steps), workspace.ptr, workspace.nbytes,
                                 _dptr(status), _on(dev, stream)), "ctr_muon_update")
