"""GB300-native (sm_103a) MultiTowerDIN sparse forward.

The compute lives in libdinsparse.so (CUDA kernels behind the C ABI in
include/dinsparse.h); this package is its Python binding, the build script and
the seeded workload generator.
"""
from .binding import (AttnMLP, DenseLayer, DenseWorkspace, DsfError, EmbeddingTables,  # noqa: F401
                      RmsNormWorkspace, Workspace, ctr_dense_bwd, ctr_dense_fwd, ctr_glu_bwd, ctr_glu_fwd,
                      ctr_rms_norm_bwd, ctr_rms_norm_fwd, din_jagged_attn, din_sparse_fwd, emb_bag_pool,
                      grid_size, lib, status_string)
