"""POET-X orthogonal-equivalence linear layer on AMD MI355X (gfx950).

The compute lives in libpoetx.so (hand-written HIP kernels behind a C ABI,
include/poetx.h); `binding` is its ctypes binding with the same function names
`layer.PoetxLinear` owns the device buffers of one linear, and `layer.PoetxGroup`
runs the CNP work of several linears (e.g. one decoder layer) as one batch.
`layer.PoetxNorm` is the norm in front of them, `layer.PoetxAdam` and
`layer.PoetxMuon` step their packed parameters, and `layer.PoetxOrthogonalizer`
orthogonalises the updates of matrices that stay dense.  `layer.PoetxRope` and
`layer.PoetxAttention` are what stands between the q, k, v linears and the o
linear, and `layer.PoetxLogProb` the log probabilities behind the last one.
"""

from .binding import (  # noqa: F401
    POETX_BF16,
    POETX_F32,
    POETX_I8,
    POETX_OP_BWD,
    POETX_OP_CNP,
    POETX_OP_FWD,
    POETX_OP_MERGE,
    LayerDesc,
    PoetxError,
    attn_desc,
    desc,
    lib,
    logp_desc,
    muon_params,
    norm_desc,
    ns_params,
    poetx_adam_step_batch,
    poetx_attn_bwd,
    poetx_attn_fwd,
    poetx_attn_workspace_size,
    poetx_cnp_backward_batch,
    poetx_cnp_batch_workspace_size,
    poetx_cnp_build,
    poetx_cnp_build_batch,
    poetx_cnp_grad_bytes,
    poetx_g_bytes,
    poetx_last_error,
    poetx_linear_bwd,
    poetx_linear_bwd_dx,
    poetx_linear_fwd,
    poetx_logp_bwd,
    poetx_logp_fwd,
    poetx_logp_workspace_size,
    poetx_merge_reinit,
    poetx_muon_step_batch,
    poetx_muon_workspace_size,
    poetx_norm_bwd,
    poetx_norm_fwd,
    poetx_norm_stats_bytes,
    poetx_norm_workspace_size,
    poetx_orthogonalize,
    poetx_orthogonalize_workspace_size,
    poetx_packed_len,
    poetx_perm_from_seed,
    poetx_premerge,
    poetx_rope,
    poetx_rope_freqs,
    poetx_saved_bytes,
    poetx_spo_bwd,
    poetx_spo_fwd,
    poetx_spo_saved_bytes,
    poetx_spo_workspace_size,
    poetx_version,
    poetx_weight_bytes,
    poetx_workspace_size,
    rope_desc,
    rope_params,
)
