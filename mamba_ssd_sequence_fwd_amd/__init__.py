"""Mamba-2 SSD forward pass for AMD Instinct MI355X (gfx950).

The hot path is the C-ABI library ``libssd.so`` (HIP kernels, declared in
``include/ssd.h``); this package is its thin Python binding. Build the library
with ``python -m mamba_ssd_sequence_fwd_amd.build``.

    y, final_state = forward(x, dt, A, B, C, D, initial_state, chunk_size=256,
                             cu_seqlens=None)
    y_t = step(x_t, dt_t, A, B_t, C_t, D, state)   # one decode step, state in place
    y, h = selective_scan(x, delta, A, B, C, D)     # the Mamba-1 scan (comparator)
    x, B, C, hist = conv1d_silu(xbc, w, b, x_dim, bc_dim)  # conv front producing x, B, C
    grads = backward(x, dt, A, B, C, D, h0, dy)  # dx, ddt, dA, dB, dC, dD, dinitial_state
    g = conv1d_silu_backward(xbc, w, b, dx, dB, dC)   # the front backwards
    o = group_norm_silu(y, weight, bias, z, groups=G)  # the norm and gate behind the layer
    g = group_norm_silu_backward(do, y, weight, bias, z, groups=G)
    y, h = delta_forward(x, g, beta, B, C, h0, cu_seqlens)  # the gated delta rule
    y_t = delta_step(x_t, g_t, beta_t, B_t, C_t, h)     # one decode step of it, state in place
    grads = delta_backward(x, g, beta, B, C, h0, dy)    # dx, dg, dbeta, dB, dC, dinitial_state
    B, C = bc_norm(B, C, bw, cw, positions, freqs)      # keys and queries: norm per head, rotation
    g = bc_norm_backward(dB, dC, B, C, bw, cw, positions, freqs)
    k = checkpoint_save(t); k.load()   # a Checkpoint: an activation in 8 bits, which the
                                       # front, the norm and their backward passes write and read
"""
from ._lib import (  # noqa: F401
    EXPORTED, LIB_PATH, BackwardPlan, BcNormProblem, Checkpoint, CheckpointProblem, ConvProblem, NormProblem, Plan, Problem, ScanProblem, SSDError,
    StageTimes, WorkspaceLayout, backward, conv1d_silu, forward, forward_noalloc, load,
    bc_norm, bc_norm_backward, delta_backward, delta_forward, delta_step,
    selective_scan, checkpoint_save, conv1d_silu_backward, group_norm_silu,
    group_norm_silu_backward,
    make_problem, step, validate, validate_cu_seqlens, workspace_layout, workspace_size,
    SSD_DTYPE_BF16, SSD_DTYPE_F32, SSD_FLAG_GENERIC_KERNELS, SSD_FLAG_UNFUSED, SSD_FLAG_PER_SEQUENCE,
    SSD_BC_NORM_INTERLEAVED, SSD_BC_NORM_UNIT, SSD_NORM_BEFORE_GATE, SSD_NORM_CENTER,
    SSD_OK,
    SSD_ERR_INVALID_ARG, SSD_ERR_UNSUPPORTED, SSD_ERR_WORKSPACE, SSD_ERR_HIP,
)
