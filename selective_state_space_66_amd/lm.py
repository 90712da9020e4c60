"""The operators of a linear-attention layer and of its training step: the Python
binding of include/ssm66_lm.h.  Like the rest of the package it only marshals
arguments; every step of the computation runs in the library's HIP kernels.

    o, last_state = linattn_fwd(q, k, v, log_decay, scale=None, h0=None, seq_lens=None,
                                reset=None)
    grads = linattn_bwd(q, k, v, log_decay, do, scale=None, h0=None, dlast=None,
                        seq_lens=None, reset=None)
    o = linattn_step(state, q, k, v, log_decay, scale=None)      # state updated in place
"""
import ctypes

SSM_F32, SSM_BF16 = 0, 1


def declare(lib):
    """The argument types of the calls in include/ssm66_lm.h."""
    vp, i64, ci, sz, cf = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t,
                           ctypes.c_float)
    lib.ssm_linattn_fwd_workspace_size.restype = sz
    lib.ssm_linattn_fwd_workspace_size.argtypes = [i64] * 6 + [ci]
    lib.ssm_linattn_bwd_workspace_size.restype = sz
    lib.ssm_linattn_bwd_workspace_size.argtypes = [i64] * 6 + [ci, ci]
    lib.ssm_linattn_fwd.restype = ci
    lib.ssm_linattn_fwd.argtypes = [vp] * 4 + [cf] + [vp] * 6 + [sz] + [i64] * 6 + [ci, vp]
    lib.ssm_linattn_bwd.restype = ci
    lib.ssm_linattn_bwd.argtypes = [vp] * 4 + [cf] + [vp] * 11 + [sz] + [i64] * 6 + [ci, vp]
    lib.ssm_linattn_step.restype = ci
    lib.ssm_linattn_step.argtypes = [vp] * 5 + [cf, vp] + [i64] * 5 + [ci, vp]


def _core():
    import selective_state_space_66_amd as ssm
    return ssm


def _workspace(workspace, need, device):
    """The caller's workspace, checked, or a new one; None where none is needed."""
    import torch
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device) if need else None
    if workspace.dtype != torch.uint8 or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous uint8 tensor on {device}")
    if workspace.numel() < need:
        raise ValueError(f"workspace: need {need} bytes, got {workspace.numel()}")
    return workspace


def _flags(reset):
    import torch
    return reset.view(torch.uint8) if reset is not None and reset.dtype == torch.bool else reset


def _on_gpu(t, name, dims, layout):
    if t.dim() != dims:
        raise ValueError(f"{name} must be {layout}")
    if t.device.type != "cuda":
        raise ValueError("tensors must be on the GPU")


def _linattn_check(q, k, v, log_decay, h0, seq_lens, reset):
    import torch
    c = _core()
    _on_gpu(q, "q", 4, "(batch, L, kheads, dk)")
    _on_gpu(v, "v", 4, "(batch, L, nheads, dv)")
    batch, L, Hk, Dk = q.shape
    H, Dv = v.shape[2:]
    io, dev = q.dtype, q.device
    c._io_code(q)
    c._check(q, "q", (batch, L, Hk, Dk), io, dev)
    c._check(k, "k", (batch, L, Hk, Dk), io, dev)
    c._check(v, "v", (batch, L, H, Dv), io, dev)
    c._check(log_decay, "log_decay", (H,), torch.float32, dev)
    c._check(h0, "h0", (batch, H, Dv, Dk), torch.float32, dev)
    c._check(seq_lens, "seq_lens", (batch,), torch.int32, dev)
    c._check(reset, "reset", (batch, L), torch.uint8, dev)
    return batch, L, H, Hk, Dk, Dv


def linattn_fwd_workspace_size(batch, L, nheads, kheads, dk, dv, io_dtype):
    """Bytes of workspace ssm_linattn_fwd needs (io_dtype: a torch dtype)."""
    import torch
    code = SSM_F32 if io_dtype == torch.float32 else SSM_BF16
    return int(_core().load_library().ssm_linattn_fwd_workspace_size(batch, L, nheads, kheads, dk,
                                                                     dv, code))


def linattn_bwd_workspace_size(batch, L, nheads, kheads, dk, dv, io_dtype, need_dlog_decay=True):
    """Bytes of workspace ssm_linattn_bwd needs (io_dtype: a torch dtype)."""
    import torch
    code = SSM_F32 if io_dtype == torch.float32 else SSM_BF16
    return int(_core().load_library().ssm_linattn_bwd_workspace_size(
        batch, L, nheads, kheads, dk, dv, int(bool(need_dlog_decay)), code))


def linattn_fwd(q, k, v, log_decay, scale=None, h0=None, seq_lens=None, reset=None, o=None,
                last_state=None, return_last_state=True, workspace=None):
    """Linear attention with a decay for each head, over whole sequences on the GPU.

    S_t = exp(log_decay) S_{t-1} + v_t k_t^T, o_t = scale S_t q_t, per head.
    q, k: (batch, L, kheads, dk); v: (batch, L, nheads, dv), all float32 or all bfloat16;
    kheads divides nheads, and consecutive heads share keys; dk, dv multiples of 8 up to 256.
    log_decay: (nheads,) float32; scale: dk ** -0.5 by default;
    h0: optional (batch, nheads, dv, dk) float32 initial state;
    seq_lens: optional (batch,) int32 real lengths (o = 0 past them, the state kept);
    reset: optional (batch, L) bool or uint8, state zeroed before each flagged token.
    Returns (o like v, last_state (batch, nheads, dv, dk) float32, or None if not requested).
    """
    import torch
    c = _core()
    lib = c.load_library()
    reset = _flags(reset)
    batch, L, H, Hk, Dk, Dv = _linattn_check(q, k, v, log_decay, h0, seq_lens, reset)
    dev = q.device
    if o is None:
        o = torch.empty_like(v)
    c._check(o, "o", (batch, L, H, Dv), q.dtype, dev)
    if last_state is None and return_last_state:
        last_state = torch.empty((batch, H, Dv, Dk), dtype=torch.float32, device=dev)
    c._check(last_state, "last_state", (batch, H, Dv, Dk), torch.float32, dev)
    io = c._io_code(q)
    ws = _workspace(workspace, int(lib.ssm_linattn_fwd_workspace_size(batch, L, H, Hk, Dk, Dv, io)),
                    dev)
    st = lib.ssm_linattn_fwd(c._ptr(q), c._ptr(k), c._ptr(v), c._ptr(log_decay),
                             Dk ** -0.5 if scale is None else float(scale), c._ptr(h0),
                             c._ptr(seq_lens), c._ptr(reset), c._ptr(o), c._ptr(last_state),
                             c._ptr(ws), 0 if ws is None else ws.numel(), batch, L, H, Hk, Dk, Dv,
                             io, c._stream(dev))
    if st != 0:
        raise c.SsmError(st, "ssm_linattn_fwd")
    return o, last_state


def linattn_bwd(q, k, v, log_decay, do, scale=None, h0=None, dlast=None, seq_lens=None, reset=None,
                need_dlog_decay=True, workspace=None):
    """Gradients of linattn_fwd on the GPU (same arguments; the states are recomputed).

    do: like v; dlast: optional (batch, nheads, dv, dk) float32, the gradient of last_state.
    Returns a dict: dq, dk, dv (io dtype), dlog_decay (float32, None if not needed) and,
    where h0 was given, dh0 (float32).
    """
    import torch
    c = _core()
    lib = c.load_library()
    reset = _flags(reset)
    batch, L, H, Hk, Dk, Dv = _linattn_check(q, k, v, log_decay, h0, seq_lens, reset)
    dev = q.device
    c._check(do, "do", (batch, L, H, Dv), q.dtype, dev)
    c._check(dlast, "dlast", (batch, H, Dv, Dk), torch.float32, dev)
    f32 = dict(dtype=torch.float32, device=dev)
    g = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
             dlog_decay=torch.empty((H,), **f32) if need_dlog_decay else None,
             dh0=torch.empty((batch, H, Dv, Dk), **f32) if h0 is not None else None)
    io = c._io_code(q)
    need = int(lib.ssm_linattn_bwd_workspace_size(batch, L, H, Hk, Dk, Dv,
                                                  int(bool(need_dlog_decay)), io))
    ws = _workspace(workspace, need, dev)
    st = lib.ssm_linattn_bwd(c._ptr(q), c._ptr(k), c._ptr(v), c._ptr(log_decay),
                             Dk ** -0.5 if scale is None else float(scale), c._ptr(h0),
                             c._ptr(seq_lens), c._ptr(reset), c._ptr(do), c._ptr(dlast),
                             c._ptr(g["dq"]), c._ptr(g["dk"]), c._ptr(g["dv"]),
                             c._ptr(g["dlog_decay"]), c._ptr(g["dh0"]), c._ptr(ws),
                             0 if ws is None else ws.numel(), batch, L, H, Hk, Dk, Dv, io,
                             c._stream(dev))
    if st != 0:
        raise c.SsmError(st, "ssm_linattn_bwd")
    return g


def linattn_step(state, q, k, v, log_decay, scale=None, o=None):
    """One token of linear attention on the GPU; `state` (batch, nheads, dv, dk) float32 is
    updated in place.  q, k: (batch, kheads, dk); v: (batch, nheads, dv). Returns o like v."""
    import torch
    c = _core()
    lib = c.load_library()
    _on_gpu(q, "q", 3, "(batch, kheads, dk)")
    _on_gpu(v, "v", 3, "(batch, nheads, dv)")
    batch, Hk, Dk = q.shape
    H, Dv = v.shape[1:]
    io, dev = q.dtype, q.device
    c._io_code(q)
    c._check(state, "state", (batch, H, Dv, Dk), torch.float32, dev)
    c._check(q, "q", (batch, Hk, Dk), io, dev)
    c._check(k, "k", (batch, Hk, Dk), io, dev)
    c._check(v, "v", (batch, H, Dv), io, dev)
    c._check(log_decay, "log_decay", (H,), torch.float32, dev)
    if o is None:
        o = torch.empty_like(v)
    c._check(o, "o", (batch, H, Dv), io, dev)
    st = lib.ssm_linattn_step(c._ptr(state), c._ptr(q), c._ptr(k), c._ptr(v), c._ptr(log_decay),
                              Dk ** -0.5 if scale is None else float(scale), c._ptr(o), batch, H,
                              Hk, Dk, Dv, c._io_code(q), c._stream(dev))
    if st != 0:
        raise c.SsmError(st, "ssm_linattn_step")
    return o
