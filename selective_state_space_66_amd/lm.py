"""The operators of a linear-attention layer and of its training step: the Python
binding of include/ssm66_lm.h.  Like the rest of the package it only marshals
arguments; every step of the computation runs in the library's HIP kernels.

    o, last_state = linattn_fwd(q, k, v, log_decay, scale=None, h0=None, seq_lens=None,
                                reset=None)
    grads = linattn_bwd(q, k, v, log_decay, do, scale=None, h0=None, dlast=None,
                        seq_lens=None, reset=None)
    o = linattn_step(state, q, k, v, log_decay, scale=None)      # state updated in place
    y, mean, rstd = group_norm_fwd(x, groups, weight=None, bias=None, z=None, act="none",
                                   eps=1e-5)
    grads = group_norm_bwd(x, groups, dy, mean, rstd, weight=None, bias=None, z=None,
                           act="none")
    norm = clip_grad_norm(grads, max_norm, outs=None)            # grads clipped in place
"""
import ctypes

SSM_F32, SSM_BF16 = 0, 1
_ACTS = {"none": 0, "silu": 1}


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
    lib.ssm_group_norm_workspace_size.restype = sz
    lib.ssm_group_norm_workspace_size.argtypes = [i64] * 4 + [ci, ci]
    lib.ssm_group_norm_fwd.restype = ci
    lib.ssm_group_norm_fwd.argtypes = [vp] * 4 + [ci, cf] + [vp] * 4 + [sz] + [i64] * 4 + [ci, vp]
    lib.ssm_group_norm_bwd.restype = ci
    lib.ssm_group_norm_bwd.argtypes = [vp] * 4 + [ci] + [vp] * 8 + [sz] + [i64] * 4 + [ci, vp]
    lib.ssm_clip_grad_norm_workspace_size.restype = sz
    lib.ssm_clip_grad_norm_workspace_size.argtypes = [i64]
    lib.ssm_clip_grad_norm.restype = ci
    lib.ssm_clip_grad_norm.argtypes = [vp] * 4 + [i64, cf, vp, vp, sz, vp]


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


def group_norm_workspace_size(batch, rows, channels, groups, io_dtype, backward=False):
    """Bytes of workspace group_norm_fwd (or, with backward, group_norm_bwd) needs."""
    import torch
    code = SSM_F32 if io_dtype == torch.float32 else SSM_BF16
    return int(_core().load_library().ssm_group_norm_workspace_size(
        batch, rows, channels, groups, int(bool(backward)), code))


def _group_norm_check(x, groups, weight, bias, z, act):
    import torch
    c = _core()
    _on_gpu(x, "x", 3, "(batch, rows, channels)")
    batch, rows, C = x.shape
    io, dev = x.dtype, x.device
    c._io_code(x)
    if act not in _ACTS:
        raise ValueError(f"act: expected one of {sorted(_ACTS)}, got {act!r}")
    if groups < 1 or C < 1 or C % groups != 0:
        raise ValueError(f"groups: {groups} does not divide {C} channels")
    c._check(x, "x", (batch, rows, C), io, dev)
    c._check(weight, "weight", (C,), torch.float32, dev)
    c._check(bias, "bias", (C,), torch.float32, dev)
    c._check(z, "z", (batch, rows, C), io, dev)
    return batch, rows, C


def group_norm_fwd(x, groups, weight=None, bias=None, z=None, act="none", eps=1e-5, y=None,
                   return_stats=True, workspace=None):
    """Group norm over a channels-last tensor on the GPU, with an activation and a gate.

    x, z: (batch, rows, channels) float32 or bfloat16; each entry's groups are normalised over
    the rows and the group's channels together (rows = 1: the heads of each token).
    weight, bias: optional (channels,) float32; act: "none" or "silu", applied to the
    normalised, scaled value; z: optional gate, silu(z) multiplies the result.
    Returns (y like x, mean, rstd): mean and rstd (batch, groups) float32, what
    group_norm_bwd takes (None if not requested).
    """
    import torch
    c = _core()
    lib = c.load_library()
    batch, rows, C = _group_norm_check(x, groups, weight, bias, z, act)
    dev = x.device
    if y is None:
        y = torch.empty_like(x)
    c._check(y, "y", (batch, rows, C), x.dtype, dev)
    mean = rstd = None
    if return_stats:
        mean = torch.empty((batch, groups), dtype=torch.float32, device=dev)
        rstd = torch.empty((batch, groups), dtype=torch.float32, device=dev)
    io = c._io_code(x)
    ws = _workspace(workspace, int(lib.ssm_group_norm_workspace_size(batch, rows, C, groups, 0, io)),
                    dev)
    st = lib.ssm_group_norm_fwd(c._ptr(x), c._ptr(weight), c._ptr(bias), c._ptr(z), _ACTS[act],
                                float(eps), c._ptr(y), c._ptr(mean), c._ptr(rstd), c._ptr(ws),
                                0 if ws is None else ws.numel(), batch, rows, C, groups, io,
                                c._stream(dev))
    if st != 0:
        raise c.SsmError(st, "ssm_group_norm_fwd")
    return y, mean, rstd


def group_norm_bwd(x, groups, dy, mean, rstd, weight=None, bias=None, z=None, act="none",
                   workspace=None):
    """Gradients of group_norm_fwd on the GPU (same arguments, and the mean and rstd it gave).

    dy: like x.  Returns a dict: dx (io dtype) and, where their inputs were given, dweight,
    dbias (float32) and dz (io dtype).
    """
    import torch
    c = _core()
    lib = c.load_library()
    batch, rows, C = _group_norm_check(x, groups, weight, bias, z, act)
    dev = x.device
    c._check(dy, "dy", (batch, rows, C), x.dtype, dev)
    c._check(mean, "mean", (batch, groups), torch.float32, dev)
    c._check(rstd, "rstd", (batch, groups), torch.float32, dev)
    g = dict(dx=torch.empty_like(x),
             dweight=torch.empty_like(weight) if weight is not None else None,
             dbias=torch.empty_like(bias) if bias is not None else None,
             dz=torch.empty_like(z) if z is not None else None)
    io = c._io_code(x)
    ws = _workspace(workspace, int(lib.ssm_group_norm_workspace_size(batch, rows, C, groups, 1, io)),
                    dev)
    st = lib.ssm_group_norm_bwd(c._ptr(x), c._ptr(weight), c._ptr(bias), c._ptr(z), _ACTS[act],
                                c._ptr(mean), c._ptr(rstd), c._ptr(dy), c._ptr(g["dx"]),
                                c._ptr(g["dweight"]), c._ptr(g["dbias"]), c._ptr(g["dz"]),
                                c._ptr(ws), 0 if ws is None else ws.numel(), batch, rows, C,
                                groups, io, c._stream(dev))
    if st != 0:
        raise c.SsmError(st, "ssm_group_norm_bwd")
    return g


def clip_grad_norm(grads, max_norm, outs=None, workspace=None):
    """The global norm of many gradients on the GPU, and the gradients clipped to it.

    grads: a list of contiguous float32 or bfloat16 tensors of any shapes, all on one GPU;
    outs: optional tensors like them for the clipped gradients (in place when omitted).
    out = grad * min(1, max_norm / (norm + 1e-6)).  Returns the norm before clipping, a
    float32 tensor with no dimensions, on the GPU (nothing waits for it).
    """
    import torch
    c = _core()
    lib = c.load_library()
    grads = list(grads)
    outs = grads if outs is None else list(outs)
    n = len(grads)
    if n == 0:
        raise ValueError("grads: at least one tensor is needed (they say which GPU)")
    if len(outs) != n:
        raise ValueError(f"outs: expected {n} tensors, got {len(outs)}")
    dev = grads[0].device
    if dev.type != "cuda":
        raise ValueError("tensors must be on the GPU")
    codes = {torch.float32: SSM_F32, torch.bfloat16: SSM_BF16}
    for i, t in enumerate(grads):
        if t.dtype not in codes:
            raise TypeError(f"grads[{i}]: expected float32 or bfloat16, got {t.dtype}")
        if t.device != dev:
            raise ValueError(f"grads[{i}]: expected device {dev}, got {t.device}")
        if not t.is_contiguous():
            raise ValueError(f"grads[{i}]: must be contiguous")
    if outs is not grads:
        for i, (t, o) in enumerate(zip(grads, outs)):
            if o.shape != t.shape or o.dtype != t.dtype or o.device != dev or not o.is_contiguous():
                raise ValueError(f"outs[{i}]: expected a contiguous {t.dtype} tensor of shape "
                                 f"{tuple(t.shape)} on {dev}")
    pointers = ctypes.c_void_p * n
    src = pointers(*[t.data_ptr() for t in grads])
    dst = src if outs is grads else pointers(*[o.data_ptr() for o in outs])
    counts = (ctypes.c_int64 * n)(*[t.numel() for t in grads])
    types = (ctypes.c_int32 * n)(*[codes[t.dtype] for t in grads])
    norm = torch.empty((), dtype=torch.float32, device=dev)
    ws = _workspace(workspace, int(lib.ssm_clip_grad_norm_workspace_size(n)), dev)
    st = lib.ssm_clip_grad_norm(src, dst, counts, types, n, float(max_norm), c._ptr(norm),
                                c._ptr(ws), 0 if ws is None else ws.numel(), c._stream(dev))
    if st != 0:
        raise c.SsmError(st, "ssm_clip_grad_norm")
    return norm
