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
import functools
from array import array

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


_SSM = None
_TORCH = None


def _core():
    """The package and torch (imported at the first call: the package imports without it)."""
    global _SSM, _TORCH
    if _SSM is None:
        import torch

        import selective_state_space_66_amd
        _TORCH, _SSM = torch, selective_state_space_66_amd
    return _SSM, _TORCH


# The small calls take a few microseconds on the GPU, so the checks before them are kept as
# short: one expression per tensor, and the checks that name what is wrong only where it fails.


def _want(t, name, shape, dtype, device, index):
    if t is None or (t.shape == shape and t.dtype is dtype and t.get_device() == index
                     and t.is_contiguous()):
        return
    _core()[0]._check(t, name, shape, dtype, device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(torch, index):
    """The current stream of GPU `index`, as an integer."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _workspace(torch, workspace, need, device):
    """The caller's workspace, checked, or a new one, and its size."""
    if workspace is None:
        if not need:
            return None, 0
        return torch.empty(need, dtype=torch.uint8, device=device), need
    if workspace.dtype != torch.uint8 or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous uint8 tensor on {device}")
    if workspace.numel() < need:
        raise ValueError(f"workspace: need {need} bytes, got {workspace.numel()}")
    return workspace, workspace.numel()


def _flags(torch, reset):
    return reset.view(torch.uint8) if reset is not None and reset.dtype == torch.bool else reset


def _on_gpu(t, name, dims, layout):
    """The GPU's index."""
    if t.dim() != dims:
        raise ValueError(f"{name} must be {layout}")
    if not t.is_cuda:
        raise ValueError("tensors must be on the GPU")
    return t.get_device()


def _code(c, torch, t):
    return SSM_BF16 if t.dtype is torch.bfloat16 else c._io_code(t)


# sizes alone decide a workspace
@functools.lru_cache(maxsize=512)
def _linattn_ws(backward, batch, L, H, Hk, Dk, Dv, need_dg, io):
    lib = _core()[0].load_library()
    if backward:
        return int(lib.ssm_linattn_bwd_workspace_size(batch, L, H, Hk, Dk, Dv, need_dg, io))
    return int(lib.ssm_linattn_fwd_workspace_size(batch, L, H, Hk, Dk, Dv, io))


@functools.lru_cache(maxsize=512)
def _norm_ws(batch, rows, C, groups, backward, io):
    return int(_core()[0].load_library().ssm_group_norm_workspace_size(batch, rows, C, groups,
                                                                       backward, io))


@functools.lru_cache(maxsize=512)
def _clip_ws(n):
    return int(_core()[0].load_library().ssm_clip_grad_norm_workspace_size(n))


def _linattn_check(c, torch, q, k, v, log_decay, h0, seq_lens, reset):
    index = _on_gpu(q, "q", 4, "(batch, L, kheads, dk)")
    _on_gpu(v, "v", 4, "(batch, L, nheads, dv)")
    batch, L, Hk, Dk = qs = q.shape
    H, Dv = v.shape[2:]
    io, dev, f32 = q.dtype, q.device, torch.float32
    code = _code(c, torch, q)
    if not (k.shape == qs and v.shape == (batch, L, H, Dv) and log_decay.shape == (H,)
            and k.dtype is io and v.dtype is io and log_decay.dtype is f32
            and k.get_device() == index and v.get_device() == index
            and log_decay.get_device() == index and q.is_contiguous() and k.is_contiguous()
            and v.is_contiguous() and log_decay.is_contiguous()):
        c._check(q, "q", (batch, L, Hk, Dk), io, dev)
        c._check(k, "k", (batch, L, Hk, Dk), io, dev)
        c._check(v, "v", (batch, L, H, Dv), io, dev)
        c._check(log_decay, "log_decay", (H,), f32, dev)
    if h0 is not None:
        _want(h0, "h0", (batch, H, Dv, Dk), f32, dev, index)
    if seq_lens is not None:
        _want(seq_lens, "seq_lens", (batch,), torch.int32, dev, index)
    if reset is not None:
        _want(reset, "reset", (batch, L), torch.uint8, dev, index)
    return batch, L, H, Hk, Dk, Dv, dev, index, code


def linattn_fwd_workspace_size(batch, L, nheads, kheads, dk, dv, io_dtype):
    """Bytes of workspace ssm_linattn_fwd needs (io_dtype: a torch dtype)."""
    code = SSM_F32 if io_dtype == _core()[1].float32 else SSM_BF16
    return _linattn_ws(False, batch, L, nheads, kheads, dk, dv, 0, code)


def linattn_bwd_workspace_size(batch, L, nheads, kheads, dk, dv, io_dtype, need_dlog_decay=True):
    """Bytes of workspace ssm_linattn_bwd needs (io_dtype: a torch dtype)."""
    code = SSM_F32 if io_dtype == _core()[1].float32 else SSM_BF16
    return _linattn_ws(True, batch, L, nheads, kheads, dk, dv, int(bool(need_dlog_decay)), code)


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
    c, torch = _core()
    lib = c.load_library()
    reset = _flags(torch, reset)
    batch, L, H, Hk, Dk, Dv, dev, index, io = _linattn_check(c, torch, q, k, v, log_decay, h0,
                                                             seq_lens, reset)
    if o is None:
        o = torch.empty_like(v)
    else:
        _want(o, "o", (batch, L, H, Dv), q.dtype, dev, index)
    if last_state is not None:
        _want(last_state, "last_state", (batch, H, Dv, Dk), torch.float32, dev, index)
    elif return_last_state:
        last_state = torch.empty((batch, H, Dv, Dk), dtype=torch.float32, device=dev)
    ws, size = _workspace(torch, workspace, _linattn_ws(False, batch, L, H, Hk, Dk, Dv, 0, io), dev)
    st = lib.ssm_linattn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_decay),
                             Dk ** -0.5 if scale is None else scale, _ptr(h0), _ptr(seq_lens),
                             _ptr(reset), _ptr(o), _ptr(last_state), _ptr(ws), size, batch, L, H,
                             Hk, Dk, Dv, io, _stream(torch, index))
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
    c, torch = _core()
    lib = c.load_library()
    reset = _flags(torch, reset)
    batch, L, H, Hk, Dk, Dv, dev, index, io = _linattn_check(c, torch, q, k, v, log_decay, h0,
                                                             seq_lens, reset)
    _want(do, "do", (batch, L, H, Dv), q.dtype, dev, index)
    _want(dlast, "dlast", (batch, H, Dv, Dk), torch.float32, dev, index)
    g = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
             dlog_decay=torch.empty_like(log_decay) if need_dlog_decay else None,
             dh0=torch.empty_like(h0) if h0 is not None else None)
    ws, size = _workspace(torch, workspace, _linattn_ws(True, batch, L, H, Hk, Dk, Dv,
                                                        int(bool(need_dlog_decay)), io), dev)
    st = lib.ssm_linattn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_decay),
                             Dk ** -0.5 if scale is None else scale, _ptr(h0), _ptr(seq_lens),
                             _ptr(reset), _ptr(do), _ptr(dlast), _ptr(g["dq"]), _ptr(g["dk"]),
                             _ptr(g["dv"]), _ptr(g["dlog_decay"]), _ptr(g["dh0"]), _ptr(ws), size,
                             batch, L, H, Hk, Dk, Dv, io, _stream(torch, index))
    if st != 0:
        raise c.SsmError(st, "ssm_linattn_bwd")
    return g


def linattn_step(state, q, k, v, log_decay, scale=None, o=None):
    """One token of linear attention on the GPU; `state` (batch, nheads, dv, dk) float32 is
    updated in place.  q, k: (batch, kheads, dk); v: (batch, nheads, dv). Returns o like v."""
    c, torch = _core()
    lib = c.load_library()
    index = _on_gpu(q, "q", 3, "(batch, kheads, dk)")
    _on_gpu(v, "v", 3, "(batch, nheads, dv)")
    batch, Hk, Dk = qs = q.shape
    H, Dv = v.shape[1:]
    io, f32 = q.dtype, torch.float32
    code = _code(c, torch, q)
    if not (k.shape == qs and v.shape == (batch, H, Dv) and state.shape == (batch, H, Dv, Dk)
            and log_decay.shape == (H,) and k.dtype is io and v.dtype is io
            and state.dtype is f32 and log_decay.dtype is f32 and k.get_device() == index
            and v.get_device() == index and state.get_device() == index
            and log_decay.get_device() == index and q.is_contiguous() and k.is_contiguous()
            and v.is_contiguous() and state.is_contiguous() and log_decay.is_contiguous()):
        dev = q.device
        c._check(state, "state", (batch, H, Dv, Dk), f32, dev)
        c._check(q, "q", (batch, Hk, Dk), io, dev)
        c._check(k, "k", (batch, Hk, Dk), io, dev)
        c._check(v, "v", (batch, H, Dv), io, dev)
        c._check(log_decay, "log_decay", (H,), f32, dev)
    if o is None:
        o = torch.empty_like(v)
    else:
        _want(o, "o", (batch, H, Dv), io, q.device, index)
    st = lib.ssm_linattn_step(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay),
                              Dk ** -0.5 if scale is None else scale, _ptr(o), batch, H, Hk, Dk,
                              Dv, code, _stream(torch, index))
    if st != 0:
        raise c.SsmError(st, "ssm_linattn_step")
    return o


def group_norm_workspace_size(batch, rows, channels, groups, io_dtype, backward=False):
    """Bytes of workspace group_norm_fwd (or, with backward, group_norm_bwd) needs."""
    code = SSM_F32 if io_dtype == _core()[1].float32 else SSM_BF16
    return _norm_ws(batch, rows, channels, groups, int(bool(backward)), code)


def _group_norm_check(c, torch, x, groups, weight, bias, z, act):
    index = _on_gpu(x, "x", 3, "(batch, rows, channels)")
    batch, rows, C = x.shape
    io, dev = x.dtype, x.device
    code = _code(c, torch, x)
    if act not in _ACTS:
        raise ValueError(f"act: expected one of {sorted(_ACTS)}, got {act!r}")
    if groups < 1 or C < 1 or C % groups != 0:
        raise ValueError(f"groups: {groups} does not divide {C} channels")
    _want(x, "x", (batch, rows, C), io, dev, index)
    if weight is not None:
        _want(weight, "weight", (C,), torch.float32, dev, index)
    if bias is not None:
        _want(bias, "bias", (C,), torch.float32, dev, index)
    if z is not None:
        _want(z, "z", (batch, rows, C), io, dev, index)
    return batch, rows, C, dev, index, code


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
    c, torch = _core()
    lib = c.load_library()
    batch, rows, C, dev, index, io = _group_norm_check(c, torch, x, groups, weight, bias, z, act)
    if y is None:
        y = torch.empty_like(x)
    else:
        _want(y, "y", (batch, rows, C), x.dtype, dev, index)
    mean = rstd = None
    if return_stats:
        mean = torch.empty((batch, groups), dtype=torch.float32, device=dev)
        rstd = torch.empty_like(mean)
    ws, size = _workspace(torch, workspace, _norm_ws(batch, rows, C, groups, 0, io), dev)
    st = lib.ssm_group_norm_fwd(_ptr(x), _ptr(weight), _ptr(bias), _ptr(z), _ACTS[act], eps,
                                _ptr(y), _ptr(mean), _ptr(rstd), _ptr(ws), size, batch, rows, C,
                                groups, io, _stream(torch, index))
    if st != 0:
        raise c.SsmError(st, "ssm_group_norm_fwd")
    return y, mean, rstd


def group_norm_bwd(x, groups, dy, mean, rstd, weight=None, bias=None, z=None, act="none",
                   workspace=None):
    """Gradients of group_norm_fwd on the GPU (same arguments, and the mean and rstd it gave).

    dy: like x.  Returns a dict: dx (io dtype) and, where their inputs were given, dweight,
    dbias (float32) and dz (io dtype).
    """
    c, torch = _core()
    lib = c.load_library()
    batch, rows, C, dev, index, io = _group_norm_check(c, torch, x, groups, weight, bias, z, act)
    _want(dy, "dy", (batch, rows, C), x.dtype, dev, index)
    _want(mean, "mean", (batch, groups), torch.float32, dev, index)
    _want(rstd, "rstd", (batch, groups), torch.float32, dev, index)
    g = dict(dx=torch.empty_like(x),
             dweight=torch.empty_like(weight) if weight is not None else None,
             dbias=torch.empty_like(bias) if bias is not None else None,
             dz=torch.empty_like(z) if z is not None else None)
    ws, size = _workspace(torch, workspace, _norm_ws(batch, rows, C, groups, 1, io), dev)
    st = lib.ssm_group_norm_bwd(_ptr(x), _ptr(weight), _ptr(bias), _ptr(z), _ACTS[act], _ptr(mean),
                                _ptr(rstd), _ptr(dy), _ptr(g["dx"]), _ptr(g["dweight"]),
                                _ptr(g["dbias"]), _ptr(g["dz"]), _ptr(ws), size, batch, rows, C,
                                groups, io, _stream(torch, index))
    if st != 0:
        raise c.SsmError(st, "ssm_group_norm_bwd")
    return g


def clip_grad_norm(grads, max_norm, outs=None, workspace=None):
    """The global norm of many gradients on the GPU, and the gradients clipped to it.

    grads: a list of contiguous float32 or bfloat16 tensors of any shapes, all on one GPU;
    outs: optional tensors like them for the clipped gradients (in place when omitted); no
    memory is listed twice.
    out = grad * min(1, max_norm / (norm + 1e-6)).  Returns the norm before clipping, a
    float32 tensor with no dimensions, on the GPU (nothing waits for it).
    """
    c, torch = _core()
    lib = c.load_library()
    grads = list(grads)
    outs = grads if outs is None else list(outs)
    n = len(grads)
    if n == 0:
        raise ValueError("grads: at least one tensor is needed (they say which GPU)")
    if len(outs) != n:
        raise ValueError(f"outs: expected {n} tensors, got {len(outs)}")
    if not grads[0].is_cuda:
        raise ValueError("tensors must be on the GPU")
    dev, index = grads[0].device, grads[0].get_device()
    # whole lists at a time; the loops that name a culprit run only if there is one
    tensor = torch.Tensor
    types = [t.dtype for t in grads]
    if not set(types) <= {torch.float32, torch.bfloat16}:
        i = next(i for i, t in enumerate(types) if t not in (torch.float32, torch.bfloat16))
        raise TypeError(f"grads[{i}]: expected float32 or bfloat16, got {types[i]}")
    if set(map(tensor.get_device, grads)) != {index}:
        i = next(i for i, t in enumerate(grads) if t.device != dev)
        raise ValueError(f"grads[{i}]: expected device {dev}, got {grads[i].device}")
    if not all(map(tensor.is_contiguous, grads)):
        i = next(i for i, t in enumerate(grads) if not t.is_contiguous())
        raise ValueError(f"grads[{i}]: must be contiguous")
    if outs is not grads and not ([o.shape for o in outs] == [t.shape for t in grads]
                                  and [o.dtype for o in outs] == types
                                  and set(map(tensor.get_device, outs)) == {index}
                                  and all(map(tensor.is_contiguous, outs))):
        i = next(i for i, (t, o) in enumerate(zip(grads, outs))
                 if o.shape != t.shape or o.dtype != t.dtype or o.device != dev
                 or not o.is_contiguous())
        raise ValueError(f"outs[{i}]: expected a contiguous {types[i]} tensor of shape "
                         f"{tuple(grads[i].shape)} on {dev}")
    src = array("Q", map(tensor.data_ptr, grads))
    dst = src if outs is grads else array("Q", map(tensor.data_ptr, outs))
    counts = array("q", map(tensor.numel, grads))
    codes = array("i", [SSM_F32 if t is torch.float32 else SSM_BF16 for t in types])
    norm = torch.empty((), dtype=torch.float32, device=dev)
    ws, size = _workspace(torch, workspace, _clip_ws(n), dev)
    st = lib.ssm_clip_grad_norm(src.buffer_info()[0], dst.buffer_info()[0],
                                counts.buffer_info()[0], codes.buffer_info()[0], n, max_norm,
                                _ptr(norm), _ptr(ws), size, _stream(torch, index))
    if st != 0:
        raise c.SsmError(st, "ssm_clip_grad_norm")
    return norm
