"""A gated linear recurrence and what stands around a mixer in a layer: the Python binding
of include/ssm66_layer.h.  Like the rest of the package it only marshals arguments; every
step of the computation runs in the library's HIP kernels.

    y, last_state, states = gated_scan_fwd(x, r, i, decay, h0=None, seq_lens=None, reset=None,
                                           return_states=False)
    grads = gated_scan_bwd(x, r, i, decay, dy, states, dlast=None, seq_lens=None, reset=None)
    y = gated_scan_step(state, x, r, i, decay)                   # state updated in place
"""
import ctypes
import functools

from .lm import _code, _core, _flags, _on_gpu, _ptr, _stream, _want, _workspace

_CHUNK = 128  # tokens from one kept state of the recurrence to the next


def declare(lib):
    """The argument types of the calls in include/ssm66_layer.h."""
    vp, i64, ci, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    lib.ssm_gated_scan_workspace_size.restype = sz
    lib.ssm_gated_scan_workspace_size.argtypes = [i64] * 3 + [ci, ci]
    lib.ssm_gated_scan_fwd.restype = ci
    lib.ssm_gated_scan_fwd.argtypes = [vp] * 11 + [sz] + [i64] * 3 + [ci, vp]
    lib.ssm_gated_scan_bwd.restype = ci
    lib.ssm_gated_scan_bwd.argtypes = [vp] * 15 + [sz] + [i64] * 3 + [ci, vp]
    lib.ssm_gated_scan_step.restype = ci
    lib.ssm_gated_scan_step.argtypes = [vp] * 6 + [i64] * 2 + [ci, vp]


def _call(c, torch, index, name, *args):
    """One call on the current stream of GPU `index`, which a launch needs to be the current
    device."""
    fn = getattr(c.load_library(), name)
    if torch.cuda.current_device() == index:
        st = fn(*args, _stream(torch, index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _stream(torch, index))
    if st != 0:
        raise c.SsmError(st, name)


def _same(c, like, shape, index, **tensors):
    """Tensors of one shape and type on one GPU."""
    dtype = like.dtype
    for name, t in tensors.items():
        if not (t.shape == shape and t.dtype is dtype and t.get_device() == index
                and t.is_contiguous()):
            c._check(t, name, shape, dtype, like.device)


# sizes alone decide a workspace
@functools.lru_cache(maxsize=512)
def _scan_ws(batch, L, dim, backward, need_ddecay):
    return int(_core()[0].load_library().ssm_gated_scan_workspace_size(batch, L, dim, backward,
                                                                       need_ddecay))


def gated_scan_workspace_size(batch, L, dim, backward=False, need_ddecay=True):
    """Bytes of workspace gated_scan_fwd (or, with backward, gated_scan_bwd) needs."""
    return _scan_ws(batch, L, dim, int(bool(backward)), int(bool(backward and need_ddecay)))


def _scan_check(c, torch, x, r, i, decay, seq_lens, reset):
    index = _on_gpu(x, "x", 3, "(batch, L, dim)")
    shape = batch, L, dim = x.shape
    code = _code(c, torch, x)
    _same(c, x, shape, index, x=x, r=r, i=i)
    _want(decay, "decay", (dim,), torch.float32, x.device, index)
    if seq_lens is not None:
        _want(seq_lens, "seq_lens", (batch,), torch.int32, x.device, index)
    if reset is not None:
        _want(reset, "reset", (batch, L), torch.uint8, x.device, index)
    return batch, L, dim, x.device, index, code


def gated_scan_fwd(x, r, i, decay, h0=None, seq_lens=None, reset=None, y=None, last_state=None,
                   return_last_state=True, return_states=False, workspace=None):
    """The gated linear recurrence over whole sequences on the GPU.

    a_t = exp(-decay sigmoid(r_t)), h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t, y = h.
    x, r, i: (batch, L, dim), all float32 or all bfloat16 (r, i: the gates before their
    sigmoid); decay: (dim,) float32, not negative;
    h0: optional (batch, dim) float32 initial state;
    seq_lens: optional (batch,) int32 real lengths (y = 0 past them, the state kept);
    reset: optional (batch, L) bool or uint8, state zeroed before each flagged token.
    Returns (y like x, last_state (batch, dim) float32 or None, states or None): with
    return_states the state before every 128th token, (batch, ceil(L / 128), dim) float32,
    which gated_scan_bwd takes.
    """
    c, torch = _core()
    reset = _flags(torch, reset)
    batch, L, dim, dev, index, io = _scan_check(c, torch, x, r, i, decay, seq_lens, reset)
    f32 = torch.float32
    if h0 is not None:
        _want(h0, "h0", (batch, dim), f32, dev, index)
    if y is None:
        y = torch.empty_like(x)
    else:
        _want(y, "y", x.shape, x.dtype, dev, index)
    if last_state is not None:
        _want(last_state, "last_state", (batch, dim), f32, dev, index)
    elif return_last_state:
        last_state = torch.empty((batch, dim), dtype=f32, device=dev)
    states = torch.empty((batch, (L + _CHUNK - 1) // _CHUNK, dim), dtype=f32, device=dev) \
        if return_states else None
    ws, size = _workspace(torch, workspace, _scan_ws(batch, L, dim, 0, 0), dev)
    _call(c, torch, index, "ssm_gated_scan_fwd", _ptr(x), _ptr(r), _ptr(i), _ptr(decay), _ptr(h0),
          _ptr(seq_lens), _ptr(reset), _ptr(y), _ptr(last_state), _ptr(states), _ptr(ws), size,
          batch, L, dim, io)
    return y, last_state, states


def gated_scan_bwd(x, r, i, decay, dy, states, dlast=None, seq_lens=None, reset=None,
                   need_ddecay=True, need_dh0=False, workspace=None):
    """Gradients of gated_scan_fwd on the GPU, from its inputs and the states it returned.

    dy: like x; dlast: optional (batch, dim) float32, the gradient of last_state.
    Returns a dict: dx, dr, di (io dtype), ddecay and dh0 (float32, None if not needed).
    """
    c, torch = _core()
    reset = _flags(torch, reset)
    batch, L, dim, dev, index, io = _scan_check(c, torch, x, r, i, decay, seq_lens, reset)
    f32 = torch.float32
    _same(c, x, x.shape, index, dy=dy)
    _want(states, "states", (batch, (L + _CHUNK - 1) // _CHUNK, dim), f32, dev, index)
    _want(dlast, "dlast", (batch, dim), f32, dev, index)
    g = dict(dx=torch.empty_like(x), dr=torch.empty_like(x), di=torch.empty_like(x),
             ddecay=torch.empty_like(decay) if need_ddecay else None,
             dh0=torch.empty((batch, dim), dtype=f32, device=dev) if need_dh0 else None)
    ws, size = _workspace(torch, workspace, _scan_ws(batch, L, dim, 1, int(bool(need_ddecay))), dev)
    _call(c, torch, index, "ssm_gated_scan_bwd", _ptr(x), _ptr(r), _ptr(i), _ptr(decay),
          _ptr(states), _ptr(seq_lens), _ptr(reset), _ptr(dy), _ptr(dlast), _ptr(g["dx"]),
          _ptr(g["dr"]), _ptr(g["di"]), _ptr(g["ddecay"]), _ptr(g["dh0"]), _ptr(ws), size, batch, L,
          dim, io)
    return g


def gated_scan_step(state, x, r, i, decay, y=None):
    """One token of the gated linear recurrence on the GPU; `state` (batch, dim) float32 is
    updated in place.  x, r, i: (batch, dim).  Returns y like x."""
    c, torch = _core()
    index = _on_gpu(x, "x", 2, "(batch, dim)")
    shape = batch, dim = x.shape
    code = _code(c, torch, x)
    _same(c, x, shape, index, x=x, r=r, i=i)
    _want(state, "state", shape, torch.float32, x.device, index)
    _want(decay, "decay", (dim,), torch.float32, x.device, index)
    if y is None:
        y = torch.empty_like(x)
    else:
        _want(y, "y", shape, x.dtype, x.device, index)
    _call(c, torch, index, "ssm_gated_scan_step", _ptr(state), _ptr(x), _ptr(r), _ptr(i),
          _ptr(decay), _ptr(y), batch, dim, code)
    return y
