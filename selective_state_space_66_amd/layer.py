"""A gated linear recurrence and what stands around a mixer in a layer: the Python binding
of include/ssm66_layer.h.  Like the rest of the package it only marshals arguments; every
step of the computation runs in the library's HIP kernels.

    y, last_state, states = gated_scan_fwd(x, r, i, decay, h0=None, seq_lens=None, reset=None,
                                           return_states=False)
    grads = gated_scan_bwd(x, r, i, decay, dy, states, dlast=None, seq_lens=None, reset=None)
    y = gated_scan_step(state, x, r, i, decay)                   # state updated in place
    y, h, mean, rstd = add_norm_fwd(x, residual=None, weight=None, bias=None, kind="layer",
                                    eps=1e-5, p=0.0, rng=None, site=0)
    grads = add_norm_bwd(h, dy, mean, rstd, weight=None, kind="layer", dh=None, p=0.0, rng=None,
                         site=0)
    y = dropout_fwd(x, p, rng, site=0, residual=None)
    dx = dropout_bwd(dy, p, rng, site=0)
    freqs, mscale = rotary_freqs(rot_dim, theta=10000.0, scaling="none", device="cuda")
    q, k = rotary_fwd(q, k, freqs, positions=None, mscale=1.0, interleaved=False)
    dq, dk = rotary_bwd(dq, dk, freqs, positions=None, mscale=1.0, interleaved=False)

rng is a tensor of two int64 on the GPU, seed and offset of a counter-based generator; the
program moves the offset on from step to step (rng[1] += number of sites), a backward call
takes its forward's rng and site.

A workspace that is given serves one call at a time: calls that may run at once, on two streams
or in two graphs, take one each (each call makes its own where none is given).

An output that is given shares memory with an input only where its function says so, and then
is that tensor or a view of all of it; anything else is refused.
"""
import ctypes
import functools
import math

from .lm import SSM_BF16, SSM_F32, _code, _core, _flags, _on_gpu, _ptr, _stream, _want, _workspace

_NORMS = {"layer": 0, "rms": 1}
_CHUNK = 64   # tokens from one kept state of the recurrence to the next


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
    cf = ctypes.c_float
    lib.ssm_dropout.restype = ci
    lib.ssm_dropout.argtypes = [vp] * 3 + [i64, cf, vp, i64, ci, ci, vp]
    lib.ssm_add_norm_workspace_size.restype = sz
    lib.ssm_add_norm_workspace_size.argtypes = [i64, i64]
    lib.ssm_add_norm_fwd.restype = ci
    lib.ssm_add_norm_fwd.argtypes = [vp] * 4 + [ci, cf, cf, vp, i64] + [vp] * 4 + [i64, i64, ci, ci, vp]
    lib.ssm_add_norm_bwd.restype = ci
    lib.ssm_add_norm_bwd.argtypes = [vp] * 4 + [ci, vp, vp, cf, vp, i64] + [vp] * 5 + \
        [sz, i64, i64, ci, ci, vp]
    lib.ssm_rotary.restype = ci
    lib.ssm_rotary.argtypes = [vp] * 4 + [cf, ci, ci, vp, vp] + [i64] * 6 + [ci, vp]


def _call(c, torch, index, name, *args):
    """One call on the current stream of GPU `index`, which a launch needs to be the current
    device."""
    fn = getattr(c.load_library(), name)
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, _stream(torch, index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _stream(torch, index))
    if st != 0:
        raise c.SsmError(st, name)


def _fits(t, shape, dtype, index):
    return (t.shape == shape and t.dtype is dtype and t.get_device() == index
            and t.is_contiguous())


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
    shape, io, dev = x.shape, x.dtype, x.device
    batch, L, dim = shape
    code = _code(c, torch, x)
    if not (_fits(r, shape, io, index) and _fits(i, shape, io, index) and x.is_contiguous()
            and _fits(decay, (dim,), torch.float32, index)):
        for name, t in (("x", x), ("r", r), ("i", i)):
            c._check(t, name, shape, io, dev)
        c._check(decay, "decay", (dim,), torch.float32, dev)
    if seq_lens is not None:
        _want(seq_lens, "seq_lens", (batch,), torch.int32, dev, index)
    if reset is not None:
        _want(reset, "reset", (batch, L), torch.uint8, dev, index)
    return batch, L, dim, dev, index, code


def gated_scan_fwd(x, r, i, decay, h0=None, seq_lens=None, reset=None, y=None, last_state=None,
                   return_last_state=True, return_states=False, workspace=None):
    """The gated linear recurrence over whole sequences on the GPU.

    a_t = exp(-decay sigmoid(r_t)), h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t, y = h.
    x, r, i: (batch, L, dim), all float32 or all bfloat16 (r, i: the gates before their
    sigmoid); decay: (dim,) float32, 0 to 1e30;
    h0: optional (batch, dim) float32 initial state;
    seq_lens: optional (batch,) int32 real lengths (y = 0 past them, the state kept);
    reset: optional (batch, L) bool or uint8, state zeroed before each flagged token.
    Returns (y like x, last_state (batch, dim) float32 or None, states or None): with
    return_states the state before every 64th token, (batch, ceil(L / 64), dim) float32,
    which gated_scan_bwd takes.  y, last_state and workspace may be given, but no input may be
    any of them.
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
        last_state = decay.new_empty((batch, dim))
    states = decay.new_empty((batch, (L + _CHUNK - 1) // _CHUNK, dim)) if return_states else None
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
    _want(dy, "dy", x.shape, x.dtype, dev, index)
    _want(states, "states", (batch, (L + _CHUNK - 1) // _CHUNK, dim), f32, dev, index)
    _want(dlast, "dlast", (batch, dim), f32, dev, index)
    g = dict(dx=torch.empty_like(x), dr=torch.empty_like(x), di=torch.empty_like(x),
             ddecay=torch.empty_like(decay) if need_ddecay else None,
             dh0=decay.new_empty((batch, dim)) if need_dh0 else None)
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
    shape, io, f32 = x.shape, x.dtype, torch.float32
    batch, dim = shape
    code = _code(c, torch, x)
    if not (_fits(r, shape, io, index) and _fits(i, shape, io, index) and x.is_contiguous()
            and _fits(state, shape, f32, index) and _fits(decay, (dim,), f32, index)):
        dev = x.device
        for name, t in (("x", x), ("r", r), ("i", i)):
            c._check(t, name, shape, io, dev)
        c._check(state, "state", shape, f32, dev)
        c._check(decay, "decay", (dim,), f32, dev)
    if y is None:
        y = torch.empty_like(x)
    else:
        _want(y, "y", shape, x.dtype, x.device, index)
    _call(c, torch, index, "ssm_gated_scan_step", _ptr(state), _ptr(x), _ptr(r), _ptr(i),
          _ptr(decay), _ptr(y), batch, dim, code)
    return y


def _rng(torch, p, rng, device, index):
    if rng is None and p == 0.0:
        return
    if not 0.0 <= p < 1.0:
        raise ValueError(f"p: expected a rate in [0, 1), got {p}")
    if rng is not None:
        _want(rng, "rng", (2,), torch.int64, device, index)
    elif p > 0.0:
        raise ValueError("rng: two int64 on the GPU (seed, offset) are needed where p is not 0")


def _dense(c, torch, x, name):
    """The GPU's index of a contiguous io tensor, and its type's code."""
    index = x.get_device()
    if index < 0:
        raise ValueError("tensors must be on the GPU")
    if not x.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return index, _code(c, torch, x)


def _dropout(x, p, rng, site, residual, y, dtype, name):
    c, torch = _core()
    index, code = _dense(c, torch, x, name)
    _rng(torch, p, rng, x.device, index)
    if residual is not None:
        if residual.dtype != x.dtype and residual.dtype is not torch.float32:
            raise TypeError(f"residual: expected {x.dtype} or float32, got {residual.dtype}")
        dtype = residual.dtype
        _want(residual, "residual", x.shape, dtype, x.device, index)
    if y is None:
        y = torch.empty_like(x, dtype=dtype)
    else:
        _want(y, "dx" if name == "dy" else "y", x.shape, dtype, x.device, index)
    _call(c, torch, index, "ssm_dropout", _ptr(x), _ptr(residual), _ptr(rng), site, p, _ptr(y),
          x.numel(), code, _code(c, torch, y))
    return y


def dropout_fwd(x, p, rng, site=0, residual=None, y=None):
    """Dropout on the GPU, from a counter-based generator: the mask is never stored.

    x: any shape, float32 or bfloat16; p: the rate, 0 <= p < 1; rng: two int64 on the GPU, seed
    and offset (None where p is 0); site: a number for each place that drops, added to the
    offset; residual: optional tensor like x, of x's type or float32, which is added.
    Returns dropout(x) + residual, of the residual's type (else x's); y may be given, and may
    be x (of one type) or residual.
    """
    return _dropout(x, p, rng, site, residual, y, x.dtype, "x")


def dropout_bwd(dy, p, rng, site=0, dtype=None, dx=None):
    """Gradient of dropout_fwd's x (the residual's is dy), with its p, rng and site.

    dtype: x's type, where it is not dy's.
    """
    return _dropout(dy, p, rng, site, None, dx, dtype or dy.dtype, "dy")


def _norm_check(c, torch, x, name, kind, weight, bias, p, rng):
    index, code = _dense(c, torch, x, name)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"{name} must be (..., dim)")
    if kind not in _NORMS:
        raise ValueError(f"kind: expected one of {sorted(_NORMS)}, got {kind!r}")
    dim = x.shape[-1]
    if weight is not None:
        _want(weight, "weight", (dim,), torch.float32, x.device, index)
    if bias is not None:
        _want(bias, "bias", (dim,), torch.float32, x.device, index)
    _rng(torch, p, rng, x.device, index)
    return x.numel() // dim, dim, index, code


@functools.lru_cache(maxsize=512)
def add_norm_workspace_size(rows, dim):
    """Bytes of workspace add_norm_bwd needs where dweight or dbias is asked for."""
    return int(_core()[0].load_library().ssm_add_norm_workspace_size(rows, dim))


def add_norm_fwd(x, residual=None, weight=None, bias=None, kind="layer", eps=1e-5, p=0.0, rng=None,
                 site=0, y=None, h=None, return_stats=True):
    """A residual, a dropped-out branch and the norm of their sum, on the GPU.

    h = residual + dropout(x), y = norm(h) weight + bias over the last dimension (at most
    16384); kind: "layer" or "rms".
    x: (..., dim) float32 or bfloat16; residual: optional, like x, of x's type or float32;
    weight, bias: optional (dim,) float32; p, rng, site: as for dropout_fwd.
    h is rounded to the residual's type (else x's), and the norm is of that.
    Returns (y like x, h, mean, rstd): h is x itself where there is nothing to add or drop; mean
    and rstd (...) float32 are what add_norm_bwd takes (None if not requested, mean also with
    "rms").  y may be given, and may be x; h may be given, and may be residual.
    """
    c, torch = _core()
    rows, dim, index, code = _norm_check(c, torch, x, "x", kind, weight, bias, p, rng)
    f32 = torch.float32
    h_dtype = x.dtype
    if residual is not None:
        if residual.dtype != x.dtype and residual.dtype is not f32:
            raise TypeError(f"residual: expected {x.dtype} or float32, got {residual.dtype}")
        h_dtype = residual.dtype
        _want(residual, "residual", x.shape, h_dtype, x.device, index)
    if y is None:
        y = torch.empty_like(x)
    else:
        _want(y, "y", x.shape, x.dtype, x.device, index)
    same = h is None and residual is None and p == 0.0
    if h is not None:
        _want(h, "h", x.shape, h_dtype, x.device, index)
    elif not same:
        h = torch.empty_like(x, dtype=h_dtype)
    elif rows and y.data_ptr() == x.data_ptr():
        raise ValueError("y: may be x only where h is a tensor of its own")
    mean = rstd = None
    if return_stats:
        rstd = torch.empty(x.shape[:-1], dtype=f32, device=x.device)
        mean = torch.empty_like(rstd) if kind == "layer" else None
    _call(c, torch, index, "ssm_add_norm_fwd", _ptr(x), _ptr(residual), _ptr(weight), _ptr(bias),
          _NORMS[kind], eps, p, _ptr(rng), site, _ptr(y), _ptr(h), _ptr(mean), _ptr(rstd), rows, dim,
          code, SSM_F32 if h_dtype is f32 else SSM_BF16)
    return y, x if same else h, mean, rstd


def add_norm_bwd(h, dy, mean, rstd, weight=None, kind="layer", dh=None, p=0.0, rng=None, site=0,
                 need_dweight=None, need_dbias=False, need_dresidual=True, workspace=None):
    """Gradients of add_norm_fwd on the GPU, from the h, mean and rstd it returned.

    dy: like y; dh: optional, like h, the gradient that reaches h from elsewhere.
    Returns a dict: dx (dy's type), dresidual (h's type), dweight and dbias (float32), None where
    not needed; dweight is needed where weight is given, unless need_dweight says otherwise.
    """
    c, torch = _core()
    rows, dim, index, code = _norm_check(c, torch, dy, "dy", kind, weight, None, p, rng)
    f32, dev = torch.float32, dy.device
    if h.dtype != dy.dtype and h.dtype is not f32:
        raise TypeError(f"h: expected {dy.dtype} or float32, got {h.dtype}")
    _want(h, "h", dy.shape, h.dtype, dev, index)
    _want(dh, "dh", dy.shape, h.dtype, dev, index)
    _want(rstd, "rstd", dy.shape[:-1], f32, dev, index)
    if kind == "layer":
        _want(mean, "mean", dy.shape[:-1], f32, dev, index)
    if need_dweight is None:
        need_dweight = weight is not None
    g = dict(dx=torch.empty_like(dy), dresidual=torch.empty_like(h) if need_dresidual else None,
             dweight=torch.empty((dim,), dtype=f32, device=dev) if need_dweight else None,
             dbias=torch.empty((dim,), dtype=f32, device=dev) if need_dbias else None)
    need = add_norm_workspace_size(rows, dim) if need_dweight or need_dbias else 0
    ws, size = _workspace(torch, workspace, need, dev)
    _call(c, torch, index, "ssm_add_norm_bwd", _ptr(h), _ptr(dy), _ptr(dh), _ptr(weight),
          _NORMS[kind], _ptr(mean) if kind == "layer" else None, _ptr(rstd), p, _ptr(rng), site,
          _ptr(g["dx"]), _ptr(g["dresidual"]), _ptr(g["dweight"]), _ptr(g["dbias"]), _ptr(ws), size,
          rows, dim, code, SSM_F32 if h.dtype is f32 else SSM_BF16)
    return g


def rotary_freqs(rot_dim, theta=10000.0, scaling="none", factor=1.0, original_length=None,
                 beta_fast=32.0, beta_slow=1.0, device=None):
    """The angle per position of each pair, (rot_dim / 2,) float32, and the factor mscale of the
    outputs: what rotary_fwd takes, computed once.

    theta ** (-2 j / rot_dim), and for contexts `factor` times longer than those trained on
      "linear": all divided by the factor;
      "ntk": theta times factor ** (rot_dim / (rot_dim - 2)), so that the slowest pair is;
      "yarn": divided for the pairs that turn less than beta_slow times in original_length
      positions, kept for those that turn more than beta_fast times, with a ramp between, and
      mscale = 1 + 0.1 log(factor).
    """
    _, torch = _core()
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim: expected an even size of at least 2, got {rot_dim}")
    if scaling not in ("none", "linear", "ntk", "yarn"):
        raise ValueError(f"scaling: expected none, linear, ntk or yarn, got {scaling!r}")
    if not theta > 1.0 or not factor >= 1.0:
        raise ValueError("theta: expected more than 1, and factor: at least 1")
    pairs, mscale = rot_dim // 2, 1.0
    if scaling == "ntk" and rot_dim > 2:
        theta = theta * factor ** (rot_dim / (rot_dim - 2))
    freqs = [theta ** (-2.0 * j / rot_dim) for j in range(pairs)]
    if scaling == "linear":
        freqs = [f / factor for f in freqs]
    if scaling == "yarn":
        if not original_length or original_length < 1:
            raise ValueError("original_length: needed for scaling='yarn'")

        def pair_of(turns):  # the pair that turns so often in original_length positions
            return rot_dim * math.log(original_length / (turns * 2.0 * math.pi)) / (2.0 * math.log(theta))

        low = max(math.floor(pair_of(beta_fast)), 0)
        high = min(math.ceil(pair_of(beta_slow)), rot_dim - 1)
        ramp = [min(max((j - low) / max(high - low, 1e-3), 0.0), 1.0) for j in range(pairs)]
        freqs = [f / factor * t + f * (1.0 - t) for f, t in zip(freqs, ramp)]
        mscale = 1.0 + 0.1 * math.log(factor)
    return torch.tensor(freqs, dtype=torch.float64).float().to(device or "cuda"), mscale


def _rotary(q, k, freqs, positions, mscale, interleaved, inverse, q_out, k_out, names):
    c, torch = _core()
    index = _on_gpu(q, names[0], 4, "(batch, L, heads, dim)")
    batch, L, H, D = q.shape
    io, dev, code, Hk = q.dtype, q.device, _code(c, torch, q), 0
    if not q.is_contiguous():
        raise ValueError(f"{names[0]}: must be contiguous")
    if k is not None:
        if k.dim() != 4:
            raise ValueError(f"{names[1]} must be (batch, L, kheads, dim)")
        Hk = k.shape[2]
        _want(k, names[1], (batch, L, Hk, D), io, dev, index)
    if freqs.dim() != 1 or not 1 <= freqs.shape[0] <= D // 2:
        raise ValueError(f"freqs: expected 1 to {D // 2} values, got {tuple(freqs.shape)}")
    _want(freqs, "freqs", freqs.shape, torch.float32, dev, index)
    if positions is not None:
        _want(positions, "positions", (batch, L), torch.int32, dev, index)
    if H < 1:
        raise ValueError(f"{names[0]}: at least one head is needed")
    if q_out is None:
        q_out = torch.empty_like(q)
    else:
        _want(q_out, "q_out", q.shape, io, dev, index)
    if k is None:
        k_out = None
    elif k_out is None:
        k_out = torch.empty_like(k)
    else:
        _want(k_out, "k_out", k.shape, io, dev, index)
    _call(c, torch, index, "ssm_rotary", _ptr(q), _ptr(k), _ptr(freqs), _ptr(positions), mscale,
          int(bool(interleaved)), inverse, _ptr(q_out), _ptr(k_out), batch, L, H, Hk, D,
          2 * freqs.shape[0], code)
    return q_out, k_out


def rotary_fwd(q, k, freqs, positions=None, mscale=1.0, interleaved=False, q_out=None, k_out=None):
    """Rotary positions of queries and keys on the GPU.

    q: (batch, L, heads, dim), k: (batch, L, kheads, dim) or None, float32 or bfloat16;
    freqs: (rot / 2,) float32, the angle per position of each pair (rotary_freqs); the elements
    of a head from rot on are left as they are; positions: optional (batch, L) int32 (0 .. L - 1
    when omitted); interleaved: pairs are neighbours, else they lie rot / 2 apart.
    Returns (q_out, k_out), which may be given, and may be q and k (in place).
    """
    return _rotary(q, k, freqs, positions, mscale, interleaved, 0, q_out, k_out, ("q", "k"))


def rotary_bwd(dq, dk, freqs, positions=None, mscale=1.0, interleaved=False, q_out=None, k_out=None):
    """Gradients of rotary_fwd's q and k from those of its outputs (same arguments)."""
    return _rotary(dq, dk, freqs, positions, mscale, interleaved, 1, q_out, k_out, ("dq", "dk"))
