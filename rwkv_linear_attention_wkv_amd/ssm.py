"""State space operators: the short causal convolution, the selective scan and the 8-bit state store.

As in the rest of the package, every function checks and marshals its arguments and calls the C ABI
(include/wkv_ssm.h); the arithmetic runs in the library's HIP kernels, asynchronously on torch's
current stream of the tensors' device.

Token arrays are [B, T, width] (dense) or packed [tokens, width] (varlen), bfloat16 or float32, one
dtype per call.  Their rows need not be adjacent: a view such as ``xz[..., :D]`` of a wider projection
is passed as it is (the last dimension contiguous, one step between all rows).  States, parameters
and outputs are contiguous; states and parameters are float32.  An output may not overlap an input,
apart from a state updated in place.
"""
from __future__ import annotations

import torch

from . import _native
from ._marshal import _out_code
from ._native import check

__all__ = ["ssm_conv_forward", "ssm_conv_backward", "ssm_conv_forward_varlen", "ssm_scan_forward", "ssm_scan_forward_train",
           "ssm_scan_backward", "ssm_scan_forward_varlen",
           "state_store_alloc", "state_store_write", "state_store_read"]

_lib = _native.load()

_CODES = {torch.bfloat16: _native.WKV_BF16, torch.float32: _native.WKV_F32}
_ACTS = {None: _native.WKV_ACT_NONE, "none": _native.WKV_ACT_NONE, "silu": _native.WKV_ACT_SILU}
_FORMATS = {torch.int8: _native.WKV_STORE_INT8, torch.float8_e4m3fn: _native.WKV_STORE_E4M3}


def _first(t, name, dims):
    """The call's first token array: its dtype code; the others are held to its device and dtype."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {tuple(t.shape)}")
    if t.dtype not in _CODES:
        raise TypeError(f"unsupported input dtype {t.dtype} (bfloat16 or float32)")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return _CODES[t.dtype]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _flat(t, name, dtype, shape, ref):
    """The address of a contiguous tensor of this dtype and shape on the call's device; None for None."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == ref.get_device() and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != ref.device:
        raise ValueError(f"{name} must be on {ref.device}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _rows(t, name, lead, width, ref, same=True):
    """A token array of rows ``width`` wide: its address and the step between its rows, in elements."""
    cols = width[0] if len(width) == 1 else width[0] * width[1]
    try:
        if (t.shape == lead + width and t.get_device() == ref.get_device() and (t.dtype is ref.dtype or not same)
                and t.is_contiguous()):
            return t.data_ptr(), cols
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if same and t.dtype != ref.dtype:
        raise TypeError(f"token inputs must share one dtype: {name}={t.dtype}, {ref.dtype}")
    if t.device != ref.device:
        raise ValueError(f"{name} must be on {ref.device}, got {t.device}")
    if t.shape != lead + width:
        raise ValueError(f"{name} must have shape {tuple(lead + width)}, got {tuple(t.shape)}")
    if t.numel() == 0:
        return t.data_ptr(), cols
    st, k = t.stride(), len(lead)
    step = 1
    for i in range(t.dim() - 1, k - 1, -1):
        if t.shape[i] != 1 and st[i] != step:
            raise ValueError(f"{name} must be contiguous within a row, got strides {st}")
        step *= t.shape[i]
    outer = [i for i in range(k) if t.shape[i] != 1]
    step = st[outer[-1]] if outer else cols
    if len(outer) == 2 and st[0] != t.shape[1] * step:
        raise ValueError(f"{name} must have one step between all rows, got strides {st}")
    if step < cols:
        raise ValueError(f"{name} has rows of {cols} elements {step} apart")
    return t.data_ptr(), step


def _launch(ref, fn, *args):
    """Calls the library with the current stream of the tensors' device, that device being current."""
    dev = ref.get_device()
    if dev == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, torch.cuda.current_stream(dev).cuda_stream)
    if status:
        check(status)


def _output(y, out_dtype, shape, ref):
    code, dt = _out_code(y, out_dtype)
    if y is None:
        y = torch.empty(shape, dtype=dt, device=ref.device)
    else:
        _flat(y, "y", dt, shape, ref)
    return y, code


def _dense_states(state, state_map, state_out, return_state, B, inner, ref):
    n_state = 0
    if state is not None:
        n_state = state.shape[0] if isinstance(state, torch.Tensor) and state.dim() else 0
        _flat(state, "state", torch.float32, torch.Size((n_state, *inner)), ref)
    mp = _flat(state_map, "state_map", torch.int32, torch.Size((B,)), ref)
    if state_out is not None:
        _flat(state_out, "state_out", torch.float32, torch.Size((B, *inner)), ref)
    elif return_state:
        state_out = torch.empty((B, *inner), dtype=torch.float32, device=ref.device)
    return (_ptr(state), mp, n_state, _ptr(state_out)), state_out


def _slot_states(lengths, state, state_map, state_out, inner, ref):
    if not isinstance(lengths, torch.Tensor) or lengths.dim() != 1:
        raise TypeError("lengths must be a one-dimensional torch.Tensor")
    S = lengths.shape[0]
    ln = _flat(lengths, "lengths", torch.int32, torch.Size((S,)), ref)
    n_state = state.shape[0] if isinstance(state, torch.Tensor) and state.dim() else 0
    if state is None:
        raise TypeError("state must be a torch.Tensor")
    shape = torch.Size((n_state, *inner))
    si = _flat(state, "state", torch.float32, shape, ref)
    so = si if state_out is None else _flat(state_out, "state_out", torch.float32, shape, ref)
    mp = _flat(state_map, "state_map", torch.int32, torch.Size((S,)), ref)
    return S, ln, (si, so, mp, n_state)


def _status(dev_status, ref):
    return _flat(dev_status, "dev_status", torch.int32, torch.Size((1,)), ref)


def _conv_params(x, weight, bias, activation):
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [D, W]")
    if activation not in _ACTS:
        raise ValueError(f"unknown activation {activation!r} (None or 'silu')")
    D, W = x.shape[-1], weight.shape[1]
    return D, W, (_flat(weight, "weight", torch.float32, torch.Size((D, W)), x),
                  _flat(bias, "bias", torch.float32, torch.Size((D,)), x), _ACTS[activation])


def ssm_conv_forward(x, weight, bias=None, state=None, state_map=None, *, activation=None, y=None, state_out=None,
                     return_state=True, dev_status=None, out_dtype=torch.float32):
    """Short causal convolution of each channel: ``y_t = act(bias + sum_j weight[:, j] x_(t-W+1+j))``.

    x: [B, T, D]; weight: [D, W] fp32, W = 2, 3 or 4; bias: [D] fp32; ``activation``: None or "silu".
    ``state``: [n_state, W-1, D] fp32, the inputs before the first token, oldest first (None: zeros);
    ``state_map``: [B] int32.  With W = 2 and the taps (mu, 1 - mu) this is RWKV's token shift.
    Returns ``(y [B, T, D], state_out [B, W-1, D] or None)``; y is ``out_dtype`` unless given.
    """
    code = _first(x, "x", 3)
    B, T, D = x.shape
    _, W, par = _conv_params(x, weight, bias, activation)
    xa = _rows(x, "x", x.shape[:2], (D,), x)
    states, state_out = _dense_states(state, state_map, state_out, return_state, B, (W - 1, D), x)
    y, oc = _output(y, out_dtype, x.shape, x)
    _launch(x, _lib.wkv_ssm_conv_forward, B, T, D, W, *xa, code, *par, y.data_ptr(), oc, *states, _status(dev_status, x))
    return y, state_out


def ssm_conv_backward(x, weight, bias, dy, state=None, state_map=None, *, activation=None, d_state=None,
                      return_d_state=True, dev_status=None, grad_dtype=torch.float32):
    """Gradients of :func:`ssm_conv_forward` (the same inputs, T >= 1).

    ``dy`` [B, T, D] (float32 or bfloat16) is the gradient of y, ``d_state`` [B, W-1, D] fp32 that of the final
    state.  Returns ``(dx [B, T, D] in grad_dtype, dweight [D, W], dbias [D] or None, d_state_in [B, W-1, D] or
    None)``, the last three in float32; ``d_state_in[b]`` belongs to the initial state row b started from.
    """
    code = _first(x, "x", 3)
    B, T, D = x.shape
    _, W, par = _conv_params(x, weight, bias, activation)
    xa = _rows(x, "x", x.shape[:2], (D,), x)
    (si, mp, n_state, _), _ = _dense_states(state, state_map, None, False, B, (W - 1, D), x)
    if not isinstance(dy, torch.Tensor) or dy.dtype not in _CODES:
        raise TypeError("dy must be a bfloat16 or float32 torch.Tensor")
    if grad_dtype not in _CODES:
        raise TypeError(f"unsupported gradient dtype {grad_dtype} (bfloat16 or float32)")
    dya = _rows(dy, "dy", x.shape[:2], (D,), x, same=False)
    ds = _flat(d_state, "d_state", torch.float32, torch.Size((B, W - 1, D)), x)
    f = dict(dtype=torch.float32, device=x.device)
    dx = torch.empty(x.shape, dtype=grad_dtype, device=x.device)
    dw = torch.empty((D, W), **f)
    db = torch.empty((D,), **f) if bias is not None else None
    d_first = torch.empty((B, W - 1, D), **f) if return_d_state else None
    need = _lib.wkv_ssm_conv_backward_workspace(B, T, D, W)
    ws = torch.empty(need // 4, **f)
    _launch(x, _lib.wkv_ssm_conv_backward, B, T, D, W, *xa, code, *par, *dya, _CODES[dy.dtype], si, mp, n_state, ds,
            _ptr(dx), _CODES[grad_dtype], _ptr(dw), _ptr(db), _ptr(d_first), _ptr(ws), need, _status(dev_status, x))
    return dx, dw, db, d_first


def ssm_conv_forward_varlen(lengths, x, weight, bias, state, *, max_len, state_out=None, state_map=None,
                            activation=None, y=None, dev_status=None, out_dtype=torch.float32):
    """:func:`ssm_conv_forward` over packed rows of slots; updates ``state_out`` (default: ``state`` in place).

    ``lengths``: [S] int32 device tensor (tokens each slot consumes, at most ``max_len``); x: [tokens, D];
    ``state``: [n_state, W-1, D] fp32; ``state_map``: [S] int32.  Returns y [tokens, D].
    """
    code = _first(x, "x", 2)
    total, D = x.shape
    _, W, par = _conv_params(x, weight, bias, activation)
    xa = _rows(x, "x", x.shape[:1], (D,), x)
    S, ln, states = _slot_states(lengths, state, state_map, state_out, (W - 1, D), x)
    y, oc = _output(y, out_dtype, x.shape, x)
    _launch(x, _lib.wkv_ssm_conv_forward_varlen, S, D, W, ln, int(max_len), total, *xa, code, *par, y.data_ptr(), oc,
            *states, _status(dev_status, x))
    return y


def _scan_args(x, dt, A, B, C, D, z, dt_bias, dt_softplus, code):
    """(channels, states, groups, the C ABI's input arguments) of a scan call."""
    lead, width = x.shape[:-1], x.shape[-1]
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be [D, N]")
    N = A.shape[1]
    for name, t in (("B", B), ("C", C)):
        if not isinstance(t, torch.Tensor) or t.dim() not in (x.dim(), x.dim() + 1):
            raise ValueError(f"{name} must be [..., N] or [..., G, N] with the token dimensions of x")
    G = B.shape[-2] if B.dim() > x.dim() else 1
    inner = (G, N) if B.dim() > x.dim() else (N,)
    return width, N, G, (*_rows(x, "x", lead, (width,), x), *_rows(dt, "dt", lead, (width,), x),
                         _flat(A, "A", torch.float32, torch.Size((width, N)), x), *_rows(B, "B", lead, inner, x),
                         *_rows(C, "C", lead, inner, x), code, _flat(D, "D", torch.float32, torch.Size((width,)), x),
                         *(_rows(z, "z", lead, (width,), x) if z is not None else (None, 0)),
                         _flat(dt_bias, "dt_bias", torch.float32, torch.Size((width,)), x), int(bool(dt_softplus)))


def _workspace(rows, T, total, width, N, G, ref):
    """Memory for a scan that is cut into segments, allocated on the current stream for one call, or None; its bytes."""
    need = _lib.wkv_ssm_scan_workspace(rows, T, total, width, N, G) if T > 64 else 0
    return (torch.empty(need // 4, dtype=torch.float32, device=ref.device) if need else None), need


def ssm_scan_forward(x, dt, A, B, C, D=None, z=None, dt_bias=None, state=None, state_map=None, *, dt_softplus=True,
                     y=None, state_out=None, return_state=True, dev_status=None, out_dtype=torch.float32):
    """Selective state space scan.

    With ``delta = softplus(dt + dt_bias)`` (``dt + dt_bias`` unless ``dt_softplus``), per channel d and
    state n: ``h <- exp(delta A[d, n]) h + delta B[n] x``, ``y = sum_n C[n] h + D x``, times
    ``silu(z)`` when z is given.  x, dt, z: [B, T, D]; A: [D, N] fp32, N = 1 .. 64; B, C: [B, T, N], or
    [B, T, G, N] for G equal groups of channels; D, dt_bias: [D] fp32; ``state``: [n_state, D, N] fp32
    (None: zeros); ``state_map``: [B] int32.
    Returns ``(y [B, T, D], state_out [B, D, N] or None)``; y is ``out_dtype`` unless given.
    """
    code = _first(x, "x", 3)
    rows, T, _ = x.shape
    width, N, G, args = _scan_args(x, dt, A, B, C, D, z, dt_bias, dt_softplus, code)
    states, state_out = _dense_states(state, state_map, state_out, return_state, rows, (width, N), x)
    y, oc = _output(y, out_dtype, x.shape, x)
    ws, ws_bytes = _workspace(rows, T, rows * T, width, N, G, x)
    _launch(x, _lib.wkv_ssm_scan_forward, rows, T, width, N, G, *args, y.data_ptr(), oc, *states, _ptr(ws), ws_bytes,
            _status(dev_status, x))
    return y, state_out


def _chunks(T):
    return max((T + 15) // 16 - 1, 0)


def ssm_scan_forward_train(x, dt, A, B, C, D=None, z=None, dt_bias=None, state=None, state_map=None, *, dt_softplus=True,
                           y=None, state_out=None, return_state=True, dev_status=None, out_dtype=torch.float32,
                           chunk_states=None):
    """:func:`ssm_scan_forward` that also saves the state at every 16-token boundary for :func:`ssm_scan_backward`.

    Returns ``(y, state_out or None, chunk_states [B, ceil(T/16) - 1, D, N] fp32)``.
    """
    code = _first(x, "x", 3)
    rows, T, _ = x.shape
    width, N, G, args = _scan_args(x, dt, A, B, C, D, z, dt_bias, dt_softplus, code)
    states, state_out = _dense_states(state, state_map, state_out, return_state, rows, (width, N), x)
    y, oc = _output(y, out_dtype, x.shape, x)
    saved = torch.Size((rows, _chunks(T), width, N))
    if chunk_states is None:
        chunk_states = torch.empty(saved, dtype=torch.float32, device=x.device)
    ws, ws_bytes = _workspace(rows, T, rows * T, width, N, G, x)
    _launch(x, _lib.wkv_ssm_scan_forward_train, rows, T, width, N, G, *args, y.data_ptr(), oc, *states,
            _flat(chunk_states, "chunk_states", torch.float32, saved, x) or None, _ptr(ws), ws_bytes, _status(dev_status, x))
    return y, state_out, chunk_states


def ssm_scan_backward(x, dt, A, B, C, dy, D=None, z=None, dt_bias=None, state=None, state_map=None, *, dt_softplus=True,
                      d_state=None, return_d_state=True, chunk_states=None, dev_status=None, grad_dtype=torch.float32):
    """Gradients of :func:`ssm_scan_forward` (the same inputs, T >= 1).

    ``dy`` [B, T, D] (float32 or bfloat16) is the gradient of y, ``d_state`` [B, D, N] fp32 that of the final
    state; ``chunk_states`` what :func:`ssm_scan_forward_train` saved for these inputs (without them they are
    computed first).  Returns ``(dx, ddt, dA, dB, dC, dD, dz, d_dt_bias, d_state_in)``: dx, ddt, dz [B, T, D] and
    dB, dC (shaped as B and C) in ``grad_dtype``; dA [D, N], dD, d_dt_bias [D] and d_state_in [B, D, N] in
    float32.  dD, dz and d_dt_bias are None where their input is, d_state_in unless ``return_d_state``;
    ``d_state_in[b]`` belongs to the initial state row b started from.
    """
    code = _first(x, "x", 3)
    rows, T, _ = x.shape
    width, N, G, args = _scan_args(x, dt, A, B, C, D, z, dt_bias, dt_softplus, code)
    (si, mp, n_state, _), _ = _dense_states(state, state_map, None, False, rows, (width, N), x)
    if not isinstance(dy, torch.Tensor) or dy.dtype not in _CODES:
        raise TypeError("dy must be a bfloat16 or float32 torch.Tensor")
    if grad_dtype not in _CODES:
        raise TypeError(f"unsupported gradient dtype {grad_dtype} (bfloat16 or float32)")
    dya = _rows(dy, "dy", x.shape[:-1], (width,), x, same=False)
    chunks = _flat(chunk_states, "chunk_states", torch.float32, torch.Size((rows, _chunks(T), width, N)), x) or None
    ds = _flat(d_state, "d_state", torch.float32, torch.Size((rows, width, N)), x)
    g = dict(dtype=grad_dtype, device=x.device)
    f = dict(dtype=torch.float32, device=x.device)
    dx, ddt = torch.empty(x.shape, **g), torch.empty(x.shape, **g)
    dB, dC = torch.empty(B.shape, **g), torch.empty(C.shape, **g)
    dz = torch.empty(x.shape, **g) if z is not None else None
    dA = torch.empty((width, N), **f)
    dD = torch.empty((width,), **f) if D is not None else None
    db = torch.empty((width,), **f) if dt_bias is not None else None
    d_first = torch.empty((rows, width, N), **f) if return_d_state else None
    need = _lib.wkv_ssm_scan_backward_workspace(rows, T, width, N, G, int(chunks is not None or _chunks(T) == 0))
    ws = torch.empty(need // 4, **f)
    _launch(x, _lib.wkv_ssm_scan_backward, rows, T, width, N, G, *args, *dya, _CODES[dy.dtype], si, mp, n_state, chunks, ds,
            _ptr(dx), _ptr(ddt), _ptr(dB), _ptr(dC), _ptr(dz), _CODES[grad_dtype], _ptr(dA), _ptr(dD), _ptr(db),
            _ptr(d_first), _ptr(ws), need, _status(dev_status, x))
    return dx, ddt, dA, dB, dC, dD, dz, db, d_first


def ssm_scan_forward_varlen(lengths, x, dt, A, B, C, state, *, max_len, D=None, z=None, dt_bias=None, state_out=None,
                            state_map=None, dt_softplus=True, y=None, dev_status=None, out_dtype=torch.float32):
    """:func:`ssm_scan_forward` over packed rows of slots; updates ``state_out`` (default: ``state`` in place).

    ``lengths``: [S] int32 device tensor; x, dt, z: [tokens, D]; B, C: [tokens, N] or [tokens, G, N];
    ``state``: [n_state, D, N] fp32; ``state_map``: [S] int32.  Returns y [tokens, D].
    """
    code = _first(x, "x", 2)
    total = x.shape[0]
    width, N, G, args = _scan_args(x, dt, A, B, C, D, z, dt_bias, dt_softplus, code)
    S, ln, states = _slot_states(lengths, state, state_map, state_out, (width, N), x)
    y, oc = _output(y, out_dtype, x.shape, x)
    ws, ws_bytes = _workspace(S, int(max_len), total, width, N, G, x)
    _launch(x, _lib.wkv_ssm_scan_forward_varlen, S, width, N, G, ln, int(max_len), total, *args, y.data_ptr(), oc,
            *states, _ptr(ws), ws_bytes, _status(dev_status, x))
    return y


def state_store_alloc(n_store, row, *, format=torch.int8, device="cuda"):
    """An empty 8-bit store of ``n_store`` rows of ``row`` values: ``(data, scale)`` (format: torch.int8 or
    torch.float8_e4m3fn).  Every row reads back as zeros until it is written."""
    if format not in _FORMATS:
        raise TypeError(f"unsupported store format {format} (torch.int8 or torch.float8_e4m3fn)")
    data = torch.zeros((n_store, row), dtype=torch.int8, device=device).view(format)
    return data, torch.zeros((n_store, (row + 63) // 64), dtype=torch.float32, device=device)


def _store_args(data, scale, states, store_rows, state_rows, dev_status):
    if not isinstance(data, torch.Tensor) or data.dim() != 2:
        raise ValueError("data must be [n_store, row]")
    if data.dtype not in _FORMATS:
        raise TypeError(f"unsupported store format {data.dtype} (torch.int8 or torch.float8_e4m3fn)")
    if not data.is_cuda or not data.is_contiguous():
        raise ValueError("data must be a contiguous device tensor")
    n_store, row = data.shape
    if not isinstance(states, torch.Tensor) or states.dim() < 2:
        raise ValueError("states must be [n_state, ...]")
    n_state = states.shape[0]
    if n_state and states.numel() != n_state * row:
        raise ValueError(f"states hold {states.numel() // n_state} values a row, the store {row}")
    counts = {t.shape[0] for t in (store_rows, state_rows) if isinstance(t, torch.Tensor) and t.dim() == 1}
    if len(counts) > 1:
        raise ValueError("store_rows and state_rows must have the same length")
    count = counts.pop() if counts else n_state
    n = torch.Size((count,))
    return (_flat(data, "data", data.dtype, data.shape, data), _flat(scale, "scale", torch.float32, torch.Size((n_store, (row + 63) // 64)), data),
            n_store, _FORMATS[data.dtype], _flat(states, "states", torch.float32, states.shape, data), n_state, row,
            _flat(store_rows, "store_rows", torch.int32, n, data), _flat(state_rows, "state_rows", torch.int32, n, data), count,
            _status(dev_status, data))


def state_store_write(data, scale, states, store_rows=None, state_rows=None, *, dev_status=None):
    """Writes rows of ``states`` ([n_state, ...] fp32: WKV, convolution or scan states) into the 8-bit store
    ``data`` [n_store, row] (int8 or float8_e4m3fn), ``scale`` [n_store, ceil(row / 64)] fp32.

    Item i stores ``states[state_rows[i]]`` as row ``store_rows[i]`` (int32 device tensors; None: i).
    Groups of 64 consecutive values share the scale max|v| / 127 (int8) or / 448 (e4m3).
    """
    args = _store_args(data, scale, states, store_rows, state_rows, dev_status)
    _launch(data, _lib.wkv_state_store_write, *args)


def state_store_read(data, scale, states, store_rows=None, state_rows=None, *, dev_status=None):
    """Reads rows of the 8-bit store back into ``states`` (see :func:`state_store_write`); one stored row may
    be read into many state rows.  Returns ``states``."""
    args = _store_args(data, scale, states, store_rows, state_rows, dev_status)
    _launch(data, _lib.wkv_state_store_read, *args)
    return states
