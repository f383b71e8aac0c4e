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

import struct

import torch

from . import _native
from ._marshal import _out_code
from ._native import check

__all__ = ["ssm_conv_forward", "ssm_conv_backward", "ssm_conv_forward_varlen", "ssm_scan_forward", "ssm_scan_forward_train",
           "ssm_scan_backward", "ssm_scan_forward_varlen",
           "state_store_alloc", "state_store_write", "state_store_read"]

_lib = _native.load()
_call_words = _lib.wkv_ssm_call

# A call's arguments travel as packed words: ctypes would spend 2 us on converting thirty of them one by one.
(_CONV, _CONV_VARLEN, _CONV_BACKWARD, _SCAN, _SCAN_TRAIN, _SCAN_VARLEN, _SCAN_BACKWARD, _STORE_WRITE, _STORE_READ) = (
    (op, struct.Struct(f"{len(_native.SSM_SIGNATURES[name][1])}q").pack, len(_native.SSM_SIGNATURES[name][1]))
    for op, name in enumerate(_native.SSM_OPS))

_CODES = {torch.bfloat16: _native.WKV_BF16, torch.float32: _native.WKV_F32}
_ACTS = {None: _native.WKV_ACT_NONE, "none": _native.WKV_ACT_NONE, "silu": _native.WKV_ACT_SILU}
_FORMATS = {torch.int8: _native.WKV_STORE_INT8, torch.float8_e4m3fn: _native.WKV_STORE_E4M3}


class _Call:
    """What a call's tensors are held to: the device and dtype of its first token array."""

    __slots__ = ("ref", "dev", "dtype", "code")

    def __init__(self, ref, name, dims):
        if not isinstance(ref, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if ref.dim() != dims:
            raise ValueError(f"{name} must have {dims} dimensions, got {tuple(ref.shape)}")
        self.ref, self.dtype, self.dev = ref, ref.dtype, ref.get_device()
        self.code = _CODES.get(self.dtype)
        if self.code is None:
            raise TypeError(f"unsupported input dtype {ref.dtype} (bfloat16 or float32)")
        if self.dev < 0:
            raise ValueError(f"{name} must be a device tensor")

    def flat(self, t, name, shape, dtype=torch.float32):
        """The address of a contiguous tensor of this shape and dtype; 0 for None."""
        if t is None:
            return 0
        try:
            if t.shape == shape and t.dtype is dtype and t.get_device() == self.dev and t.is_contiguous():
                return t.data_ptr()
        except AttributeError:
            pass
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.device != self.ref.device:
            raise ValueError(f"{name} must be on {self.ref.device}, got {t.device}")
        raise ValueError(f"{name} must be contiguous")

    def rows(self, t, name, shape, lead, any_dtype=False):
        """A token array, its first ``lead`` dimensions the tokens': its address and the step between its rows."""
        try:
            if t.shape == shape and t.get_device() == self.dev and (t.dtype is self.dtype or any_dtype) and t.is_contiguous():
                return t.data_ptr(), shape[-1] if len(shape) == lead + 1 else shape[-1] * shape[-2]
        except AttributeError:
            pass
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not any_dtype and t.dtype != self.dtype:
            raise TypeError(f"token inputs must share one dtype: {name}={t.dtype}, {self.dtype}")
        if t.device != self.ref.device:
            raise ValueError(f"{name} must be on {self.ref.device}, got {t.device}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        return t.data_ptr(), _row_step(t, name, lead)

    def output(self, y, out_dtype):
        code, dt = _out_code(y, out_dtype)
        if y is not None:
            self.flat(y, "y", self.ref.shape, dt)
        else:
            y = self.like(self.ref, dt)
        return y, code

    def like(self, t, dtype):
        """An empty contiguous tensor of t's shape."""
        return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)

    def empty(self, shape, dtype=torch.float32):
        return self.ref.new_empty(shape, dtype=dtype)

    def status(self, dev_status):
        return self.flat(dev_status, "dev_status", (1,), torch.int32)


def _row_step(t, name, lead):
    """The step between the rows of a token array, in elements."""
    cols = 1
    for w in t.shape[lead:]:
        cols *= w
    if t.numel() == 0:
        return cols
    st, step = t.stride(), 1
    for i in range(t.dim() - 1, lead - 1, -1):
        if t.shape[i] != 1 and st[i] != step:
            raise ValueError(f"{name} must be contiguous within a row, got strides {st}")
        step *= t.shape[i]
    outer = [i for i in range(lead) if t.shape[i] != 1]
    step = st[outer[-1]] if outer else cols
    if len(outer) == 2 and st[0] != t.shape[1] * step:
        raise ValueError(f"{name} must have one step between all rows, got strides {st}")
    if step < cols:
        raise ValueError(f"{name} has rows of {cols} elements {step} apart")
    return step


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _launch(dev, to, *args):
    """Calls the library with the current stream of the tensors' device, that device being current."""
    op, pack, count = to
    if dev == torch._C._cuda_getDevice():
        status = _call_words(op, pack(*args, torch._C._cuda_getCurrentRawStream(dev)), count)
    else:
        with torch.cuda.device(dev):
            status = _call_words(op, pack(*args, torch.cuda.current_stream(dev).cuda_stream), count)
    if status:
        check(status)


def _dense_states(call, state, state_map, state_out, return_state, B, inner):
    n_state = 0
    if state is not None:
        n_state = state.shape[0] if isinstance(state, torch.Tensor) and state.dim() else 0
    si = call.flat(state, "state", (n_state, *inner))
    mp = call.flat(state_map, "state_map", (B,), torch.int32)
    if state_out is not None:
        so = call.flat(state_out, "state_out", (B, *inner))
    else:
        state_out = call.empty((B, *inner)) if return_state else None
        so = _ptr(state_out)
    return (si, mp, n_state, so), state_out


def _slot_states(call, lengths, state, state_map, state_out, inner):
    if not isinstance(lengths, torch.Tensor) or lengths.dim() != 1:
        raise TypeError("lengths must be a one-dimensional torch.Tensor")
    if not isinstance(state, torch.Tensor) or not state.dim():
        raise TypeError("state must be a torch.Tensor of states")
    S, n_state = lengths.shape[0], state.shape[0]
    shape = (n_state, *inner)
    si = call.flat(state, "state", shape)
    so = si if state_out is None else call.flat(state_out, "state_out", shape)
    return S, call.flat(lengths, "lengths", (S,), torch.int32), (si, so, call.flat(state_map, "state_map", (S,), torch.int32), n_state)


def _conv_params(call, weight, bias, activation):
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [D, W]")
    if activation not in _ACTS:
        raise ValueError(f"unknown activation {activation!r} (None or 'silu')")
    D, W = call.ref.shape[-1], weight.shape[1]
    return W, (call.flat(weight, "weight", (D, W)), call.flat(bias, "bias", (D,)), _ACTS[activation])


def ssm_conv_forward(x, weight, bias=None, state=None, state_map=None, *, activation=None, y=None, state_out=None,
                     return_state=True, dev_status=None, out_dtype=torch.float32):
    """Short causal convolution of each channel: ``y_t = act(bias + sum_j weight[:, j] x_(t-W+1+j))``.

    x: [B, T, D]; weight: [D, W] fp32, W = 2, 3 or 4; bias: [D] fp32; ``activation``: None or "silu".
    ``state``: [n_state, W-1, D] fp32, the inputs before the first token, oldest first (None: zeros);
    ``state_map``: [B] int32.  With W = 2 and the taps (mu, 1 - mu) this is RWKV's token shift.
    Returns ``(y [B, T, D], state_out [B, W-1, D] or None)``; y is ``out_dtype`` unless given.
    """
    call = _Call(x, "x", 3)
    B, T, D = x.shape
    W, par = _conv_params(call, weight, bias, activation)
    states, state_out = _dense_states(call, state, state_map, state_out, return_state, B, (W - 1, D))
    y, oc = call.output(y, out_dtype)
    _launch(call.dev, _CONV, B, T, D, W, *call.rows(x, "x", x.shape, 2), call.code, *par, y.data_ptr(), oc,
            *states, call.status(dev_status))
    return y, state_out


def ssm_conv_backward(x, weight, bias, dy, state=None, state_map=None, *, activation=None, d_state=None,
                      return_d_state=True, dev_status=None, grad_dtype=torch.float32):
    """Gradients of :func:`ssm_conv_forward` (the same inputs, T >= 1).

    ``dy`` [B, T, D] (float32 or bfloat16) is the gradient of y, ``d_state`` [B, W-1, D] fp32 that of the final
    state.  Returns ``(dx [B, T, D] in grad_dtype, dweight [D, W], dbias [D] or None, d_state_in [B, W-1, D] or
    None)``, the last three in float32; ``d_state_in[b]`` belongs to the initial state row b started from.
    """
    call = _Call(x, "x", 3)
    B, T, D = x.shape
    W, par = _conv_params(call, weight, bias, activation)
    (si, mp, n_state, _), _ = _dense_states(call, state, state_map, None, False, B, (W - 1, D))
    if not isinstance(dy, torch.Tensor) or dy.dtype not in _CODES:
        raise TypeError("dy must be a bfloat16 or float32 torch.Tensor")
    if grad_dtype not in _CODES:
        raise TypeError(f"unsupported gradient dtype {grad_dtype} (bfloat16 or float32)")
    ds = call.flat(d_state, "d_state", (B, W - 1, D))
    dx, dw = call.like(x, grad_dtype), call.like(weight, torch.float32)
    db = call.like(bias, torch.float32) if bias is not None else None
    d_first = call.empty((B, W - 1, D)) if return_d_state else None
    need = _lib.wkv_ssm_conv_backward_workspace(B, T, D, W)
    ws = call.empty((need // 4,))
    _launch(call.dev, _CONV_BACKWARD, B, T, D, W, *call.rows(x, "x", x.shape, 2), call.code, *par,
            *call.rows(dy, "dy", x.shape, 2, any_dtype=True), _CODES[dy.dtype], si, mp, n_state, ds, _ptr(dx), _CODES[grad_dtype],
            _ptr(dw), _ptr(db), _ptr(d_first), _ptr(ws), need, call.status(dev_status))
    return dx, dw, db, d_first


def ssm_conv_forward_varlen(lengths, x, weight, bias, state, *, max_len, state_out=None, state_map=None,
                            activation=None, y=None, dev_status=None, out_dtype=torch.float32):
    """:func:`ssm_conv_forward` over packed rows of slots; updates ``state_out`` (default: ``state`` in place).

    ``lengths``: [S] int32 device tensor (tokens each slot consumes, at most ``max_len``); x: [tokens, D];
    ``state``: [n_state, W-1, D] fp32; ``state_map``: [S] int32.  Returns y [tokens, D].
    """
    call = _Call(x, "x", 2)
    total, D = x.shape
    W, par = _conv_params(call, weight, bias, activation)
    S, ln, states = _slot_states(call, lengths, state, state_map, state_out, (W - 1, D))
    y, oc = call.output(y, out_dtype)
    _launch(call.dev, _CONV_VARLEN, S, D, W, ln, int(max_len), total, *call.rows(x, "x", x.shape, 1), call.code,
            *par, y.data_ptr(), oc, *states, call.status(dev_status))
    return y


def _scan_args(call, x, dt, A, B, C, D, z, dt_bias, dt_softplus):
    """(channels, states, groups, the C ABI's input arguments) of a scan call."""
    shape = x.shape
    k, width = len(shape) - 1, shape[-1]
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be [D, N]")
    if not isinstance(B, torch.Tensor) or B.dim() not in (k + 1, k + 2):
        raise ValueError("B must be [..., N] or [..., G, N] with the token dimensions of x")
    N = A.shape[1]
    G = B.shape[-2] if B.dim() == k + 2 else 1
    inner = (*shape[:k], G, N) if B.dim() == k + 2 else (*shape[:k], N)
    return width, N, G, (*call.rows(x, "x", shape, k), *call.rows(dt, "dt", shape, k), call.flat(A, "A", (width, N)),
                         *call.rows(B, "B", inner, k), *call.rows(C, "C", inner, k), call.code, call.flat(D, "D", (width,)),
                         *(call.rows(z, "z", shape, k) if z is not None else (0, 0)),
                         call.flat(dt_bias, "dt_bias", (width,)), 1 if dt_softplus else 0)


def _workspace(call, rows, T, total, width, N, G):
    """Memory for a scan that is cut into segments, allocated on the current stream for one call, or None; its bytes."""
    need = _lib.wkv_ssm_scan_workspace(rows, T, total, width, N, G) if T > 64 else 0
    return (call.empty((need // 4,)) if need else None), need


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
    call = _Call(x, "x", 3)
    rows, T, _ = x.shape
    width, N, G, args = _scan_args(call, x, dt, A, B, C, D, z, dt_bias, dt_softplus)
    states, state_out = _dense_states(call, state, state_map, state_out, return_state, rows, (width, N))
    y, oc = call.output(y, out_dtype)
    ws, ws_bytes = _workspace(call, rows, T, rows * T, width, N, G)
    _launch(call.dev, _SCAN, rows, T, width, N, G, *args, y.data_ptr(), oc, *states, _ptr(ws), ws_bytes,
            call.status(dev_status))
    return y, state_out


def _chunks(T):
    return max((T + 15) // 16 - 1, 0)


def ssm_scan_forward_train(x, dt, A, B, C, D=None, z=None, dt_bias=None, state=None, state_map=None, *, dt_softplus=True,
                           y=None, state_out=None, return_state=True, dev_status=None, out_dtype=torch.float32,
                           chunk_states=None):
    """:func:`ssm_scan_forward` that also saves the state at every 16-token boundary for :func:`ssm_scan_backward`.

    Returns ``(y, state_out or None, chunk_states [B, ceil(T/16) - 1, D, N] fp32)``.
    """
    call = _Call(x, "x", 3)
    rows, T, _ = x.shape
    width, N, G, args = _scan_args(call, x, dt, A, B, C, D, z, dt_bias, dt_softplus)
    states, state_out = _dense_states(call, state, state_map, state_out, return_state, rows, (width, N))
    y, oc = call.output(y, out_dtype)
    saved = (rows, _chunks(T), width, N)
    if chunk_states is None:
        chunk_states = call.empty(saved)
    ws, ws_bytes = _workspace(call, rows, T, rows * T, width, N, G)
    _launch(call.dev, _SCAN_TRAIN, rows, T, width, N, G, *args, y.data_ptr(), oc, *states,
            call.flat(chunk_states, "chunk_states", saved), _ptr(ws), ws_bytes, call.status(dev_status))
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
    call = _Call(x, "x", 3)
    rows, T, _ = x.shape
    width, N, G, args = _scan_args(call, x, dt, A, B, C, D, z, dt_bias, dt_softplus)
    (si, mp, n_state, _), _ = _dense_states(call, state, state_map, None, False, rows, (width, N))
    if not isinstance(dy, torch.Tensor) or dy.dtype not in _CODES:
        raise TypeError("dy must be a bfloat16 or float32 torch.Tensor")
    if grad_dtype not in _CODES:
        raise TypeError(f"unsupported gradient dtype {grad_dtype} (bfloat16 or float32)")
    dya = call.rows(dy, "dy", x.shape, 2, any_dtype=True)
    chunks = call.flat(chunk_states, "chunk_states", (rows, _chunks(T), width, N))
    ds = call.flat(d_state, "d_state", (rows, width, N))
    dx, ddt = call.like(x, grad_dtype), call.like(dt, grad_dtype)
    dB, dC = call.like(B, grad_dtype), call.like(C, grad_dtype)
    dz = call.like(z, grad_dtype) if z is not None else None
    dA = call.like(A, torch.float32)
    dD = call.like(D, torch.float32) if D is not None else None
    db = call.like(dt_bias, torch.float32) if dt_bias is not None else None
    d_first = call.empty((rows, width, N)) if return_d_state else None
    need = _lib.wkv_ssm_scan_backward_workspace(rows, T, width, N, G, int(chunks != 0 or _chunks(T) == 0))
    ws = call.empty((need // 4,))
    _launch(call.dev, _SCAN_BACKWARD, rows, T, width, N, G, *args, *dya, _CODES[dy.dtype], si, mp, n_state, chunks, ds,
            _ptr(dx), _ptr(ddt), _ptr(dB), _ptr(dC), _ptr(dz), _CODES[grad_dtype], _ptr(dA), _ptr(dD), _ptr(db),
            _ptr(d_first), _ptr(ws), need, call.status(dev_status))
    return dx, ddt, dA, dB, dC, dD, dz, db, d_first


def ssm_scan_forward_varlen(lengths, x, dt, A, B, C, state, *, max_len, D=None, z=None, dt_bias=None, state_out=None,
                            state_map=None, dt_softplus=True, y=None, dev_status=None, out_dtype=torch.float32):
    """:func:`ssm_scan_forward` over packed rows of slots; updates ``state_out`` (default: ``state`` in place).

    ``lengths``: [S] int32 device tensor; x, dt, z: [tokens, D]; B, C: [tokens, N] or [tokens, G, N];
    ``state``: [n_state, D, N] fp32; ``state_map``: [S] int32.  Returns y [tokens, D].
    """
    call = _Call(x, "x", 2)
    total = x.shape[0]
    width, N, G, args = _scan_args(call, x, dt, A, B, C, D, z, dt_bias, dt_softplus)
    S, ln, states = _slot_states(call, lengths, state, state_map, state_out, (width, N))
    y, oc = call.output(y, out_dtype)
    ws, ws_bytes = _workspace(call, S, int(max_len), total, width, N, G)
    _launch(call.dev, _SCAN_VARLEN, S, width, N, G, ln, int(max_len), total, *args, y.data_ptr(), oc,
            *states, _ptr(ws), ws_bytes, call.status(dev_status))
    return y


def state_store_alloc(n_store, row, *, format=torch.int8, device="cuda"):
    """An empty 8-bit store of ``n_store`` rows of ``row`` values: ``(data, scale)`` (format: torch.int8 or
    torch.float8_e4m3fn).  Every row reads back as zeros until it is written."""
    if format not in _FORMATS:
        raise TypeError(f"unsupported store format {format} (torch.int8 or torch.float8_e4m3fn)")
    data = torch.zeros((n_store, row), dtype=torch.int8, device=device).view(format)
    return data, torch.zeros((n_store, (row + 63) // 64), dtype=torch.float32, device=device)


def _store_call(fn, data, scale, states, store_rows, state_rows, dev_status):
    if not isinstance(data, torch.Tensor) or data.dim() != 2:
        raise ValueError("data must be [n_store, row]")
    fmt = _FORMATS.get(data.dtype)
    if fmt is None:
        raise TypeError(f"unsupported store format {data.dtype} (torch.int8 or torch.float8_e4m3fn)")
    if not data.is_cuda or not data.is_contiguous():
        raise ValueError("data must be a contiguous device tensor")
    call = _Call(states, "states", states.dim() if isinstance(states, torch.Tensor) else 0)
    (n_store, row), n_state = data.shape, states.shape[0] if states.dim() else 0
    if states.dim() < 2 or (n_state and states.numel() != n_state * row):
        raise ValueError(f"states must be [n_state, ...] with {row} values a row, got {tuple(states.shape)}")
    n = store_rows.shape if store_rows is not None else state_rows.shape if state_rows is not None else (n_state,)
    if len(n) != 1:
        raise ValueError("store_rows and state_rows must be one-dimensional")
    _launch(call.dev, fn, call.flat(data, "data", data.shape, data.dtype), call.flat(scale, "scale", (n_store, (row + 63) // 64)),
            n_store, fmt, call.flat(states, "states", states.shape), n_state, row, call.flat(store_rows, "store_rows", n, torch.int32),
            call.flat(state_rows, "state_rows", n, torch.int32), n[0], call.status(dev_status))


def state_store_write(data, scale, states, store_rows=None, state_rows=None, *, dev_status=None):
    """Writes rows of ``states`` ([n_state, ...] fp32: WKV, convolution or scan states) into the 8-bit store
    ``data`` [n_store, row] (int8 or float8_e4m3fn), ``scale`` [n_store, ceil(row / 64)] fp32.

    Item i stores ``states[state_rows[i]]`` as row ``store_rows[i]`` (int32 device tensors; None: i).
    Groups of 64 consecutive values share the scale max|v| / 127 (int8) or / 448 (e4m3).
    """
    _store_call(_STORE_WRITE, data, scale, states, store_rows, state_rows, dev_status)


def state_store_read(data, scale, states, store_rows=None, state_rows=None, *, dev_status=None):
    """Reads rows of the 8-bit store back into ``states`` (see :func:`state_store_write`); one stored row may
    be read into many state rows.  Returns ``states``."""
    _store_call(_STORE_READ, data, scale, states, store_rows, state_rows, dev_status)
    return states
