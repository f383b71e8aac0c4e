"""Gradients of the state space operators on the GPU: against automatic differentiation of their definitions in 64 bits,
against differences of those definitions, across segments, groups, views, options and captured graphs."""
import pytest
import torch

import rwkv_linear_attention_wkv_amd as wkv
import ssm_reference as ref
from ssm_reference import allowed, assert_within, d64
from test_ssm_forward_gpu import conv_case, draw, gpu, scan_case

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------------------------------------ convolution

def conv_back(c, dy, d_state, act, state=True, bias=True, **kw):
    return wkv.ssm_conv_backward(gpu(c["x"]), gpu(c["weight"]), gpu(c["bias"]) if bias else None, gpu(dy),
                                 gpu(c["state"]) if state else None, activation=act, d_state=gpu(d_state), **kw)


def check_conv_grads(c, dy, d_state, act, got, state=True, bias=True, grad=F32):
    """An activation's slope is at most 1.1 and changes by at most 0.5 per unit of its argument, whose own error counts
    the W + 1 roundings of its sum; the rest are the products' and the sums' own, in 16 interleaved parts."""
    B, T, D = c["x"].shape
    W = c["weight"].shape[1]
    dx, dw, db, d_first = got
    tw, tb, mw, mb = 0, 0, 0, 0
    for b in range(B):
        first = d64(c["state"][b]) if state else torch.zeros(W - 1, D, dtype=torch.float64)
        x, w, bi = d64(c["x"][b]), d64(c["weight"]), d64(c["bias"]) if bias else None
        rx, rw, rb, rf = ref.conv_grads(x, w, bi, first, act, d64(dy[b]), None if d_state is None else d64(d_state[b]))
        _, mag, _ = ref.conv(x, w, bi, first, act)
        g = d64(dy[b]).abs() * (1.1 + mag)  # what one output passes back, with room for its slope's error
        line = torch.cat((first, x)).abs()
        mx = torch.zeros_like(line)
        for j in range(W):
            mx[j:j + T] += w[:, j].abs() * g
        if d_state is not None:
            mx[T:] += d64(d_state[b]).abs()
        assert_within(dx[b], rx, allowed(mx[W - 1:], 64, rx, grad), f"dx[{b}]")
        assert_within(d_first[b], rf, allowed(mx[:W - 1], 64), f"d_state_in[{b}]")
        tw, mw = tw + rw, mw + torch.stack([(g * line[j:j + T]).sum(0) for j in range(W)], 1)
        if bias:
            tb, mb = tb + rb, mb + g.sum(0)
    assert_within(dw, tw, allowed(mw, 64 + B * T), "dweight")
    if bias:
        assert_within(db, tb, allowed(mb, 64 + B * T), "dbias")
    else:
        assert db is None


@pytest.mark.parametrize("B,T,D,W,dtype,grad,act", [
    (2, 1, 64, 4, BF16, BF16, "silu"),
    (1, 2, 8, 4, F32, F32, "silu"),
    (2, 3, 7, 3, BF16, F32, None),
    (3, 64, 33, 2, F32, BF16, "silu"),
    (2, 66, 36, 4, F32, F32, "silu"),
    (2, 130, 130, 3, BF16, BF16, "silu"),
    (1, 257, 520, 4, BF16, BF16, "silu"),
])
@pytest.mark.parametrize("with_state", [True, False])
def test_conv_backward(B, T, D, W, dtype, grad, act, with_state):
    c = conv_case(B, T, D, W, dtype)
    dy, ds = draw(7, B, T, D, dtype=grad), draw(8, B, W - 1, D) if with_state else None
    got = conv_back(c, dy, ds, act, with_state, grad_dtype=grad)
    assert got[0].dtype == grad
    check_conv_grads(c, dy, ds, act, got, with_state, grad=grad)


def test_conv_backward_of_views_and_without_bias():
    c = conv_case(2, 37, 64, 4, BF16)
    wide, wide_dy = draw(9, 2, 37, 150, dtype=BF16), draw(10, 2, 37, 130)
    c["x"] = wide[..., 5:69]
    dy = wide_dy[..., 64:128]
    on = dict(c, x=gpu(wide)[..., 5:69])
    got = conv_back(on, gpu(wide_dy)[..., 64:128], None, "silu", bias=False)
    check_conv_grads(c, dy, None, "silu", got, bias=False)


def test_conv_backward_rejected_row_has_no_share():
    c = conv_case(3, 70, 40, 4, F32, n_state=4)
    dy = draw(7, 3, 70, 40)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = gpu(torch.tensor([3, 4, 0], dtype=torch.int32))
    got = wkv.ssm_conv_backward(gpu(c["x"]), gpu(c["weight"]), gpu(c["bias"]), gpu(dy), gpu(c["state"]), rows,
                                activation="silu", dev_status=status)
    assert int(status) == wkv.WKV_DEV_BAD_STATE_MAP
    keep = dict(c, x=c["x"][[0, 2]], state=c["state"][[3, 0]])
    check_conv_grads(keep, dy[[0, 2]], None, "silu", (got[0][[0, 2]], got[1], got[2], got[3][[0, 2]]))


# ------------------------------------------------------------------------------------------------------- scan

NAMES = ("x", "dt", "A", "B", "C", "skip", "z", "bias", "first")


def scan_back(c, dy, d_state, state=True, **kw):
    return wkv.ssm_scan_backward(*(gpu(c[k]) for k in ("x", "dt", "A", "B", "C")), gpu(dy), gpu(c["D"]), gpu(c["z"]),
                                 gpu(c["dt_bias"]), gpu(c["state"]) if state else None, d_state=gpu(d_state), **kw)


def check_scan_grads(c, dy, d_state, got, state=True, grad=F32, softplus_on=True):
    """Every term passes the 2 T decays between its token and the state or gradient that it meets (4 roundings each, as
    in the forward pass), its own factors, and the sums over states, channels and tokens."""
    rows, T, D = c["x"].shape
    N = c["A"].shape[1]
    got = dict(zip(NAMES, (got[0], got[1], got[2], got[3], got[4], got[5], got[6], got[7], got[8])))
    count = 8 * T + 128
    total, mags = {}, {}
    for b in range(rows):
        first = c["state"][b] if state else torch.zeros(D, N)
        tok = lambda v: None if c[v] is None else d64(c[v][b])  # noqa: E731
        wide = lambda v: d64(c[v][b]).reshape(T, -1, N)  # noqa: E731
        want, mag = ref.scan_grads(tok("x"), tok("dt"), d64(c["A"]), wide("B"), wide("C"), d64(c["D"]), tok("z"),
                                   d64(c["dt_bias"]), d64(first), d64(dy[b]), None if d_state is None else d64(d_state[b]),
                                   softplus_on)
        for k in ("x", "dt", "z"):
            if c[k] is not None:
                assert_within(got[k][b], want[k], allowed(mag[k], count, want[k], grad), f"d{k}[{b}]")
        for k in ("B", "C"):
            w, m = (v[k].reshape(got[k][b].shape) for v in (want, mag))
            assert_within(got[k][b], w, allowed(m, count + D, w, grad), f"d{k}[{b}]")
        if got["first"] is not None:
            assert_within(got["first"][b], want["first"], allowed(mag["first"], count), f"d_state_in[{b}]")
        for k in ("A", "skip", "bias"):
            if want.get(k) is not None:
                total[k], mags[k] = total.get(k, 0) + want[k], mags.get(k, 0) + mag[k]
    for k in total:
        assert_within(got[k], total[k], allowed(mags[k], count + T + rows), f"d{k}")


SCANS = [
    (2, 1, 64, 16, 0, BF16, BF16),
    (1, 2, 4, 1, 0, F32, F32),
    (2, 9, 33, 4, 1, F32, F32),
    (1, 16, 68, 16, 0, BF16, F32),
    (2, 17, 130, 8, 0, BF16, BF16),
    (1, 33, 66, 16, 2, F32, BF16),
    (2, 65, 21, 11, 3, F32, F32),
    (1, 50, 40, 32, 1, BF16, F32),
    (1, 49, 18, 64, 2, F32, F32),
    (1, 70, 9, 37, 1, F32, F32),
    (2, 100, 200, 5, 1, BF16, BF16),
]


@pytest.mark.parametrize("B,T,D,N,G,dtype,grad", SCANS)
@pytest.mark.parametrize("with_state", [True, False])
def test_scan_backward(B, T, D, N, G, dtype, grad, with_state):
    c = scan_case(B, T, D, N, G, dtype)
    dy, ds = draw(11, B, T, D, dtype=grad), draw(12, B, D, N) if with_state else None
    got = scan_back(c, dy, ds, with_state, grad_dtype=grad)
    assert got[0].dtype == got[3].dtype == got[6].dtype == grad and got[2].dtype == F32
    check_scan_grads(c, dy, ds, got, with_state, grad)


@pytest.mark.parametrize("z,skip,bias,sp", [(False, False, False, True), (True, False, True, False), (False, True, False, True)])
def test_scan_backward_without_options(z, skip, bias, sp):
    c = scan_case(2, 40, 36, 16, 0, F32, z=z, skip=skip, bias=bias)
    if not sp:
        c["dt"], c["dt_bias"] = 0.1 * c["dt"], torch.full((36,), 0.05)
    dy = draw(11, 2, 40, 36)
    got = scan_back(c, dy, None, dt_softplus=sp, return_d_state=False)
    assert got[8] is None and (got[6] is None) == (not z) and (got[5] is None) == (not skip)
    check_scan_grads(c, dy, None, got, softplus_on=sp)


@pytest.mark.parametrize("D,G", [(65, 1), (67, 1), (70, 1), (130, 2)])
def test_scan_backward_channels_of_part_blocks(D, G):
    """The last block of channels of a group with 1, 3, 6 and 1 of its 64: their sums hold nothing else."""
    c = scan_case(1, 20, D, 16, G, F32)
    dy, ds = draw(11, 1, 20, D), draw(12, 1, D, 16)
    check_scan_grads(c, dy, ds, scan_back(c, dy, ds))


@pytest.mark.parametrize("D", [1, 3, 5, 9, 261])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_conv_backward_any_channel_count(D, dtype):
    c = conv_case(2, 33, D, 4, dtype)
    dy, ds = draw(7, 2, 33, D, dtype=dtype), draw(8, 2, 3, D)
    check_conv_grads(c, dy, ds, "silu", conv_back(c, dy, ds, "silu", grad_dtype=dtype), grad=dtype)


@pytest.mark.parametrize("T,D,N,dtype", [(300, 70, 16, F32), (450, 40, 32, BF16), (333, 24, 7, F32)])
def test_scan_backward_across_segments(T, D, N, dtype):
    """Rows that are cut into segments, in both passes."""
    assert wkv.library().wkv_ssm_scan_workspace(1, T, T, D, N, 1) > 0
    c = scan_case(1, T, D, N, 0, dtype)
    dy, ds = draw(11, 1, T, D), draw(12, 1, D, N)
    check_scan_grads(c, dy, ds, scan_back(c, dy, ds))


@pytest.mark.parametrize("B,T,D,N", [(2, 50, 64, 16), (1, 400, 40, 16), (2, 16, 24, 8), (1, 9, 24, 8), (3, 130, 20, 40)])
def test_scan_forward_train_and_saved_states(B, T, D, N):
    """The saving forward pass gives the plain one's results; the gradients are bitwise those without saved states."""
    c = scan_case(B, T, D, N, 0, F32)
    args = [gpu(c[k]) for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "state")]
    y, last = wkv.ssm_scan_forward(*args)
    yt, lt, chunks = wkv.ssm_scan_forward_train(*args)
    assert torch.equal(y, yt) and torch.equal(last, lt) and chunks.shape == (B, -(-T // 16) - 1, D, N)
    for k in range(chunks.shape[1]):
        cut = {n: v[:, :16 * (k + 1)].contiguous() if n in ("x", "dt", "B", "C", "z") else v for n, v in c.items()}
        _, s = wkv.ssm_scan_forward(*(gpu(cut[n]) for n in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "state")))
        torch.testing.assert_close(chunks[:, k], s, rtol=1e-4, atol=1e-5)
    dy, ds = draw(11, B, T, D), draw(12, B, D, N)
    with_saved, without = scan_back(c, dy, ds, chunk_states=chunks), scan_back(c, dy, ds)
    for a, b in zip(with_saved, without):
        assert torch.equal(a, b)


def test_scan_backward_of_views():
    B, T, D, N = 2, 40, 64, 16
    c = scan_case(B, T, D, N, 0, BF16)
    xz, dbc, wdy = draw(30, B, T, 2 * D + 3, dtype=BF16), draw(31, B, T, D + 2 * N, dtype=BF16, std=0.5), draw(32, B, T, D + 1)
    host = dict(x=xz[..., 3:D + 3], z=xz[..., D + 3:], dt=dbc[..., :D], B=dbc[..., D:D + N], C=dbc[..., D + N:])
    a, b, w = gpu(xz), gpu(dbc), gpu(wdy)
    on = dict(c, x=a[..., 3:D + 3], z=a[..., D + 3:], dt=b[..., :D], B=b[..., D:D + N], C=b[..., D + N:])
    got = scan_back(on, w[..., 1:], None)
    check_scan_grads(dict(c, **host), wdy[..., 1:], None, got)


def test_scan_backward_padding_and_strong_decays():
    """Steps of zero (dt = -inf) pass gradients through; decays down to 0 and of exactly 1."""
    c = scan_case(1, 40, 32, 16, 0, F32)
    c["A"][:, 0], c["A"][:, 1], c["A"][:8, 2] = 0.0, -1e20, -300.0
    c["dt"][:, 30:] = -200.0  # e^-200: a step of zero in fp32, with a slope of zero
    dy, ds = draw(11, 1, 40, 32), draw(12, 1, 32, 16)
    got = scan_back(c, dy, ds)
    assert all(torch.isfinite(g).all() for g in got)
    check_scan_grads(c, dy, ds, got)
    c["dt"][:, 30:] = float("-inf")
    again = scan_back(c, dy, ds)
    for a, b in zip(got, again):
        assert torch.equal(a, b)


def test_scan_backward_rejected_row_has_no_share():
    c = scan_case(3, 40, 24, 16, 0, F32, n_state=4)
    dy = draw(11, 3, 40, 24)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = gpu(torch.tensor([3, 4, 0], dtype=torch.int32))
    got = scan_back(c, dy, None, state_map=rows, dev_status=status)
    assert int(status) == wkv.WKV_DEV_BAD_STATE_MAP
    keep = {k: v[[0, 2]] if k in ("x", "dt", "B", "C", "z") else v for k, v in c.items()}
    keep["state"] = c["state"][[3, 0]]
    pick = lambda i, g: g[[0, 2]] if i in (0, 1, 3, 4, 6, 8) else g  # noqa: E731
    check_scan_grads(keep, dy[[0, 2]], None, tuple(pick(i, g) for i, g in enumerate(got)))


@pytest.mark.parametrize("T", [30, 200])
def test_gradients_against_differences(T):
    """The change of the loss in 64 bits along a direction in every input at once equals the kernels' gradients along it."""
    B, D, N = 1, 24, 16
    c = scan_case(B, T, D, N, 0, F32)
    dy, ds = draw(11, B, T, D), draw(12, B, D, N)
    got = dict(zip(("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "state"), scan_back(c, dy, ds)))
    move = {k: draw(40 + i, *c[k].shape) for i, k in enumerate(got)}

    def loss(eps):
        m = {k: d64(c[k]) + eps * d64(move[k]) for k in c}
        y, last = ref.scan(m["x"][0], m["dt"][0], m["A"], m["B"][0][:, None], m["C"][0][:, None], m["D"], m["z"][0],
                           m["dt_bias"], m["state"][0])
        return float((y * d64(dy[0])).sum() + (last * d64(ds[0])).sum())

    eps = 1e-5  # a third derivative of a thousand times the loss would show at 1e-7
    slope = (loss(eps) - loss(-eps)) / (2 * eps)
    along = [float((d64(g).reshape(-1) * d64(move[k]).reshape(-1)).sum()) for k, g in got.items()]
    size = sum(float((d64(g).reshape(-1) * d64(move[k]).reshape(-1)).abs().sum()) for k, g in got.items())
    assert abs(slope - sum(along)) <= size * (8 * T + 128) * 2.0 ** -24, (slope, sum(along), size)


def train_step(p, c, dy):
    """One layer's training step: convolution, scan, and their gradients."""
    D, N = p["A"].shape
    u, last = wkv.ssm_conv_forward(c["x"], p["weight"], p["bias"], activation="silu")
    y, _, chunks = wkv.ssm_scan_forward_train(u, c["dt"], p["A"], c["B"], c["C"], p["D"], c["z"], p["dt_bias"])
    g = wkv.ssm_scan_backward(u, c["dt"], p["A"], c["B"], c["C"], dy, p["D"], c["z"], p["dt_bias"], chunk_states=chunks)
    h = wkv.ssm_conv_backward(c["x"], p["weight"], p["bias"], g[0], activation="silu")
    return [y, *(t for t in g if t is not None), *h]


def test_training_step_equals_differentiated_definition():
    """Convolution and scan together: the gradients that reach the convolution's parameters."""
    B, T, D, N = 1, 40, 24, 16
    c = scan_case(B, T, D, N, 0, F32)
    p = dict(weight=draw(60, D, 4, std=0.5), bias=draw(61, D), A=c["A"], D=c["D"], dt_bias=c["dt_bias"])
    dy = draw(11, B, T, D)
    out = train_step({k: gpu(v) for k, v in p.items()}, {k: gpu(c[k]) for k in ("x", "dt", "B", "C", "z")}, gpu(dy))
    w, b, x = (d64(v).requires_grad_() for v in (p["weight"], p["bias"], c["x"][0]))
    u, _, _ = ref.conv(x, w, b, torch.zeros(3, D, dtype=torch.float64), True)
    y, _ = ref.scan(u, d64(c["dt"][0]), d64(c["A"]), d64(c["B"][0])[:, None], d64(c["C"][0])[:, None], d64(c["D"]), d64(c["z"][0]),
                    d64(c["dt_bias"]), torch.zeros(D, N, dtype=torch.float64))
    want = torch.autograd.grad((y * d64(dy[0])).sum(), (x, w, b))
    for got, g in zip((out[-4][0], out[-3], out[-2]), want):
        assert_within(got, g, allowed(g.abs().max() * torch.ones_like(g), 8 * T + 256), "through both")


@pytest.mark.parametrize("T", [20, 300])
def test_training_step_captured_and_replayed(T):
    """Eager steps on the same tensors between the replays; every replay equals the eager result on its inputs."""
    B, D, N = 1, 40, 16
    c = scan_case(B, T, D, N, 0, F32)
    p = {k: gpu(v) for k, v in dict(weight=draw(60, D, 4, std=0.5), bias=draw(61, D), A=c["A"], D=c["D"], dt_bias=c["dt_bias"]).items()}
    on = {k: gpu(c[k]) for k in ("x", "dt", "B", "C", "z")}
    dy = gpu(draw(11, B, T, D))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train_step(p, on, dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = train_step(p, on, dy)
    for k in range(3):
        on["x"].copy_(gpu(draw(90 + k, B, T, D)))
        dy.copy_(gpu(draw(95 + k, B, T, D)))
        want = train_step(p, on, dy)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
