"""Forward passes of the state space operators on the GPU against their definitions in 64 bits: dense rows, slots of
different lengths, single tokens, odd sizes, views, state maps, data errors."""
import pytest
import torch

import rwkv_linear_attention_wkv_amd as wkv
import ssm_reference as ref
from ssm_reference import allowed, assert_within, d64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def draw(seed, *shape, dtype=F32, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def gpu(t):
    return None if t is None else t if t.is_cuda else t.cuda()


# ------------------------------------------------------------------------------------------------ convolution

# W + 1 roundings of the sum; the activation passes it on with a slope of at most 1.1 and adds the errors of the
# exponential (its argument's rounding times |pre| < 16, 2 steps of its own), the reciprocal and two products.
CONV_ROUNDINGS = 32


def conv_case(B, T, D, W, dtype, seed=0, n_state=None):
    return dict(x=draw(seed, B, T, D, dtype=dtype), weight=draw(seed + 1, D, W, std=0.5), bias=draw(seed + 2, D),
                state=draw(seed + 3, n_state or B, W - 1, D))


def check_conv(x, weight, bias, firsts, act, y, last, out, what=""):
    for b in range(x.shape[0]):
        want, mag, wlast = ref.conv(d64(x[b]), d64(weight), d64(bias), d64(firsts[b]), act)
        assert_within(y[b], want, allowed(mag, CONV_ROUNDINGS, want, out), f"{what} y[{b}]")
        if last is not None:
            assert torch.equal(last[b].cpu().double(), wlast), f"{what}: state {b}"


@pytest.mark.parametrize("B,T,D,W,dtype,out,act", [
    (2, 1, 64, 4, BF16, BF16, "silu"),
    (1, 2, 8, 4, F32, F32, None),
    (2, 3, 7, 3, BF16, F32, "silu"),
    (1, 64, 1, 2, F32, BF16, "silu"),
    (3, 65, 33, 4, F32, F32, "silu"),
    (2, 130, 130, 3, BF16, BF16, None),
    (1, 257, 520, 4, BF16, BF16, "silu"),
    (2, 5, 2050, 2, BF16, F32, "silu"),
])
@pytest.mark.parametrize("with_state", [True, False])
def test_conv_forward(B, T, D, W, dtype, out, act, with_state):
    c = conv_case(B, T, D, W, dtype)
    state = c["state"] if with_state else None
    y, last = wkv.ssm_conv_forward(gpu(c["x"]), gpu(c["weight"]), gpu(c["bias"]), gpu(state), activation=act, out_dtype=out)
    assert y.dtype == out
    check_conv(c["x"], c["weight"], c["bias"], state if with_state else torch.zeros_like(c["state"]), act, y, last, out)


def test_conv_forward_without_bias_or_final_state():
    c = conv_case(2, 9, 48, 4, F32)
    y, last = wkv.ssm_conv_forward(gpu(c["x"]), gpu(c["weight"]), return_state=False)
    assert last is None
    check_conv(c["x"], c["weight"], None, torch.zeros(2, 3, 48), None, y, None, F32)


def test_conv_forward_empty_rows_hand_their_state_on():
    c = conv_case(2, 0, 48, 4, F32)
    y, last = wkv.ssm_conv_forward(gpu(c["x"]), gpu(c["weight"]), gpu(c["bias"]), gpu(c["state"]))
    assert y.shape == (2, 0, 48) and torch.equal(last.cpu(), c["state"])


@pytest.mark.parametrize("T", [1, 2, 70, 200])
def test_conv_in_place_state_and_carry(T):
    """Two calls that update the state in place equal one call over all tokens, bitwise."""
    c = conv_case(2, 2 * T, 96, 4, BF16)
    w, b, x = gpu(c["weight"]), gpu(c["bias"]), gpu(c["x"])
    whole, last = wkv.ssm_conv_forward(x, w, b, gpu(c["state"]), activation="silu")
    st = gpu(c["state"])
    parts = [wkv.ssm_conv_forward(x[:, i * T:(i + 1) * T].contiguous(), w, b, st, activation="silu", state_out=st)[0] for i in (0, 1)]
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(st, last)


@pytest.mark.parametrize("D", [1, 3, 5, 8, 9, 2051])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_conv_any_channel_count_in_place(D, dtype):
    """Channels past the last whole load, in their own block: rows and states of every count, updated in place."""
    c = conv_case(2, 33, D, 4, dtype)
    st = gpu(c["state"])
    y, last = wkv.ssm_conv_forward(gpu(c["x"]), gpu(c["weight"]), gpu(c["bias"]), st, activation="silu", state_out=st, out_dtype=dtype)
    check_conv(c["x"], c["weight"], c["bias"], c["state"], "silu", y, last, dtype)


def test_conv_state_map_and_shared_state():
    c = conv_case(3, 10, 40, 3, F32, n_state=5)
    rows = torch.tensor([4, 0, 4], dtype=torch.int32)
    y, last = wkv.ssm_conv_forward(gpu(c["x"]), gpu(c["weight"]), gpu(c["bias"]), gpu(c["state"]), gpu(rows))
    check_conv(c["x"], c["weight"], c["bias"], c["state"][rows.long()], None, y, last, F32)
    y, last = wkv.ssm_conv_forward(gpu(c["x"]), gpu(c["weight"]), gpu(c["bias"]), gpu(c["state"][:1]))
    check_conv(c["x"], c["weight"], c["bias"], c["state"][:1].expand(3, -1, -1), None, y, last, F32)


@pytest.mark.parametrize("dtype,lo", [(BF16, 64), (BF16, 3), (F32, 8), (F32, 5)])
def test_conv_rows_of_a_wider_array(dtype, lo):
    """x as columns lo .. lo + D of a projection's output, aligned to whole loads or not."""
    B, T, D = 2, 37, 64
    wide = draw(9, B, T, 2 * D + 8, dtype=dtype)
    c = conv_case(B, T, D, 4, dtype)
    view = gpu(wide)[..., lo:lo + D]
    y, last = wkv.ssm_conv_forward(view, gpu(c["weight"]), gpu(c["bias"]), gpu(c["state"]), activation="silu")
    check_conv(wide[..., lo:lo + D], c["weight"], c["bias"], c["state"], "silu", y, last, F32)


def test_token_shift_is_the_two_tap_form():
    """RWKV's token shift x_t + mu (x_(t-1) - x_t), the last token of the previous call carried."""
    x, mu, before = draw(1, 2, 20, 64), torch.rand(64, generator=torch.Generator().manual_seed(2)), draw(3, 2, 1, 64)
    y, last = wkv.ssm_conv_forward(gpu(x), gpu(torch.stack((mu, 1 - mu), 1)), state=gpu(before))
    prev = torch.cat((before, x[:, :-1]), 1).double()
    want = x.double() + mu.double() * (prev - x.double())
    assert_within(y, want, allowed(prev.abs() + x.double().abs(), 4), "token shift")
    assert torch.equal(last.cpu(), x[:, -1:])


LENGTHS = [[1] * 9, [0, 5, 1, 0, 70, 2, 200, 3], [3], [0, 0], [129, 64, 63, 65, 1, 0]]


def slots_of(lengths, seed, extra=3):
    """(state row of each slot, rows of the table): a permutation into a larger table."""
    n = len(lengths) + extra
    return torch.randperm(n, generator=torch.Generator().manual_seed(seed))[:len(lengths)].to(torch.int32), n


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("dtype,D,W", [(BF16, 72, 4), (F32, 33, 3), (BF16, 11, 2)])
def test_conv_varlen(lengths, dtype, D, W):
    """Slots of any length against their own sequences; other state rows and rows past the last slot stay."""
    total = sum(lengths)
    rows, n_state = slots_of(lengths, 5)
    x, state = draw(20, total + 4, D, dtype=dtype), draw(21, n_state, W - 1, D)
    weight, bias = draw(22, D, W, std=0.5), draw(23, D)
    st, status = gpu(state), torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full((total + 4, D), 77.0, device="cuda")
    ln = torch.tensor(lengths, dtype=torch.int32)
    wkv.ssm_conv_forward_varlen(gpu(ln), gpu(x), gpu(weight), gpu(bias), st, max_len=max(lengths), state_map=gpu(rows),
                                activation="silu", y=y, dev_status=status)
    assert int(status) == 0 and (y[total:] == 77).all()
    off, want = 0, d64(state)
    for s, n in enumerate(lengths):
        wy, mag, last = ref.conv(d64(x[off:off + n]), d64(weight), d64(bias), d64(state[rows[s]]), "silu")
        assert_within(y[off:off + n], wy, allowed(mag, CONV_ROUNDINGS), f"slot {s}")
        want[rows[s]] = last
        off += n
    assert torch.equal(st.cpu().double(), want)
    out = torch.full_like(st, 5.0)  # out of place: the slots' rows only, empty slots copied
    wkv.ssm_conv_forward_varlen(gpu(ln), gpu(x), gpu(weight), gpu(bias), gpu(state), max_len=max(lengths),
                                state_map=gpu(rows), state_out=out)
    keep = torch.ones(n_state, dtype=torch.bool)
    keep[rows.long()] = False
    assert (out[gpu(keep)] == 5).all() and torch.equal(out[gpu(~keep)].cpu().double(), want[~keep])


# ------------------------------------------------------------------------------------------------------- scan

def scan_roundings(T):
    """A state passes T decays, each with the roundings of its exponent (|delta A| small against 2) and its own two,
    and one multiply-add; a step's own factors, the sum over the states and the gate add under 64."""
    return 4 * T + 64


def scan_case(B, T, D, N, G, dtype, seed=0, n_state=None, z=True, skip=True, bias=True, lead=None):
    lead = lead or (B, T)
    bc = (G, N) if G else (N,)
    step = torch.exp(draw(seed + 5, D, std=1.0) - 3.5)
    return dict(x=draw(seed, *lead, D, dtype=dtype), dt=draw(seed + 1, *lead, D, dtype=dtype, std=0.5),
                A=-torch.exp(draw(seed + 2, D, N, std=0.7)), B=draw(seed + 3, *lead, *bc, dtype=dtype),
                C=draw(seed + 4, *lead, *bc, dtype=dtype), D=1 + draw(seed + 6, D) if skip else None,
                z=draw(seed + 7, *lead, D, dtype=dtype) if z else None,
                dt_bias=step + torch.log(-torch.expm1(-step)) if bias else None,
                state=draw(seed + 8, n_state or B, D, N))


def scan_ref(c, first, at=slice(None), **kw):
    """The definition of one sequence of a case: tokens ``at`` of row or packed arrays, from state ``first``."""
    D, N = c["A"].shape
    tok = lambda v: None if c[v] is None else d64(c[v][at])  # noqa: E731
    wide = lambda v: d64(c[v][at]).reshape(-1, c[v].shape[-2] if c[v].dim() > c["x"].dim() else 1, N)  # noqa: E731
    return ref.scan(tok("x"), tok("dt"), d64(c["A"]), wide("B"), wide("C"), d64(c["D"]), tok("z"), d64(c["dt_bias"]),
                    d64(first), **kw)


def check_scan(c, firsts, y, last, out, softplus_on=True):
    T = c["x"].shape[1]
    for b in range(c["x"].shape[0]):
        want, wl = scan_ref(c, firsts[b], b, softplus_on=softplus_on)
        mag, ml = scan_ref(c, firsts[b], b, softplus_on=softplus_on, absolute=True)
        assert_within(y[b], want, allowed(mag, scan_roundings(T), want, out), f"y[{b}]")
        if last is not None:
            assert_within(last[b], wl, allowed(ml, scan_roundings(T)), f"state {b}")


def run_scan(c, state, **kw):
    return wkv.ssm_scan_forward(gpu(c["x"]), gpu(c["dt"]), gpu(c["A"]), gpu(c["B"]), gpu(c["C"]), gpu(c["D"]), gpu(c["z"]),
                                gpu(c["dt_bias"]), gpu(state), **kw)


SCANS = [
    (2, 1, 64, 16, 0, BF16, BF16),
    (1, 2, 4, 1, 0, F32, F32),
    (2, 9, 33, 4, 1, F32, F32),
    (1, 31, 70, 8, 0, BF16, F32),
    (2, 33, 66, 16, 2, F32, BF16),
    (1, 100, 130, 16, 0, BF16, BF16),
    (2, 65, 21, 11, 3, F32, F32),
    (1, 64, 40, 32, 1, BF16, F32),
    (1, 97, 18, 64, 2, F32, F32),
    (1, 129, 9, 37, 1, F32, F32),
    (3, 130, 520, 5, 1, BF16, BF16),
]


@pytest.mark.parametrize("B,T,D,N,G,dtype,out", SCANS)
@pytest.mark.parametrize("with_state", [True, False])
def test_scan_forward(B, T, D, N, G, dtype, out, with_state):
    c = scan_case(B, T, D, N, G, dtype)
    state = c["state"] if with_state else None
    y, last = run_scan(c, state, out_dtype=out)
    assert y.dtype == out
    check_scan(c, state if with_state else torch.zeros_like(c["state"]), y, last, out)


@pytest.mark.parametrize("z,skip,bias,sp", [(False, False, False, True), (True, False, True, False), (False, True, False, True)])
def test_scan_forward_without_options(z, skip, bias, sp):
    c = scan_case(2, 40, 36, 16, 0, F32, z=z, skip=skip, bias=bias)
    if not sp:  # steps as they are, both signs
        c["dt"], c["dt_bias"] = 0.1 * c["dt"], 0.05 * c["D"].abs() if skip else torch.full((36,), 0.05)
    y, last = run_scan(c, c["state"], dt_softplus=sp)
    check_scan(c, c["state"], y, last, F32, softplus_on=sp)


def test_scan_forward_empty_rows_hand_their_state_on():
    c = scan_case(2, 0, 20, 16, 0, F32)
    y, last = run_scan(c, c["state"])
    assert y.shape == (2, 0, 20) and torch.equal(last.cpu(), c["state"])


@pytest.mark.parametrize("T", [1, 40, 300])
def test_scan_in_place_state_and_carry(T):
    """Two calls that update the state in place agree with one call over all tokens."""
    c = scan_case(2, 2 * T, 70, 16, 0, F32)
    st = gpu(c["state"])
    ys = []
    for i in (0, 1):
        part = {k: v[:, i * T:(i + 1) * T].contiguous() if k in ("x", "dt", "B", "C", "z") else v for k, v in c.items()}
        ys.append(run_scan(part, st, state_out=st)[0])
    check_scan(c, c["state"], torch.cat(ys, 1), st, F32)


@pytest.mark.parametrize("T,D,N,dtype", [(1025, 70, 16, F32), (777, 300, 7, BF16), (641, 24, 48, F32), (700, 40, 32, F32), (2000, 9, 3, F32)])
def test_scan_one_long_row(T, D, N, dtype):
    """A row that is cut into segments, with and without a workspace, and as a slot next to short ones."""
    c = scan_case(1, T, D, N, 0, dtype)
    assert wkv.library().wkv_ssm_scan_workspace(1, T, T, D, N, 1) > 0
    st = gpu(c["state"])
    y, last = run_scan(c, st, state_out=st)
    check_scan(c, c["state"], y, last, F32)
    lengths = [0, 3, T, 1]
    first = draw(50, 4, D, N)
    first[2] = c["state"][0]
    flat = {k: torch.cat([draw(51, 3, *c[k].shape[2:], dtype=dtype), c[k][0], draw(52, 1, *c[k].shape[2:], dtype=dtype)])
            for k in ("x", "dt", "B", "C", "z")}
    st = gpu(first)
    yv = wkv.ssm_scan_forward_varlen(gpu(torch.tensor(lengths, dtype=torch.int32)), *(gpu(flat[k]) for k in ("x", "dt")), gpu(c["A"]),
                                     gpu(flat["B"]), gpu(flat["C"]), st, max_len=T + 9, D=gpu(c["D"]), z=gpu(flat["z"]),
                                     dt_bias=gpu(c["dt_bias"]))
    assert torch.equal(st[0].cpu(), first[0])
    check_scan(c, c["state"], yv[None, 3:T + 3], st[2:3], F32)
    short = {**c, **{k: v[None, :3] for k, v in flat.items()}}
    check_scan(short, first[1:2], yv[None, :3], st[1:2], F32)


def test_scan_state_map_and_shared_state():
    c = scan_case(3, 12, 40, 16, 0, F32, n_state=5)
    rows = torch.tensor([4, 0, 4], dtype=torch.int32)
    y, last = run_scan(c, c["state"], state_map=gpu(rows))
    check_scan(c, c["state"][rows.long()], y, last, F32)
    y, last = run_scan(c, c["state"][:1])
    check_scan(c, c["state"][:1].expand(3, -1, -1), y, last, F32)


@pytest.mark.parametrize("dtype,lo", [(BF16, 64), (BF16, 3), (F32, 7)])
@pytest.mark.parametrize("T", [5, 70])
def test_scan_rows_of_wider_arrays(dtype, lo, T):
    """x and z as columns of one array, dt, B and C as columns of another, at any alignment."""
    B, D, N = 2, 64, 16
    c = scan_case(B, T, D, N, 0, dtype)
    xz, dbc = draw(30, B, T, 3 * D, dtype=dtype), draw(31, B, T, D + 2 * N + lo, dtype=dtype, std=0.5)
    cut = dict(x=(xz, lo, D), z=(xz, D + lo, D), dt=(dbc, lo, D), B=(dbc, lo + D, N), C=(dbc, lo + D + N, N))
    host, on = {}, {"xz": gpu(xz), "dbc": gpu(dbc)}
    for k, (src, at, w) in cut.items():
        host[k] = src[..., at:at + w]
        c[k] = on["xz" if src is xz else "dbc"][..., at:at + w]
    y, last = run_scan(c, c["state"])
    c.update(host)
    check_scan(c, c["state"], y, last, F32)


@pytest.mark.parametrize("D,G", [(65, 1), (67, 1), (70, 1), (130, 2), (198, 3)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_channels_of_part_blocks(D, G, dtype):
    """The last block of channels of a group with 1, 3, 6, 1 and 2 of its 64: single, overlapping and whole rows."""
    c = scan_case(1, 40, D, 16, G, dtype)
    y, last = run_scan(c, c["state"])
    check_scan(c, c["state"], y, last, F32)


@pytest.mark.parametrize("S", [65, 300])
def test_scan_varlen_many_slots(S):
    """More slots than a wave has lanes, and more than are ranked by length."""
    r = torch.Generator().manual_seed(S)
    lengths = torch.randint(0, 40, (S,), generator=r).to(torch.int32)
    total, D, N = int(lengths.sum()), 12, 8
    c = scan_case(0, 0, D, N, 0, F32, lead=(total,), n_state=S)
    st, status = gpu(c["state"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    y = wkv.ssm_scan_forward_varlen(gpu(lengths), *(gpu(c[k]) for k in ("x", "dt", "A", "B", "C")), st, max_len=40, D=gpu(c["D"]),
                                    z=gpu(c["z"]), dt_bias=gpu(c["dt_bias"]), dev_status=status)
    assert int(status) == 0
    off = 0
    for s, n in enumerate(lengths.tolist()):
        at = slice(off, off + n)
        want, wl = scan_ref(c, c["state"][s], at)
        mag, ml = scan_ref(c, c["state"][s], at, absolute=True)
        assert_within(y[at], want, allowed(mag, scan_roundings(n)), f"slot {s}")
        assert_within(st[s], wl, allowed(ml, scan_roundings(n)), f"state {s}")
        off += n


def test_scan_padding_by_a_step_of_zero():
    """Tokens with dt = -inf leave the state bitwise as it is, on either side of a row."""
    c = scan_case(1, 40, 32, 16, 0, F32)
    c["dt"][:, :7] = float("-inf")
    c["dt"][:, 33:] = float("-inf")
    _, last = run_scan(c, c["state"])
    inner = {k: v[:, 7:33].contiguous() if k in ("x", "dt", "B", "C", "z") else v for k, v in c.items()}
    _, want = run_scan(inner, c["state"])
    tol = allowed(want.cpu().double().abs() + 1, scan_roundings(40))
    assert_within(last, want.cpu().double(), tol, "padded state")
    c["dt"][:] = float("-inf")
    _, last = run_scan(c, c["state"])
    assert torch.equal(last.cpu(), c["state"])


def test_scan_strong_and_zero_decays():
    """Decays down to exactly 0 and exactly 1, and steps so small that ln(1 + e^v) must keep its relative accuracy."""
    c = scan_case(2, 50, 32, 16, 0, F32, bias=False)
    c["A"][:, 0], c["A"][:, 1], c["A"][:8, 2] = 0.0, -1e30, -300.0
    c["dt"] = c["dt"] * 4 - 8
    y, last = run_scan(c, c["state"])
    check_scan(c, c["state"], y, last, F32)


@pytest.mark.parametrize("T", [3, 35])
@pytest.mark.parametrize("low", [float("-inf"), torch.finfo(F32).min])
def test_scan_decays_to_nothing(T, low):
    """A of minus infinity or the lowest number: a state is its last token's input; tokens past the end, and steps of
    zero, change nothing."""
    c = scan_case(2, T, 20, 16, 0, F32)
    c["A"][:, ::2] = low
    y, last = run_scan(c, c["state"])
    check_scan(c, c["state"], y, last, F32)
    c["dt"][:, -1] = float("-inf")
    short = {k: v[:, :-1].contiguous() if k in ("x", "dt", "B", "C", "z") else v for k, v in c.items()}
    _, last = run_scan(c, c["state"])
    _, before = run_scan(short, c["state"])
    assert torch.equal(last, before)


def test_nothing_leaks_between_slots_and_channels():
    """NaN and infinities in one slot's tokens and state, and in one channel of another, stay there."""
    lengths, D, N = [40, 9, 70, 3], 24, 16
    total = sum(lengths)
    c = scan_case(0, 0, D, N, 0, F32, lead=(total,), n_state=4)
    ln = gpu(torch.tensor(lengths, dtype=torch.int32))
    rest = dict(max_len=70, D=gpu(c["D"]), dt_bias=gpu(c["dt_bias"]))

    def run(c):
        st, cs = gpu(c["state"].clone()), gpu(draw(7, 4, 3, D))
        y = wkv.ssm_scan_forward_varlen(ln, *(gpu(c[k]) for k in ("x", "dt", "A", "B", "C")), st, z=gpu(c["z"]), **rest)
        u = wkv.ssm_conv_forward_varlen(ln, gpu(c["x"]), gpu(draw(8, D, 4)), None, cs, max_len=70, activation="silu")
        return [t.cpu() for t in (y, st, u, cs)]

    clean = run(c)
    bad = {k: v.clone() if v is not None else None for k, v in c.items()}
    bad["x"][40:49], bad["dt"][40:49], bad["B"][40:49], bad["C"][40:49], bad["z"][40:49] = (float(v) for v in ("nan", "inf", "nan", "inf", "-inf"))
    bad["state"][1] = float("inf")
    bad["x"][49:119, 5] = float("nan")  # channel 5 of slot 2
    got = run(bad)
    rows = torch.ones(total, D, dtype=torch.bool)
    rows[40:49] = rows[49:119, 5] = False
    slots = torch.ones(4, D, dtype=torch.bool)
    slots[1] = slots[2, 5] = False
    assert torch.equal(got[0][rows], clean[0][rows]) and torch.equal(got[2][rows], clean[2][rows])
    assert torch.equal(got[1][slots], clean[1][slots])
    assert torch.equal(got[3].transpose(1, 2)[slots], clean[3].transpose(1, 2)[slots])


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("dtype,D,N,G", [(BF16, 72, 16, 0), (F32, 34, 16, 2), (F32, 9, 5, 1), (BF16, 20, 40, 1)])
def test_scan_varlen(lengths, dtype, D, N, G):
    total = sum(lengths)
    rows, n_state = slots_of(lengths, 6)
    c = scan_case(0, 0, D, N, G, dtype, seed=40, lead=(total + 4,), n_state=n_state)
    st, status = gpu(c["state"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    ln = torch.tensor(lengths, dtype=torch.int32)
    args = [gpu(ln)] + [gpu(c[k]) for k in ("x", "dt", "A", "B", "C")]
    kw = dict(max_len=max(lengths), D=gpu(c["D"]), z=gpu(c["z"]), dt_bias=gpu(c["dt_bias"]), state_map=gpu(rows))
    y = torch.full((total + 4, D), 77.0, device="cuda")
    wkv.ssm_scan_forward_varlen(*args, st, y=y, dev_status=status, **kw)
    assert int(status) == 0 and (y[total:] == 77).all()
    off = 0
    touched = torch.zeros(n_state, dtype=torch.bool)
    for s, n in enumerate(lengths):
        first, at = c["state"][rows[s]], slice(off, off + n)
        want, wl = scan_ref(c, first, at)
        mag, ml = scan_ref(c, first, at, absolute=True)
        assert_within(y[at], want, allowed(mag, scan_roundings(n)), f"slot {s}")
        assert_within(st[int(rows[s])], wl, allowed(ml, scan_roundings(n)), f"state of slot {s}")
        touched[rows[s].long()] = n > 0
        off += n
    assert torch.equal(st.cpu()[~touched], c["state"][~touched])
    out = torch.full_like(st, 5.0)
    wkv.ssm_scan_forward_varlen(*args, gpu(c["state"]), state_out=out, **kw)
    keep = torch.ones(n_state, dtype=torch.bool)
    keep[rows.long()] = False
    assert (out.cpu()[keep] == 5).all() and torch.equal(out.cpu()[~keep], st.cpu()[~keep])


def test_varlen_bound_far_above_the_tokens():
    """The host's bound may be anything: work is launched for the tokens there are."""
    lengths, D, N = [5, 30, 0, 1], 40, 16
    c = scan_case(0, 0, D, N, 0, F32, seed=77, lead=(sum(lengths),), n_state=len(lengths))
    ln = gpu(torch.tensor(lengths, dtype=torch.int32))
    args, weight = [gpu(c[k]) for k in ("x", "dt", "A", "B", "C")], gpu(draw(78, D, 4))
    got = []
    for bound in (max(lengths), (1 << 30)):
        st, tail = gpu(c["state"]), gpu(draw(79, len(lengths), 3, D))
        got.append((wkv.ssm_scan_forward_varlen(ln, *args, st, max_len=bound),
                    wkv.ssm_conv_forward_varlen(ln, args[0], weight, None, tail, max_len=bound), st, tail))
    for a, b in zip(*got):
        assert torch.equal(a, b)


# ------------------------------------------------------------------------------------------- data errors, slots

def slot_call(kind, lengths, state_map, n_state, total, max_len):
    D, N, W = 24, 8, 3
    ln, mp = torch.tensor(lengths, dtype=torch.int32), torch.tensor(state_map, dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = scan_case(0, 0, D, N, 0, F32, lead=(total,), n_state=n_state)
    y = torch.full((total, D), 77.0, device="cuda")
    if kind == "conv":
        st = torch.full((n_state, W - 1, D), 3.0, device="cuda")
        wkv.ssm_conv_forward_varlen(gpu(ln), gpu(c["x"]), gpu(draw(1, D, W)), None, st, max_len=max_len, state_map=gpu(mp),
                                    y=y, dev_status=status)
    else:
        st = torch.full((n_state, D, N), 3.0, device="cuda")
        wkv.ssm_scan_forward_varlen(gpu(ln), *(gpu(c[k]) for k in ("x", "dt", "A", "B", "C")), st, max_len=max_len,
                                    state_map=gpu(mp), y=y, dev_status=status)
    return int(status), y.cpu(), st.cpu()


@pytest.mark.parametrize("kind", ["conv", "scan"])
@pytest.mark.parametrize("max_len", [4, 40])
def test_varlen_data_errors(kind, max_len):
    """Each error sets its bit; a rejected slot writes neither outputs nor its state."""
    s, y, st = slot_call(kind, [2, 3, 1], [0, 9, 1], 4, 6, max_len)  # a row outside the table
    assert s == wkv.WKV_DEV_BAD_STATE_MAP and (y[2:5] == 77).all() and (y[5:] != 77).all() and (st[2:] == 3).all()
    s, y, st = slot_call(kind, [2, 3, 1], [2, 0, 2], 4, 6, max_len)  # two slots of one row
    assert s == wkv.WKV_DEV_DUPLICATE_ROW and (y[:2] == 77).all() and (y[2:5] != 77).all() and (st[1:] == 3).all()
    s, y, st = slot_call(kind, [2, -1, 1], [0, 1, 2], 4, 6, max_len)
    assert s == wkv.WKV_DEV_BAD_LENGTH and (y == 77).all() and (st == 3).all()
    s, y, st = slot_call(kind, [2, max_len + 1, 1], [0, 1, 2], 4, 100, max_len)
    assert s == wkv.WKV_DEV_BAD_LENGTH and (y == 77).all() and (st == 3).all()
    s, y, st = slot_call(kind, [2, 3, 1], [0, 1, 2], 4, 5, max_len)  # one token too few
    assert s == wkv.WKV_DEV_TOKEN_OVERFLOW and (y != 77).all() and (st[2:] == 3).all()


def test_dense_state_map_errors():
    c = conv_case(3, 10, 40, 3, F32, n_state=5)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full((3, 10, 40), 77.0, device="cuda")
    rows = gpu(torch.tensor([4, -1, 0], dtype=torch.int32))
    _, last = wkv.ssm_conv_forward(gpu(c["x"]), gpu(c["weight"]), None, gpu(c["state"]), rows, y=y, dev_status=status,
                                   state_out=torch.full((3, 2, 40), 9.0, device="cuda"))
    assert int(status) == wkv.WKV_DEV_BAD_STATE_MAP and (y[1] == 77).all() and (last[1] == 9).all() and (last[2] != 9).all()


# --------------------------------------------------------------------------------------------------- the store

def store_ref(x, fmt):
    """Codes as numbers, and scales, of rows [R, E]: both quotients in fp32, to nearest; a group with an infinity or NaN
    has the scale NaN and codes of 0."""
    R, E = x.shape
    top = 127.0 if fmt == torch.int8 else 448.0
    codes, scales = [], []
    for c in range(0, E, 64):
        part = x[:, c:c + 64]
        scale = torch.where(torch.isfinite(part).all(1), part.abs().amax(1) / top, torch.nan)
        q = torch.where(scale[:, None] > 0, part / scale[:, None], torch.zeros_like(part)).clamp(-top, top)
        codes.append(q.round() if fmt == torch.int8 else q.to(torch.float8_e4m3fn).float())
        scales.append(scale)
    return torch.cat(codes, 1), torch.stack(scales, 1)


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("R,E", [(1, 1), (2, 63), (3, 64), (2, 65), (4, 130), (2, 4096), (1, 1027)])
def test_store_write_and_read(fmt, R, E):
    x = draw(1, R, E) * torch.exp(draw(2, R, E, std=2.0))
    x[0, : E // 2] = 0
    data, scale = wkv.state_store_alloc(R + 2, E, format=fmt)
    perm = torch.randperm(R + 2, generator=torch.Generator().manual_seed(3))[:R].to(torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    wkv.state_store_write(data, scale, gpu(x), gpu(perm), dev_status=status)
    codes, scales = store_ref(x, fmt)
    want = torch.zeros(R + 2, E)
    want[perm.long()] = codes
    wants = torch.zeros(R + 2, scales.shape[1])
    wants[perm.long()] = scales
    assert int(status) == 0 and torch.equal(data.cpu().float(), want) and torch.equal(scale.cpu(), wants)
    out = torch.full((R + 3, E), 7.0, device="cuda")  # the written rows, reversed and one twice, into rows 1 ..
    src = torch.cat((perm.flip(0), perm[:1]))
    dst = torch.arange(1, R + 2, dtype=torch.int32)
    wkv.state_store_read(data, scale, out, gpu(src), gpu(dst), dev_status=status)
    full = want * wants.repeat_interleave(64, 1)[:, :E]
    assert int(status) == 0 and torch.equal(out[1:R + 2].cpu(), full[src.long()])
    assert (out[0] == 7).all() and (out[R + 2] == 7).all()
    # half a step of the code: 1/2 of the scale for int8; 2^-4 of the value for e4m3, 2^-10 of the scale below its
    # smallest normal number; the two quotients and the product add three roundings of the value
    step = 0.5 * wants.repeat_interleave(64, 1)[:, :E][perm.long()].double() if fmt == torch.int8 else torch.maximum(
        x.double().abs() * 2.0 ** -4, wants.repeat_interleave(64, 1)[:, :E][perm.long()].double() * 2.0 ** -10)
    assert ((full[perm.long()].double() - x.double()).abs() <= step + 4 * 2.0 ** -24 * x.double().abs()).all()


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
def test_store_quotients_are_correctly_rounded(fmt):
    """Codes and scales bitwise those of the rounded quotients: a million values, scales of every binary exponent,
    mantissas of all ones, values next to the border between two codes, and the smallest numbers."""
    top = 127.0 if fmt == torch.int8 else 448.0
    exponent = torch.arange(-140, 120, dtype=torch.float64).repeat_interleave(64)  # one group each
    groups = exponent.numel()
    x = (draw(8, groups, 64).double() * 2.0 ** exponent[:, None]).float()
    ones = torch.tensor([0x3fffffff], dtype=torch.int32).view(F32)  # a scale whose mantissa is all ones
    x[::7, 0] = (ones.double() * top * 2.0 ** exponent[::7]).float()
    scale = x.abs().amax(1) / top
    border = (torch.randint(-126, 126, (groups, 16), generator=torch.Generator().manual_seed(9)) + 0.5) * scale[:, None]
    x[:, 16:32] = torch.where(border.abs() <= x[:, :1].abs(), border, x[:, 16:32])
    x[:, 32:36] = torch.nextafter(x[:, 16:20], torch.zeros(groups, 4))
    x = x.reshape(4, -1)
    data, scales = wkv.state_store_alloc(4, x.shape[1], format=fmt)
    wkv.state_store_write(data, scales, gpu(x))
    codes, want = store_ref(x, fmt)
    # (the largest exponents overflow to infinities: groups that are not numbers)
    assert torch.equal(scales.cpu().nan_to_num(-1.0), want.nan_to_num(-1.0)) and torch.equal(data.cpu().float(), codes)


def test_store_of_states_by_rows():
    """WKV states [rows, H, 64, 64] through state_rows and the identity."""
    st = draw(4, 5, 2, 64, 64, std=0.3)
    data, scale = wkv.state_store_alloc(3, 2 * 64 * 64)
    wkv.state_store_write(data, scale, gpu(st), state_rows=gpu(torch.tensor([4, 0, 2], dtype=torch.int32)))
    out = wkv.state_store_read(data, scale, torch.empty(3, 2, 64, 64, device="cuda"))
    step = st[[4, 0, 2]].abs().amax(-1, keepdim=True) / 127
    assert ((out.cpu() - st[[4, 0, 2]]).abs() <= 0.51 * step).all()


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
def test_store_of_values_that_are_not_numbers(fmt):
    x = draw(5, 2, 192)
    x[0, 70], x[1, 3], x[1, 130] = float("nan"), float("inf"), float("-inf")
    data, scale = wkv.state_store_alloc(2, 192, format=fmt)
    wkv.state_store_write(data, scale, gpu(x))
    out = wkv.state_store_read(data, scale, torch.empty(2, 192, device="cuda")).cpu()
    bad = torch.zeros(2, 192, dtype=torch.bool)
    bad[0, 64:128] = bad[1, :64] = bad[1, 128:] = True
    assert torch.isnan(out[bad]).all() and torch.isfinite(out[~bad]).all()


def test_store_data_errors():
    x = gpu(draw(6, 3, 64))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    data, scale = wkv.state_store_alloc(4, 64)
    wkv.state_store_write(data, scale, x, i32(1, 4, -1), dev_status=status)
    assert int(status) == wkv.WKV_DEV_BAD_STATE_MAP and (scale[[0, 2, 3]] == 0).all() and scale[1] > 0
    status.zero_()
    data, scale = wkv.state_store_alloc(4, 64)
    wkv.state_store_write(data, scale, x, i32(2, 0, 2), dev_status=status)
    assert int(status) == wkv.WKV_DEV_DUPLICATE_ROW and (scale[1:] == 0).all() and scale[0] > 0
    status.zero_()
    out = torch.full((3, 64), 7.0, device="cuda")
    wkv.state_store_read(data, scale, out, i32(0, 0, 0), i32(1, 2, 1), dev_status=status)
    assert int(status) == wkv.WKV_DEV_DUPLICATE_ROW and (out[:2] == 7).all() and (out[2] != 7).any()


# --------------------------------------------------------------------------------- together, graphs and streams

def layer(seed, D, N):
    """Parameters of one layer: convolution, projections to the step, B and C, scan."""
    return dict(weight=gpu(draw(seed, D, 4, std=0.5)), bias=gpu(draw(seed + 1, D)), proj=gpu(draw(seed + 2, D, D + 2 * N, std=D ** -0.5)),
                A=gpu(-torch.exp(draw(seed + 3, D, N, std=0.5))), D=gpu(draw(seed + 4, D)), dt_bias=gpu(draw(seed + 5, D) - 3))


def layer_slots(p, lengths, max_len, x, z, conv_state, scan_state, rows):
    """One layer over the tokens of many slots: convolution, projection, scan."""
    D, N = p["A"].shape
    u = wkv.ssm_conv_forward_varlen(lengths, x, p["weight"], p["bias"], conv_state, max_len=max_len, state_map=rows, activation="silu")
    dbc = u @ p["proj"]
    return wkv.ssm_scan_forward_varlen(lengths, u, dbc[:, :D], p["A"], dbc[:, D:D + N], dbc[:, D + N:], scan_state,
                                       max_len=max_len, D=p["D"], z=z, dt_bias=p["dt_bias"], state_map=rows)


def test_prompt_snapshot_fork_and_decode():
    """A prompt runs through a layer, its states are stored in 8 bits, two slots continue from the store token by token:
    the same outputs as a dense run that starts from the states as stored."""
    D, N, T, steps = 48, 16, 50, 5
    p = layer(60, D, N)
    x, z = gpu(draw(70, T + steps, D)), gpu(draw(71, T + steps, D))
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cs, ss = torch.zeros(4, 3, D, device="cuda"), torch.zeros(4, D, N, device="cuda")
    y = layer_slots(p, i32(T), T, x[:T], z[:T], cs, ss, i32(2))
    dense, last = wkv.ssm_conv_forward(x[None, :T], p["weight"], p["bias"], activation="silu")
    dbc = dense @ p["proj"]
    yd, sd = wkv.ssm_scan_forward(dense, dbc[..., :D], p["A"], dbc[..., D:D + N], dbc[..., D + N:], p["D"], z[None, :T], p["dt_bias"])
    assert torch.equal(last[0], cs[2])
    torch.testing.assert_close(y, yd[0], rtol=1e-4, atol=1e-4)
    store = [wkv.state_store_alloc(2, t[0].numel()) for t in (cs, ss)]
    for (d, s), t in zip(store, (cs, ss)):
        wkv.state_store_write(d, s, t, i32(1), i32(2))
        wkv.state_store_read(d, s, t, i32(1, 1), i32(0, 3))
    assert torch.equal(ss[0], ss[3]) and ((ss[0] - ss[2]).abs() <= ss[2].abs().max() / 127).all()
    first, conv_first = ss[:1].clone(), cs[:1].clone()
    got = []
    for t in range(T, T + steps):
        two = layer_slots(p, i32(1, 1), 1, x[[t, t]], z[[t, t]], cs, ss, i32(3, 0))
        assert torch.equal(two[0], two[1])
        got.append(two[:1])
    dense, _ = wkv.ssm_conv_forward(x[None, T:], p["weight"], p["bias"], conv_first, activation="silu")
    dbc = dense @ p["proj"]
    yd, sd = wkv.ssm_scan_forward(dense, dbc[..., :D], p["A"], dbc[..., D:D + N], dbc[..., D + N:], p["D"], z[None, T:], p["dt_bias"], first)
    torch.testing.assert_close(torch.cat(got), yd[0], rtol=1e-4, atol=1e-4)
    torch.testing.assert_close(ss[0], sd[0], rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("T", [1, 300])
def test_captured_and_replayed(T):
    """A layer captured into a graph: every replay equals the eager result on the inputs of that replay."""
    D, N, S = 48, 16, 3
    p = layer(80, D, N)
    ln, rows = torch.full((S,), T, dtype=torch.int32, device="cuda"), torch.tensor([1, 0, 3], dtype=torch.int32, device="cuda")
    x, z = torch.empty(S * T, D, device="cuda"), torch.empty(S * T, D, device="cuda")
    cs, ss = torch.zeros(4, 3, D, device="cuda"), torch.zeros(4, D, N, device="cuda")
    x.normal_(); z.normal_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer_slots(p, ln, T, x, z, cs, ss, rows)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer_slots(p, ln, T, x, z, cs, ss, rows)
    for k in range(3):
        x.copy_(gpu(draw(90 + k, S * T, D))); z.copy_(gpu(draw(95 + k, S * T, D)))
        ec, es = cs.clone(), ss.clone()
        want = layer_slots(p, ln, T, x.clone(), z.clone(), ec, es, rows)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(cs, ec) and torch.equal(ss, es)


def test_two_streams_at_once():
    """Calls on two streams, each with its own tensors, give what they give alone."""
    cs = [scan_case(2, 700, 96, 16, 0, BF16, seed=100 * i) for i in (1, 2)]
    on = [{k: gpu(v) for k, v in c.items()} for c in cs]
    call = lambda c: wkv.ssm_scan_forward(c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], c["z"], c["dt_bias"], c["state"])  # noqa: E731
    alone = [call(c) for c in on]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in on]
    got = []
    for _ in range(3):
        for st, c in zip(streams, on):
            with torch.cuda.stream(st):
                got.append(call(c))
    torch.cuda.synchronize()
    for i, (y, last) in enumerate(got):
        assert torch.equal(y, alone[i % 2][0]) and torch.equal(last, alone[i % 2][1])


# ------------------------------------------------------------------------------------------- past 32 bits

def test_token_offsets_past_32_bits():
    """More than 2^31 elements of a token array: silence up to the last tokens, which must be those of a call of their own."""
    D, tail = 4096, 70
    T = (1 << 31) // D + 33 + tail
    x = torch.zeros(1, T, D, dtype=BF16, device="cuda")
    x[:, -tail:] = gpu(draw(90, 1, tail, D, dtype=BF16))
    weight = gpu(draw(91, D, 4))
    y, last = wkv.ssm_conv_forward(x, weight, activation="silu", out_dtype=BF16)
    want, end = wkv.ssm_conv_forward(x[:, -tail:].contiguous(), weight, activation="silu", out_dtype=BF16)
    assert torch.equal(y[:, -tail:], want) and torch.equal(last, end) and not y[:, :-tail].any()
    bc = gpu(draw(92, 1, T, 4, dtype=BF16))
    A = -gpu(draw(93, D, 4)).abs()
    y, last = wkv.ssm_scan_forward(x, x, A, bc, bc, out_dtype=BF16, y=y)
    near = [t[:, -tail:].contiguous() for t in (x, bc)]
    want, end = wkv.ssm_scan_forward(near[0], near[0], A, near[1], near[1], out_dtype=BF16)
    # a state of zeros stays one over any segment: the same operations on the same values
    assert torch.equal(y[:, -tail:], want) and torch.equal(last, end) and not y[:, :-tail].any()


def test_state_offsets_past_32_bits():
    """State tables of more than 2^31 values: steps, and the store's rows, at their ends."""
    D, N = 2048, 32
    rows = (1 << 31) // (D * N) + 5
    c = scan_case(0, 0, D, N, 0, BF16, seed=94, lead=(2,), n_state=2)
    table = torch.zeros(rows, D, N, device="cuda")
    table[rows - 2:] = gpu(c["state"])
    few = gpu(c["state"])
    ln, at = gpu(torch.tensor([1, 1], dtype=torch.int32)), gpu(torch.tensor([rows - 1, rows - 2], dtype=torch.int32))
    args = [gpu(c[k]) for k in ("x", "dt", "A", "B", "C")]
    got = wkv.ssm_scan_forward_varlen(ln, *args, table, max_len=1, state_map=at)
    want = wkv.ssm_scan_forward_varlen(ln, *args, few, max_len=1, state_map=gpu(torch.tensor([1, 0], dtype=torch.int32)))
    assert torch.equal(got, want) and torch.equal(table[rows - 2:], few) and not table[rows - 4:rows - 2].any()
    data, scale = wkv.state_store_alloc(rows, D * N)
    wkv.state_store_write(data, scale, table, store_rows=at, state_rows=at)
    small, small_scale = wkv.state_store_alloc(2, D * N)
    wkv.state_store_write(small, small_scale, few)
    assert torch.equal(data[rows - 2:], small) and torch.equal(scale[rows - 2:], small_scale) and not data[rows - 4:rows - 2].any()
    back = torch.ones(2, D, N, device="cuda")
    wkv.state_store_read(data, scale, back, store_rows=at, state_rows=gpu(torch.tensor([1, 0], dtype=torch.int32)))
    want = torch.empty_like(back)
    wkv.state_store_read(small, small_scale, want)
    assert torch.equal(back, want)
