"""The state space operators on the CPU: exported symbols, host validation of the C ABI and of the binding.  Nothing
here launches a kernel: every call fails validation, which comes before any HIP call, or has nothing to do."""
import os
import re

import pytest
import torch

import rwkv_linear_attention_wkv_amd as wkv
from rwkv_linear_attention_wkv_amd import _native as nat
from rwkv_linear_attention_wkv_amd import ssm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, MIS, ODD = 0x10000, 0x10002, 0x10001  # never dereferenced
E, U, OK = nat.WKV_ERR_INVALID_ARG, nat.WKV_ERR_UNSUPPORTED, nat.WKV_OK


@pytest.fixture(scope="module")
def lib():
    return nat.load()


def test_exports_every_declared_symbol(lib):
    text = open(os.path.join(ROOT, "include", "wkv_ssm.h")).read()
    names = re.findall(r"WKV_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)
    assert set(names) == set(nat.SSM_SIGNATURES) and len(names) == len(set(names))
    for name in names:
        assert hasattr(lib, name), name


def conv(lib, B=2, T=8, D=64, W=4, x=P, xs=64, dt=1, w=P, b=P, act=1, y=2 * P, od=0, si=None, sm=None, ns=0, so=None, ds=None):
    return lib.wkv_ssm_conv_forward(B, T, D, W, x, xs, dt, w, b, act, y, od, si, sm, ns, so, ds, None)


def conv_slots(lib, S=2, D=64, W=4, ln=P, ml=8, tt=16, x=P, xs=64, dt=1, w=P, b=P, act=1, y=2 * P, od=0, si=P, so=P, sm=None, ns=2, ds=None):
    return lib.wkv_ssm_conv_forward_varlen(S, D, W, ln, ml, tt, x, xs, dt, w, b, act, y, od, si, so, sm, ns, ds, None)


def scan(lib, B=2, T=8, D=64, N=16, G=1, x=P, xs=64, d=P, dst=64, A=P, b=P, bs=16, c=P, cs=16, dt=1, sk=P, z=P, zs=64, db=P, sp=1,
         y=2 * P, od=0, si=None, sm=None, ns=0, so=None, ws=None, wb=0, ds=None):
    return lib.wkv_ssm_scan_forward(B, T, D, N, G, x, xs, d, dst, A, b, bs, c, cs, dt, sk, z, zs, db, sp, y, od, si, sm, ns, so, ws, wb, ds, None)


def scan_slots(lib, S=2, D=64, N=16, G=1, ln=P, ml=8, tt=16, x=P, xs=64, d=P, dst=64, A=P, b=P, bs=16, c=P, cs=16, dt=1, sk=P, z=P,
               zs=64, db=P, sp=1, y=2 * P, od=0, si=P, so=P, sm=None, ns=2, ws=None, wb=0, ds=None):
    return lib.wkv_ssm_scan_forward_varlen(S, D, N, G, ln, ml, tt, x, xs, d, dst, A, b, bs, c, cs, dt, sk, z, zs, db, sp, y, od, si,
                                           so, sm, ns, ws, wb, ds, None)


@pytest.mark.parametrize("fn", [conv, scan])
def test_dense_refusals(lib, fn):
    for kw in (dict(B=0), dict(T=-1), dict(T=(1 << 30) + 1), dict(B=70000), dict(D=0), dict(D=1 << 25), dict(x=None), dict(x=ODD), dict(xs=63),
               dict(y=None), dict(y=0x10008), dict(y=P), dict(si=0x10008, ns=1), dict(si=P, ns=0), dict(si=P, ns=3), dict(sm=P),
               dict(si=P, sm=MIS, ns=3), dict(si=P, so=P, ns=1), dict(si=P, so=P, sm=P, ns=2), dict(so=0x10008), dict(ds=MIS)):
        assert fn(lib, **kw) == E, kw
        assert lib.wkv_last_error()
    assert fn(lib, dt=5) == U and fn(lib, od=5) == U
    assert fn(lib, T=0) == OK  # no tokens and no state to hand on


@pytest.mark.parametrize("fn", [conv_slots, scan_slots])
def test_varlen_refusals(lib, fn):
    for kw in (dict(S=-1), dict(S=70000), dict(ml=-1), dict(ml=(1 << 30) + 1), dict(tt=-1), dict(ln=None), dict(ln=MIS), dict(si=None), dict(so=None),
               dict(si=0x10008), dict(ns=0), dict(ns=1), dict(sm=MIS), dict(x=None), dict(y=None), dict(ds=MIS)):
        assert fn(lib, **kw) == E, kw
    assert fn(lib, S=0) == OK


def test_conv_refusals(lib):
    for W in (0, 1, 5):
        assert conv(lib, W=W) == U
    assert conv(lib, act=2) == U
    assert conv(lib, w=None) == E and conv(lib, w=MIS) == E and conv(lib, b=MIS) == E


def test_scan_refusals(lib):
    assert scan(lib, N=0) == U and scan(lib, N=65, bs=65, cs=65) == U
    for kw in (dict(G=0), dict(G=3), dict(A=None), dict(A=0x10008), dict(d=None), dict(b=None), dict(c=None), dict(dst=10),
               dict(bs=15), dict(cs=15), dict(G=2, bs=16), dict(zs=10), dict(sk=MIS), dict(db=MIS), dict(z=ODD), dict(d=2 * P), dict(z=2 * P)):
        assert scan(lib, **kw) == E, kw


def test_scan_workspace(lib):
    need = lib.wkv_ssm_scan_workspace(1, 4096, 4096, 64, 16, 1)
    assert need > 0 and lib.wkv_ssm_scan_workspace(1, 64, 64, 64, 16, 1) == 0 and lib.wkv_ssm_scan_workspace(64, 4096, 64 * 4096, 4096, 16, 1) == 0
    for bad in ((0, 4096, 4096, 64, 16, 1), (1, 4096, 4096, 64, 0, 1), (1, 4096, 4096, 64, 65, 1), (1, 4096, 4096, 64, 16, 3),
                (1, -1, 4096, 64, 16, 1), (1, 4096, -1, 64, 16, 1)):
        assert lib.wkv_ssm_scan_workspace(*bad) == 0
    assert scan(lib, B=1, T=4096, ws=P, wb=need - 1) == E and b"workspace" in lib.wkv_last_error()
    assert scan(lib, B=1, T=4096, ws=0x10008, wb=need) == E
    # a bound on the lengths above the tokens of the call counts as the tokens
    assert lib.wkv_ssm_scan_workspace(4, 1 << 30, 5000, 256, 16, 1) == lib.wkv_ssm_scan_workspace(4, 5000, 5000, 256, 16, 1) > 0


def store(fn, data=P, scale=P, n=4, fmt=0, st=P, ns=4, row=64, sr=None, tr=None, count=4, ds=None):
    return fn(data, scale, n, fmt, st, ns, row, sr, tr, count, ds, None)


@pytest.mark.parametrize("name", ["wkv_state_store_write", "wkv_state_store_read"])
def test_store_refusals(lib, name):
    fn = getattr(lib, name)
    for kw in (dict(count=-1), dict(n=-1), dict(ns=-1), dict(row=0), dict(count=70000, sr=P, tr=P), dict(data=None), dict(scale=None),
               dict(st=None), dict(data=0x10008), dict(st=0x10008), dict(scale=MIS), dict(n=3), dict(ns=3), dict(sr=MIS), dict(tr=MIS),
               dict(ds=MIS)):
        assert store(fn, **kw) == E, kw
    assert store(fn, fmt=2) == U
    assert store(fn, count=0) == OK


def test_row_steps_of_views():
    """The step between the rows of token arrays, and the views that have none."""
    t = torch.zeros(3, 5, 40)
    step = lambda v, inner: ssm._row_step(v, "x", v.dim() - len(inner))  # noqa: E731
    assert step(t, (40,)) == 40 and step(t[..., 8:24], (16,)) == 40 and step(t[:, :, ::40], (1,)) == 40
    assert step(t[:1, 1:4, :8], (8,)) == 40 and step(t[:, :1, :8], (8,)) == 200 and step(t[0, :, 4:9], (5,)) == 40
    assert step(t[:1, :1, :8], (8,)) == 8 and step(t[..., :12].unflatten(-1, (3, 4)), (3, 4)) == 40
    for bad, inner in ((t[:, :3], (40,)), (t[..., ::2], (20,)), (t.transpose(0, 1), (40,)), (t[:, :1].expand(3, 5, 40), (40,)),
                       (t.unflatten(-1, (5, 8))[..., :4], (5, 4))):
        with pytest.raises(ValueError):
            step(bad, inner)


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError, match="device tensor"):
        wkv.ssm_conv_forward(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="dimensions"):
        wkv.ssm_conv_forward(x[0], torch.zeros(8, 4))
    with pytest.raises(TypeError, match="dtype"):
        wkv.ssm_scan_forward(x.half(), x, torch.zeros(8, 4), x, x)
    with pytest.raises(TypeError, match="store format"):
        wkv.state_store_alloc(1, 64, format=torch.uint8, device="cpu")
    with pytest.raises(TypeError, match="store format"):
        wkv.state_store_write(torch.zeros(2, 64), torch.zeros(2, 1), torch.zeros(2, 64))
    with pytest.raises(ValueError, match="device tensor"):
        wkv.state_store_write(torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2, 1), torch.zeros(2, 64))


def conv_back(lib, B=2, T=8, D=64, W=4, x=P, xs=64, dt=1, w=P, b=P, act=1, dy=2 * P, ys=64, yt=0, si=None, sm=None, ns=0, dso=None,
              dx=3 * P, gt=0, dw=P, db=P, dsi=None, ws=P, wb=None, ds=None):
    wb = lib.wkv_ssm_conv_backward_workspace(B, T, D, W) if wb is None else wb
    return lib.wkv_ssm_conv_backward(B, T, D, W, x, xs, dt, w, b, act, dy, ys, yt, si, sm, ns, dso, dx, gt, dw, db, dsi, ws, wb, ds, None)


def scan_back(lib, B=2, T=8, D=64, N=16, G=1, x=P, xs=64, d=P, dst=64, A=P, b=P, bs=16, c=P, cs=16, dt=1, sk=P, z=P, zs=64, db=P, sp=1,
              dy=P, ys=64, yt=0, si=None, sm=None, ns=0, ch=None, dso=None, dx=2 * P, ddt=3 * P, dB=4 * P, dC=5 * P, dz=6 * P, gt=0,
              dA=P, dsk=P, ddb=P, dsi=None, ws=P, wb=None, ds=None):
    wb = lib.wkv_ssm_scan_backward_workspace(B, T, D, N, G, int(bool(ch))) if wb is None else wb
    return lib.wkv_ssm_scan_backward(B, T, D, N, G, x, xs, d, dst, A, b, bs, c, cs, dt, sk, z, zs, db, sp, dy, ys, yt, si, sm, ns, ch,
                                     dso, dx, ddt, dB, dC, dz, gt, dA, dsk, ddb, dsi, ws, wb, ds, None)


@pytest.mark.parametrize("fn", [conv_back, scan_back])
def test_backward_refusals(lib, fn):
    for kw in (dict(B=0), dict(T=0), dict(D=0), dict(x=None), dict(xs=10), dict(dy=None), dict(ys=10), dict(dy=MIS), dict(dx=None),
               dict(dx=0x10008), dict(dx=P), dict(ws=None), dict(ws=0x10008), dict(wb=16), dict(si=P, ns=3), dict(sm=P),
               dict(dso=0x10008), dict(dsi=0x10008), dict(ds=MIS)):
        assert fn(lib, **kw) == E, kw
        assert lib.wkv_last_error()
    for kw in (dict(dt=5), dict(yt=5), dict(gt=5)):
        assert fn(lib, **kw) == U, kw


def test_scan_backward_refusals(lib):
    for kw in (dict(dz=None), dict(z=None), dict(dA=None), dict(dB=None), dict(dC=0x50008), dict(ddt=None), dict(dz=P), dict(ch=0x10008),
               dict(dsk=MIS), dict(ddb=MIS), dict(G=3)):
        assert scan_back(lib, **kw) == E, kw
    assert scan_back(lib, N=65, bs=65, cs=65, wb=1 << 30) == U
    plain, saved = (lib.wkv_ssm_scan_backward_workspace(2, 100, 64, 16, 1, k) for k in (0, 1))
    assert plain - saved == 2 * 6 * 64 * 16 * 4 and lib.wkv_ssm_scan_backward_workspace(2, 0, 64, 16, 1, 0) == 0
    assert scan_back(lib, T=100, wb=saved) == E and b"workspace" in lib.wkv_last_error()


def test_forward_train_needs_room_for_its_states(lib):
    args = lambda T, ch: (2, T, 64, 16, 1, P, 64, P, 64, P, P, 16, P, 16, 1, P, P, 64, P, 1, 2 * P, 0, None, None, 0, None, ch, None, 0,  # noqa: E731
                          None, None)
    assert lib.wkv_ssm_scan_forward_train(*args(17, None)) == E and b"chunk_states" in lib.wkv_last_error()
    assert lib.wkv_ssm_scan_forward_train(*args(17, 0x10008)) == E
    assert lib.wkv_ssm_scan_forward_train(*args(0, None)) == OK


def test_calls_by_words(lib):
    import struct
    text = open(os.path.join(ROOT, "include", "wkv_ssm.h")).read()
    ops = {int(n): "wkv_" + ("state_" if name.startswith("STORE") else "ssm_") + name.lower()
           for name, n in re.findall(r"#define WKV_OP_(\w+) (\d+)", text)}
    assert [ops[i] for i in range(len(ops))] == list(nat.SSM_OPS)
    for op, name in enumerate(nat.SSM_OPS):
        n = len(nat.SSM_SIGNATURES[name][1])
        zeros = struct.pack(f"{n}q", *[0] * n)
        for count in (n - 1, n + 1, -1):
            assert lib.wkv_ssm_call(op, zeros, count) == E and b"arguments" in lib.wkv_last_error()
        # a call of zeros is refused, by the same words either way
        want = lib[name]
        want.restype, want.argtypes = nat.SSM_SIGNATURES[name]
        assert lib.wkv_ssm_call(op, zeros, n) == want(*[0] * n) != OK, name
        said = lib.wkv_last_error()
        want(*[0] * n)
        assert said == lib.wkv_last_error() and name.encode() in said
        for big in (1 << 31, -(1 << 31) - 1):
            first = next(i for i, t in enumerate(nat.SSM_SIGNATURES[name][1]) if t is nat.SSM_SIGNATURES["wkv_ssm_conv_forward"][1][0])
            words = [0] * n
            words[first] = big
            assert lib.wkv_ssm_call(op, struct.pack(f"{n}q", *words), n) == E and b"range" in lib.wkv_last_error()
    assert lib.wkv_ssm_call(len(nat.SSM_OPS), zeros, 1) == E and lib.wkv_ssm_call(-1, zeros, 1) == E
    assert lib.wkv_ssm_call(0, None, 19) == E
    words = [0, 64, 4, P, 8, 16, P, 64, 1, P, P, 1, 2 * P, 0, P, P, 0, 2, 0, 0]  # no slots: nothing to do
    assert lib.wkv_ssm_call(nat.SSM_OPS.index("wkv_ssm_conv_forward_varlen"), struct.pack("20q", *words), 20) == OK
