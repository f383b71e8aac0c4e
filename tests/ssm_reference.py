"""The state space operators in 64 bits on the CPU, from their definitions, one sequence and one token at a time.

Each function also returns the magnitude of every result: the same formula with every term taken by its absolute
value.  A kernel that rounds every operation to fp32 is off by at most (number of roundings that a term passes) times
2^-24 of that magnitude, which is what the tests allow (see ``allowed``).
"""
import torch

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def allowed(magnitude, roundings, value=None, dtype=torch.float32):
    """Largest error of an fp32 computation whose terms pass ``roundings`` roundings, stored as ``dtype``."""
    tol = magnitude * (roundings * 2.0 ** -24)
    if value is not None and dtype == torch.bfloat16:
        tol = tol + value.abs() * 2.0 ** -8 * (1 + 2.0 ** -7)
    return tol + 1e-37


def assert_within(got, want, tol, what):
    got = got.detach().double().cpu()
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)} != {tuple(want.shape)}"
    if not got.numel():
        return
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    off = (got - want).abs() / tol
    worst = float(off.max())
    assert worst <= 1, f"{what}: {worst:.3g} times the allowed error at {int(off.argmax())} of {off.numel()}"


def d64(t):
    return None if t is None else t.detach().cpu().double()


def conv(x, weight, bias, first, act):
    """One sequence: x [T, D], first [W-1, D] -> (y, magnitude of the pre-activation, last inputs)."""
    T, W = x.shape[0], weight.shape[1]
    line = torch.cat((first, x))
    pre, mag = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(T):
        for j in range(W):
            pre[t] += weight[:, j] * line[t + j]
            mag[t] += (weight[:, j] * line[t + j]).abs()
    if bias is not None:
        pre, mag = pre + bias, mag + bias.abs()
    return pre * torch.sigmoid(pre) if act else pre, mag, line[T:]


def conv_grads(x, weight, bias, first, act, dy, d_last):
    """One sequence's gradients by automatic differentiation of the definition, and their magnitudes."""
    leaves = [v.clone().requires_grad_() for v in (x, weight, first)] + [None if bias is None else bias.clone().requires_grad_()]
    y, _, last = conv(leaves[0], leaves[1], leaves[3], leaves[2], act)
    loss = (y * dy).sum() + ((last * d_last).sum() if d_last is not None else 0)
    wanted = [v for v in leaves if v is not None]
    grads = list(torch.autograd.grad(loss, wanted, allow_unused=True))
    grads = [torch.zeros_like(v) if g is None else g for v, g in zip(wanted, grads)]
    dx, dw, d_first = grads[:3]
    return dx, dw, grads[3] if bias is not None else None, d_first


def softplus(v):
    return torch.logaddexp(v, torch.zeros_like(v))


def scan(x, dt, A, B, C, skip, z, bias, first, softplus_on=True, absolute=False):
    """One sequence: x, dt, z [T, D]; B, C [T, G, N]; first [D, N] -> (y, last state, states before each token)."""
    T, D = x.shape
    G = B.shape[1]
    raw = dt if bias is None else dt + bias
    delta = softplus(raw) if softplus_on else raw
    per = D // G
    Bd, Cd = (v.repeat_interleave(per, dim=1) for v in (B, C))
    gate = None if z is None else z * torch.sigmoid(z)
    sk = torch.zeros(D, dtype=x.dtype) if skip is None else skip
    if absolute:
        x, Bd, Cd, sk, first = x.abs(), Bd.abs(), Cd.abs(), sk.abs(), first.abs()
        gate = None if gate is None else gate.abs()
    h, y = first, []
    for t in range(T):
        step = delta[t].abs() if absolute else delta[t]
        h = torch.exp(delta[t][:, None] * A) * h + (step * x[t])[:, None] * Bd[t]
        o = (h * Cd[t]).sum(-1) + sk * x[t]
        y.append(o if gate is None else o * gate[t])
    return torch.stack(y) if y else x.new_zeros(0, D), h


def scan_grads(x, dt, A, B, C, skip, z, bias, first, dy, d_last, softplus_on=True):
    """Gradients of one sequence by automatic differentiation of the definition, and their magnitudes.

    Returns two dicts with x, dt, A, B, C, skip, z, bias, first.  A magnitude is the gradient with every term taken by
    its absolute value (A is not positive, so that no two terms of a decay's derivative differ in sign).
    """
    def run(absolute):
        pos = (lambda v: None if v is None else v.abs()) if absolute else (lambda v: v)
        raw = dt if bias is None else dt + bias
        delta = softplus(raw) if softplus_on else raw
        leaf = lambda v: None if v is None else v.clone().requires_grad_()  # noqa: E731
        X, Bl, Cl, S, F = (leaf(pos(v)) for v in (x, B, C, skip, first))
        Al = leaf(-A.abs() if absolute else A)
        decay, step = leaf(delta), leaf(pos(delta))
        gate = leaf(pos(z * torch.sigmoid(z))) if z is not None else None
        T, D = x.shape
        per = D // B.shape[1]
        h, total = F, 0.0
        w = pos(dy)
        for t in range(T):
            h = torch.exp(decay[t][:, None] * Al) * h + (step[t] * X[t])[:, None] * Bl[t].repeat_interleave(per, dim=0)
            o = (h * Cl[t].repeat_interleave(per, dim=0)).sum(-1) + (S * X[t] if S is not None else 0)
            total = total + (w[t] * (o * gate[t] if gate is not None else o)).sum()
        if d_last is not None:
            total = total + (h * pos(d_last)).sum()
        leaves = dict(x=X, decay=decay, step=step, A=Al, B=Bl, C=Cl, skip=S, gate=gate, first=F)
        names = [k for k, v in leaves.items() if v is not None]
        got = dict(zip(names, torch.autograd.grad(total, [leaves[k] for k in names], allow_unused=True)))
        got = {k: torch.zeros_like(leaves[k]) if v is None else v for k, v in got.items()}
        slope = torch.sigmoid(raw) if softplus_on else torch.ones_like(raw)
        d = got.pop("decay"), got.pop("step")
        got["dt"] = (pos(d[0]) + d[1]) * slope
        got["bias"] = got["dt"].sum(0) if bias is not None else None
        if z is not None:
            sg = torch.sigmoid(z)
            # the gate's slope is a sum, sg + sg z (1 - sg): near z = -1.278 its terms cancel, and a rounding of either
            # (2^-24 of sg) is many roundings of what is left, so the magnitude adds |z|
            got["z"] = got.pop("gate") * (sg * (1 + pos(z) * (1 - sg)))
        return got

    return run(False), run(True)
