"""What the state space operators are measured on: the short causal convolution, the selective scan and the 8-bit
state store, each as a user of the package calls it.

Every case says what it stands for.  With ``own`` false, ``run`` computes the operators from elementary torch
operations in 32 bits; with ``own`` true it makes the package's calls.  Both return whole outputs.

Shapes: token arrays are [B, T, D] (dense) or packed [tokens, D] (slots of different lengths); the convolution's
state is [rows, W - 1, D] (the last inputs, oldest first), the scan's [rows, D, N]; the store holds rows of states in
groups of 64 values with one scale each.
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"
_DT = {BF16: torch.bfloat16, F32: torch.float32}


# ---------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # One decode step of 64 slots through the convolution: the smallest call, where latency counts.
        dict(name="conv step 64 slots", kind="conv_slots", slots=64, longest=1, D=2048, W=4, dtype=BF16, silu=True),
        # A serving call whose slots take no token, one, or a part of their prompt; an odd channel count.
        dict(name="conv slots mixed", kind="conv_slots", slots=48, longest=700, D=1551, W=3, dtype=F32, silu=True),
        # The prompt pass of a batch, a wide layer.
        dict(name="conv prompt", kind="conv", B=8, T=4096, D=4096, W=4, dtype=BF16, silu=True),
        # One training step's convolution (forward and all gradients), ragged length.
        dict(name="conv train", kind="conv_train", B=4, T=2047, D=2048, W=4, dtype=BF16, silu=True),
        # One decode step of 64 slots through the scan.
        dict(name="scan step 64 slots", kind="scan_slots", slots=64, longest=1, D=2048, N=16, G=1, dtype=BF16),
        # A serving call of mixed lengths, two groups of B and C, an odd channel count per group.
        dict(name="scan slots mixed", kind="scan_slots", slots=48, longest=700, D=1550, N=16, G=2, dtype=F32),
        # The prompt pass of a batch.
        dict(name="scan prompt", kind="scan", B=8, T=4096, D=2048, N=16, G=1, dtype=BF16),
        # One long document: few rows, so the length has to be split.
        dict(name="scan long row", kind="scan", B=1, T=32765, D=1536, N=16, G=1, dtype=BF16),
        # One training step's scan (forward and all gradients).
        dict(name="scan train", kind="scan_train", B=8, T=2048, D=2048, N=16, G=1, dtype=BF16),
        # Training in 32 bits with a larger state, two groups, ragged sizes.
        dict(name="scan train ragged", kind="scan_train", B=2, T=777, D=1030, N=32, G=2, dtype=F32),
        # Parking the WKV states of 64 slots (32 heads of 64 x 64) in the store.
        dict(name="store write", kind="store_write", rows=64, row=32 * 64 * 64, store="e4m3"),
        # A snapshot of few prefixes, forked into many slots: written and read back.
        dict(name="store write and fork", kind="store_fork", rows=16, forks=96, row=2048 * 16 + 3 * 2048 + 36, store="int8"),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["conv_slots", "conv", "conv_train", "scan_slots", "scan_slots", "scan", "scan", "scan_train", "scan_train",
                       "store_write", "store_fork"])
    dtype = rng.choice([BF16, BF16, F32])
    if kind.startswith("store"):
        c = dict(kind=kind, rows=_logint(rng, 1, 64), row=_logint(rng, 64, 120000))
        return dict(c, store="e4m3") if kind == "store_write" else dict(c, forks=_logint(rng, 1, 128), store="int8")
    if kind.endswith("slots"):
        c = dict(kind=kind, slots=_logint(rng, 1, 96), longest=rng.choice([1, 1, _logint(rng, 1, 8), _logint(rng, 9, 1000)]))
        top = 2500
    else:
        c = dict(kind=kind, B=_logint(rng, 1, 8), T=_logint(rng, 1, 4096))
        top = 4096 if kind.startswith("conv") else 2048
        if kind.endswith("train") or dtype == F32:
            c["T"] = min(c["T"], 2048)
    if kind.startswith("conv"):
        c.update(D=_logint(rng, 48, top), W=rng.choice([2, 3, 4, 4]), dtype=dtype, silu=rng.random() < 0.8)
    else:
        N, G = rng.choice([(16, 1), (16, 1), (8, 1), (16, 2), (11, 3), (32, 1)])
        D = _logint(rng, 48, top * 16 // max(N, 16) // (2 if kind.endswith("train") and N > 16 else 1))
        c.update(D=max(1, D // G) * G, N=N, G=G, dtype=dtype)
    return c


def _lengths(case):
    """Tokens of each slot: none, one, or up to `longest`; the first takes `longest`."""
    S, longest = case["slots"], case["longest"]
    if longest == 1:
        return [1] * S
    r = random.Random(S * 100003 + longest)
    return [longest] + [r.choice([0, 1, 1, r.randint(1, longest), r.randint(1, max(1, longest // 8))]) for _ in range(S - 1)]


def work(case):
    k = case["kind"]
    if k.startswith("store"):
        E, groups = case["row"], -(-case["row"] // 64)
        if k == "store_write":
            return {"bytes": case["rows"] * (5 * E + 4 * groups), "flops": case["rows"] * 4 * E}
        return {"bytes": case["rows"] * (6 * E + 8 * groups) + case["forks"] * 4 * E, "flops": case["rows"] * 4 * E + case["forks"] * E}
    e = 2 if case["dtype"] == BF16 else 4
    slots = k.endswith("slots")
    rows = case["slots"] if slots else case["B"]
    tokens = sum(_lengths(case)) if slots else case["B"] * case["T"]
    D = case["D"]
    if k.startswith("conv"):
        W = case["W"]
        state = rows * 2 * (W - 1) * D * 4
        fwd, ops = tokens * D * 2 * e, tokens * D * (2 * W + 5)
        if k == "conv_train":
            return {"bytes": 2 * fwd + tokens * D * e + state + 2 * D * (W + 1) * 4, "flops": 3 * ops}
        return {"bytes": fwd + state + D * (W + 1) * 4, "flops": ops}
    N, G = case["N"], case["G"]
    state, par = rows * 2 * D * N * 4, D * (N + 2) * 4
    fwd, ops = tokens * (4 * D + 2 * G * N) * e, tokens * D * (7 * N + 20)
    if k == "scan_train":
        return {"bytes": fwd + tokens * (7 * D + 4 * G * N) * e + 2 * state + 3 * par, "flops": ops + tokens * D * (22 * N + 50)}
    return {"bytes": fwd + state + par, "flops": ops}


# --------------------------------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def prepare(case, seed):
    g = _generator(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, device="cuda", generator=g) * (hi - lo) + lo

    def order(n, k):
        return torch.randperm(n, device="cuda", generator=g)[:k].to(torch.int32)

    k = case["kind"]
    s = {"kind": k, "case": case}
    if k.startswith("store"):
        rows, E, groups = case["rows"], case["row"], -(-case["row"] // 64)
        # states of rows of very different magnitude, as carried states have; some are still empty
        mag = torch.exp(uniform(rows, groups, 1, lo=-6.0, hi=2.0))
        x = (normal(rows, groups, 64) * mag).reshape(rows, groups * 64)[:, :E].contiguous()
        x[:, : min(E, 64)] = 0
        dt = torch.int8 if case["store"] == "int8" else torch.float8_e4m3fn
        s.update(states=x, data=torch.zeros(rows + 3, E, dtype=torch.int8, device="cuda").view(dt),
                 scale=torch.zeros(rows + 3, groups, device="cuda"), to=order(rows + 3, rows))
        if k == "store_fork":
            pick = torch.randint(0, rows, (case["forks"],), device="cuda", generator=g)
            s.update(fork=s["to"][pick].contiguous(), out=torch.empty(case["forks"], E, device="cuda"))
        return s
    dt, D = _DT[case["dtype"]], case["D"]
    slots = k.endswith("slots")
    if slots:
        lengths = torch.tensor(_lengths(case), device="cuda", dtype=torch.int32)
        lengths = lengths[order(len(lengths), len(lengths)).long()].contiguous()
        S, total = case["slots"], sum(_lengths(case))
        s.update(lengths=lengths, max_len=case["longest"], rows=order(S + 5, S))
        tok, n_state = (total,), S + 5
    else:
        tok, n_state = (case["B"], case["T"]), case["B"]
    out = dict(device="cuda", dtype=dt)
    if k.startswith("conv"):
        W = case["W"]
        s.update(x=normal(*tok, D, dtype=dt), weight=uniform(D, W, lo=-1 / math.sqrt(W), hi=1 / math.sqrt(W)),
                 bias=uniform(D, lo=-1 / math.sqrt(W), hi=1 / math.sqrt(W)), state=normal(n_state, W - 1, D),
                 act="silu" if case["silu"] else None)
    else:
        N, G = case["N"], case["G"]
        step = torch.exp(uniform(D, lo=math.log(1e-3), hi=math.log(1e-1)))
        n = torch.arange(1, N + 1, device="cuda", dtype=torch.float32)
        bc = (G, N) if G > 1 else (N,)
        s.update(x=torch.nn.functional.silu(normal(*tok, D)).to(dt), z=normal(*tok, D, dtype=dt),
                 dt=normal(*tok, D, std=0.5, dtype=dt), dt_bias=step + torch.log(-torch.expm1(-step)),
                 A=-n * torch.exp(normal(D, N, std=0.2)), B=normal(*tok, *bc, dtype=dt), C=normal(*tok, *bc, dtype=dt),
                 D=1 + normal(D, std=0.1), state=normal(n_state, D, N, std=0.1))
    if k.endswith("train"):
        s.update(dy=normal(*tok, D, dtype=dt), d_state=normal(*s["state"].shape, std=0.1))
    return s


# -------------------------------------------------------------------------------------------- the package's calls

def _own(s):
    import rwkv_linear_attention_wkv_amd as wkv
    k = s["kind"]
    if k == "conv_slots":
        y = wkv.ssm_conv_forward_varlen(s["lengths"], s["x"], s["weight"], s["bias"], s["state"], max_len=s["max_len"],
                                        state_map=s["rows"], activation=s["act"], out_dtype=s["x"].dtype)
        return y, s["state"]
    if k == "conv":
        return wkv.ssm_conv_forward(s["x"], s["weight"], s["bias"], s["state"], activation=s["act"], out_dtype=s["x"].dtype)
    if k == "conv_train":
        y, last = wkv.ssm_conv_forward(s["x"], s["weight"], s["bias"], s["state"], activation=s["act"], out_dtype=s["x"].dtype)
        return (y, last, *wkv.ssm_conv_backward(s["x"], s["weight"], s["bias"], s["dy"], s["state"], activation=s["act"],
                                                d_state=s["d_state"], grad_dtype=s["x"].dtype))
    if k == "store_write":
        wkv.state_store_write(s["data"], s["scale"], s["states"], store_rows=s["to"])
        return s["data"], s["scale"]
    if k == "store_fork":
        wkv.state_store_write(s["data"], s["scale"], s["states"], store_rows=s["to"])
        return wkv.state_store_read(s["data"], s["scale"], s["out"], store_rows=s["fork"]), s["scale"]
    args = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    rest = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    if k == "scan_slots":
        y = wkv.ssm_scan_forward_varlen(s["lengths"], *args, s["state"], max_len=s["max_len"], state_map=s["rows"],
                                        out_dtype=s["x"].dtype, **rest)
        return y, s["state"]
    if k == "scan":
        return wkv.ssm_scan_forward(*args, state=s["state"], out_dtype=s["x"].dtype, **rest)
    y, last, chunks = wkv.ssm_scan_forward_train(*args, state=s["state"], out_dtype=s["x"].dtype, **rest)
    return (y, last, *wkv.ssm_scan_backward(*args, s["dy"], state=s["state"], d_state=s["d_state"], chunk_states=chunks,
                                            grad_dtype=s["x"].dtype, **rest))


# ------------------------------------------------------------------------------------------------- plain forms

def _spans(s):
    """(first token of each sequence, its length, its state row, each token's sequence, each token's place in it)."""
    if "lengths" in s:
        n = s["lengths"].long()
        rows = s["rows"].long()
        total = s["x"].shape[0]
    else:
        B, T = s["x"].shape[:2]
        n = torch.full((B,), T, device="cuda")
        rows = torch.arange(B, device="cuda")
        total = B * T
    first = torch.cumsum(n, 0) - n
    seq = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n, output_size=total)
    return first, n, rows, seq, torch.arange(total, device="cuda") - first[seq]


def _silu(v):
    return v / (1 + torch.exp(-v))


def _conv_windows(s, x, spans):
    """[tokens, W, D]: each token's inputs, oldest first; those before the sequence come from its state."""
    first, n, rows, seq, at = spans
    W = s["weight"].shape[1]
    back = at[:, None] + torch.arange(1 - W, 1, device="cuda")  # place in the sequence, negative: in the state
    token = (first[seq][:, None] + back).clamp(min=0)
    old = s["state"][rows[seq][:, None], (back + W - 1).clamp(max=W - 2)]
    return torch.where((back >= 0)[..., None], x[token], old)


def _conv_last(s, x, spans):
    """The state after each sequence: its last W - 1 inputs, those of the state among them."""
    first, n, rows, _, _ = spans
    W = s["weight"].shape[1]
    back = n[:, None] + torch.arange(1 - W, 0, device="cuda")
    token = (first[:, None] + back).clamp(min=0, max=max(x.shape[0] - 1, 0))
    return torch.where((back >= 0)[..., None], x[token], s["state"][rows[:, None], (back + W - 1).clamp(max=W - 2)])


def _plain_conv(s):
    D = s["x"].shape[-1]
    x = s["x"].reshape(-1, D).float()
    spans = _spans(s)
    first, n, rows, seq, at = spans
    win = _conv_windows(s, x, spans)
    pre = (win * s["weight"].t()).sum(1) + s["bias"]
    y = (_silu(pre) if s["act"] else pre).to(s["x"].dtype).reshape(s["x"].shape)
    last = _conv_last(s, x, spans)
    if s["kind"] == "conv_slots":
        s["state"][rows] = last
        return y, s["state"]
    if s["kind"] == "conv":
        return y, last
    sig = 1 / (1 + torch.exp(-pre))
    dpre = s["dy"].reshape(-1, D).float() * (sig * (1 + pre * (1 - sig)) if s["act"] else torch.ones_like(pre))
    B, T = s["x"].shape[:2]
    W = s["weight"].shape[1]
    # every input, the state's among them, is seen by the W outputs that follow it
    dp = torch.nn.functional.pad(dpre.reshape(B, T, D), (0, 0, W - 1, W - 1))
    dx = (dp.unfold(1, W, 1) * s["weight"].flip(1)).sum(-1)
    dx[:, T:] += s["d_state"]  # the last W - 1 inputs are the final state
    return (y, last, dx[:, W - 1:].to(y.dtype), (dpre[:, None] * win).sum(0).t(), dpre.sum(0), dx[:, : W - 1])


def _running(a, b, longest):
    """h_t = a_t h_(t-1) + b_t over dimension 0, by doubling; a is 0 where a sequence starts."""
    step = 1
    while step < longest:
        b = torch.cat((b[:step], b[step:] + a[step:] * b[:-step]))
        a = torch.cat((a[:step], a[step:] * a[:-step]))
        step *= 2
    return b


def _plain_scan(s):
    shape, D, N = s["x"].shape, s["x"].shape[-1], s["A"].shape[1]
    flat = lambda t: t.reshape(-1, D).float()  # noqa: E731
    x, z = flat(s["x"]), flat(s["z"])
    raw = flat(s["dt"]) + s["dt_bias"]
    delta = raw.clamp(min=0) + torch.log1p(torch.exp(-raw.abs()))
    G = s["B"].shape[-2] if s["B"].dim() == s["x"].dim() + 1 else 1
    Bm, Cm = (s[v].reshape(-1, G, 1, N).float() for v in "BC")
    groups = lambda t: t.reshape(-1, G, D // G, N)  # noqa: E731
    first, n, rows, seq, at = _spans(s)
    some = n > 0
    start, end = first[some], (first + n)[some] - 1
    longest = s["max_len"] if "lengths" in s else shape[1]
    a = torch.exp(delta[:, :, None] * s["A"])
    b = (groups((delta * x)[:, :, None].expand(-1, -1, N)) * Bm).reshape(a.shape)
    h0 = s["state"][rows]
    b[start] += a[start] * h0[some]
    reset = a.clone()
    reset[start] = 0
    h = _running(reset, b, longest)
    last = h0.clone()
    last[some] = h[end]
    core = (groups(h) * Cm).sum(-1).reshape(-1, D) + s["D"] * x
    sig = 1 / (1 + torch.exp(-z))
    y = (core * z * sig).to(s["x"].dtype).reshape(shape)
    if s["kind"] == "scan_slots":
        s["state"][rows] = last
        return y, s["state"]
    if s["kind"] == "scan":
        return y, last
    del reset, b
    dy = flat(s["dy"])
    dz = dy * core * sig * (1 + z * (1 - sig))
    dcore = dy * z * sig
    dC = (groups(h) * dcore.reshape(-1, G, D // G, 1)).sum(2)
    before = torch.empty_like(h)  # the state that each token found
    before[1:] = h[:-1]
    before[start] = h0[some]
    del h
    g = (groups(dcore[:, :, None].expand(-1, -1, N)) * Cm).reshape(a.shape)
    g[end] += s["d_state"][some]
    onward = torch.zeros_like(a)
    onward[:-1] = a[1:]
    onward[end] = 0
    g = _running(onward.flip(0), g.flip(0), longest).flip(0)
    del onward
    dB = (groups(g) * (delta * x).reshape(-1, G, D // G, 1)).sum(2)
    gb = (groups(g) * Bm).sum(-1).reshape(-1, D)
    d_first = s["d_state"].clone()
    d_first[some] = a[start] * g[start]
    g = g * a * before
    dA = (g * delta[:, :, None]).sum(0)
    ddelta = (g * s["A"]).sum(-1) + x * gb
    ddt = ddelta / (1 + torch.exp(-raw))
    to = lambda t: t.to(s["x"].dtype).reshape(shape)  # noqa: E731
    return (y, last, to(delta * gb + s["D"] * dcore), to(ddt), dA, dB.to(s["x"].dtype).reshape(s["B"].shape),
            dC.to(s["x"].dtype).reshape(s["C"].shape), (dcore * x).sum(0), to(dz), ddt.sum(0), d_first)


def _plain_store(s):
    x = s["states"]
    rows, E = x.shape
    groups = -(-E // 64)
    top = 127.0 if s["data"].dtype == torch.int8 else 448.0
    v = torch.nn.functional.pad(x, (0, groups * 64 - E)).reshape(rows, groups, 64)
    scale = v.abs().amax(-1) / torch.tensor(top, device="cuda")
    q = (v / scale[..., None]).nan_to_num(0.0).clamp(-top, top).reshape(rows, groups * 64)[:, :E]
    code = q.round().to(torch.int8) if s["data"].dtype == torch.int8 else q.to(s["data"].dtype)
    to = s["to"].long()
    s["data"].view(torch.int8)[to] = code.view(torch.int8)
    s["scale"][to] = scale
    if s["kind"] == "store_write":
        return s["data"], s["scale"]
    fork = s["fork"].long()
    each = s["scale"][fork].repeat_interleave(64, dim=1)[:, :E]
    s["out"].copy_(s["data"][fork].float() * each)
    return s["out"], s["scale"]


def run(state):
    if own:
        return _own(state)
    k = state["kind"]
    return _plain_store(state) if k.startswith("store") else _plain_conv(state) if k.startswith("conv") else _plain_scan(state)


# ------------------------------------------------------------------------------------------- 64-bit definitions

def _sequences(s):
    """(first token, length, state row) of each sequence, as numbers."""
    if "lengths" in s:
        n, rows, first, got = s["lengths"].tolist(), s["rows"].tolist(), 0, []
        for length, row in zip(n, rows):
            got.append((first, length, row))
            first += length
        return got
    B, T = s["x"].shape[:2]
    return [(b * T, T, b) for b in range(B)]


def _exact_conv(s):
    D, W = s["weight"].shape
    x, w, bias = s["x"].reshape(-1, D).double(), s["weight"].double(), s["bias"].double()
    y, rows = torch.empty_like(x), s["state"].double().clone()
    train = s["kind"] == "conv_train"
    if train:
        dy, dx = s["dy"].reshape(-1, D).double(), torch.empty_like(x)
        dw, dbias, dfirst = torch.zeros_like(w), torch.zeros_like(bias), torch.empty_like(rows)
    for first, n, row in _sequences(s):
        line = torch.cat((rows[row], x[first:first + n]))  # the inputs, the state's first
        pre = bias + sum(w[:, j] * line[j:j + n] for j in range(W))
        sig = torch.sigmoid(pre)
        y[first:first + n] = pre * sig if s["act"] else pre
        if train:
            d = dy[first:first + n] * (sig + pre * sig * (1 - sig) if s["act"] else 1)
            back = torch.zeros_like(line)
            for j in range(W):
                back[j:j + n] += w[:, j] * d
                dw[:, j] += (d * line[j:j + n]).sum(0)
            back[n:] += s["d_state"][row].double()
            dbias += d.sum(0)
            dx[first:first + n], dfirst[row] = back[W - 1:], back[:W - 1]
        rows[row] = line[n:]
    y = y.reshape(s["x"].shape)
    return (y, rows, dx.reshape(s["x"].shape), dw, dbias, dfirst) if train else (y, rows)


def _exact_scan(s):
    shape, D, N = s["x"].shape, s["x"].shape[-1], s["A"].shape[1]
    G = s["B"].shape[-2] if s["B"].dim() == s["x"].dim() + 1 else 1
    seqs = _sequences(s)
    longest = max(n for _, n, _ in seqs)
    first = torch.tensor([f for f, _, _ in seqs], device="cuda")
    length = torch.tensor([n for _, n, _ in seqs], device="cuda")
    row = torch.tensor([r for _, _, r in seqs], device="cuda")
    flat = lambda v: s[v].reshape(-1, D).double()  # noqa: E731
    x, z, A = flat("x"), flat("z"), s["A"].double()
    raw = flat("dt") + s["dt_bias"].double()
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    wide = lambda v: v.reshape(-1, G, N).double()  # noqa: E731
    Bm, Cm = wide(s["B"]), wide(s["C"])
    spread = lambda v: v.repeat_interleave(D // G, dim=1)  # noqa: E731
    h = s["state"].double()[row]
    core = torch.empty_like(x)
    train = s["kind"] == "scan_train"
    kept = []
    for t in range(longest):
        live = (length > t).nonzero()[:, 0] if "lengths" in s else slice(None)
        at = first[live] + t
        if train:
            kept.append(h)
        new = torch.exp(delta[at][:, :, None] * A) * h[live] + (delta[at] * x[at])[:, :, None] * spread(Bm[at])
        if train or not isinstance(live, slice):
            h = h.clone()
        h[live] = new
        core[at] = (new * spread(Cm[at])).sum(-1)
    core = core + s["D"].double() * x
    y = (core * torch.nn.functional.silu(z)).reshape(shape)
    if "lengths" in s:
        rows = s["state"].double().clone()
        rows[row] = h
        return y, rows
    if not train:
        return y, h
    dy, sig = flat("dy"), torch.sigmoid(z)
    dcore = dy * z * sig
    dz = dy * core * (sig + z * sig * (1 - sig))
    g, after = s["d_state"].double()[row], h
    dx, ddelta, dA = torch.empty_like(x), torch.empty_like(x), torch.zeros_like(A)
    dB, dC = torch.empty_like(Bm), torch.empty_like(Cm)
    for t in reversed(range(longest)):
        at = first + t
        g = g + dcore[at][:, :, None] * spread(Cm[at])
        dC[at] = (dcore[at][:, :, None] * after).reshape(-1, G, D // G, N).sum(2)
        dB[at] = (g * (delta[at] * x[at])[:, :, None]).reshape(-1, G, D // G, N).sum(2)
        gb = (g * spread(Bm[at])).sum(-1)
        g = g * torch.exp(delta[at][:, :, None] * A)
        gh = g * kept[t]
        dx[at], ddelta[at] = delta[at] * gb, x[at] * gb + (gh * A).sum(-1)
        dA += (gh * delta[at][:, :, None]).sum(0)
        after = kept[t]
    dx = dx + s["D"].double() * dcore
    ddt = ddelta * torch.sigmoid(raw)
    return (y, h, dx.reshape(shape), ddt.reshape(shape), dA, dB.reshape(s["B"].shape), dC.reshape(s["C"].shape),
            (dcore * x).sum(0), dz.reshape(shape), ddt.sum(0), g)


def _exact_store(s):
    """A group's scale is the 32-bit quotient of its largest magnitude, a code the nearest to the 32-bit quotient by it."""
    x = s["states"].double()
    rows, E = x.shape
    each, scales = [], []
    top = 127.0 if s["data"].dtype == torch.int8 else 448.0
    for c in range(0, E, 64):
        part = x[:, c:c + 64]
        scale = (part.abs().max(dim=1).values / top).float().double()
        q = torch.where(scale[:, None] > 0, part / scale[:, None].clamp(min=1e-300), torch.zeros_like(part)).float()
        each.append(q.clamp(-top, top))
        scales.append(scale)
    q, scale = torch.cat(each, dim=1), torch.stack(scales, dim=1)
    whole = s["scale"].double()
    whole[s["to"].long()] = scale
    if s["kind"] == "store_write":
        code = torch.zeros(s["data"].shape, device="cuda")
        code[s["to"].long()] = q.to(torch.float8_e4m3fn).float()
        return code.double(), whole
    at = torch.full((s["data"].shape[0],), -1, device="cuda", dtype=torch.long)
    at[s["to"].long()] = torch.arange(rows, device="cuda")
    pick = at[s["fork"].long()]
    return torch.round(q.double())[pick] * scale.repeat_interleave(64, dim=1)[:, :E][pick], whole


def exact(case, seed):
    s = prepare(case, seed)
    k = case["kind"]
    return _exact_store(s) if k.startswith("store") else _exact_conv(s) if k.startswith("conv") else _exact_scan(s)
