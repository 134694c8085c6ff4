"""Measured cases of the layer operators around the recurrence: the selective state space scan, its short causal
convolution, and layer norm, each as prompts, single tokens or gradients.

``own`` chooses between the framework's kernels and the plain form in elementary torch operations."""
import math

import torch

own = False

BF16, F32 = "bf16", "fp32"
DTYPES = {BF16: torch.bfloat16, F32: torch.float32}
RANK = 64  # width of the low-rank step projection that lies in front of B and C in one buffer


def listed():
    return [
        # one long prompt through a wide layer: u and z are halves of one projection's output, B and C slices of another's
        dict(name="scan_prompt_long", op="scan_fwd", dtype=BF16, batch=1, tokens=16384, dim=4096, ds=16, seqs=0,
             gate=True, sliced=True),
        # a packed prefill of ragged prompts in fp32, an empty and a one-token one among them, odd width and state size
        dict(name="scan_prompts_ragged", op="scan_fwd", dtype=F32, batch=1, tokens=3001, dim=777, ds=12, seqs=9,
             gate=False, sliced=False),
        # decode of a single stream, where latency counts
        dict(name="scan_step_one", op="scan_step", dtype=BF16, batch=1, dim=2048, ds=16, gate=True),
        # decode of a full serving batch: the states stream through once
        dict(name="scan_step_batch", op="scan_step", dtype=BF16, batch=256, dim=4096, ds=16, gate=True),
        # the gradients of a training micro-batch
        dict(name="scan_train", op="scan_bwd", dtype=BF16, batch=8, tokens=2048, dim=2048, ds=16, seqs=0, gate=True,
             sliced=True),
        # the gradients of packed documents in fp32 at an odd width
        dict(name="scan_train_ragged", op="scan_bwd", dtype=F32, batch=1, tokens=2500, dim=515, ds=16, seqs=6,
             gate=False, sliced=False),
        # the convolution in front of a packed prefill
        dict(name="conv_prompts", op="conv_fwd", dtype=BF16, batch=1, tokens=32768, dim=4096, width=4, seqs=16,
             silu=True, sliced=True),
        # decode: q, k and v of 16 heads of 128 in one call
        dict(name="conv_step", op="conv_step", dtype=BF16, batch=64, dim=6144, width=4, silu=True),
        # its gradients for a training micro-batch
        dict(name="conv_train", op="conv_bwd", dtype=BF16, batch=4, tokens=4096, dim=4096, width=4, seqs=0, silu=True,
             sliced=False),
        # the pre-norm of a layer on an fp32 residual stream
        dict(name="norm_residual", op="norm_fwd", dtype=BF16, rows=16384, dim=4096, residual=True),
        # the gradients of the norm over each head's 128 outputs: 16 heads of 16,384 tokens
        dict(name="norm_heads_train", op="norm_bwd", dtype=BF16, rows=262144, dim=128, residual=False),
        # fp32 gradients at an odd width, with the residual stream's gradient added
        dict(name="norm_train_odd", op="norm_bwd", dtype=F32, rows=1999, dim=5001, residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_step", "scan_bwd", "scan_bwd", "conv_fwd", "conv_step", "conv_bwd",
                     "norm_fwd", "norm_bwd"])
    dtype = rng.choice([BF16, BF16, F32])
    case = dict(op=op, dtype=dtype)
    if op == "norm_fwd" or op == "norm_bwd":
        dim = _log(rng, 64, 8192)
        case.update(rows=_log(rng, 16, max(17, min(200000, (48 << 20) // dim))), dim=dim, residual=rng.random() < 0.5)
    elif op == "scan_step":
        case.update(batch=_log(rng, 1, 256), dim=_log(rng, 256, 4096), ds=rng.choice([8, 16, 16, 16, rng.randint(5, 32)]),
                    gate=rng.random() < 0.7)
    elif op == "conv_step":
        case.update(batch=_log(rng, 1, 512), dim=_log(rng, 256, 8192), width=rng.choice([2, 3, 4, 4]),
                    silu=rng.random() < 0.7)
    else:
        scan = op.startswith("scan")
        dim = _log(rng, 128, 4096)
        most = (24 << 20 if op == "scan_fwd" else 12 << 20 if scan else 48 << 20) // dim
        tokens = _log(rng, 32, min(16384, most))
        packed = rng.random() < 0.5
        batch = 1 if packed else max(1, min(_log(rng, 1, 16), most // tokens))
        case.update(batch=batch, tokens=tokens, dim=dim, seqs=rng.randint(2, 24) if packed else 0,
                    sliced=rng.random() < 0.5)
        if scan:
            case.update(ds=rng.choice([16, 16, 16, rng.randint(4, 24)]), gate=rng.random() < 0.7)
        else:
            case.update(width=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.7)
    return case


def _lengths(case, g):
    """Lengths of the packed sequences; from four on, one is empty and one is a single token."""
    n, total = case["seqs"], case["tokens"]
    cuts = sorted(torch.randint(0, total + 1, (n - 1,), generator=g).tolist())
    if n >= 4:
        cuts[1] = cuts[0]
        cuts[2] = max(cuts[2], cuts[1])
        cuts[-1] = total - 1
        cuts = sorted(cuts)
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op = case["op"]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    s = dict(case=case, op=op)
    D = case["dim"]
    if op.startswith("norm"):
        R = case["rows"]
        s.update(weight=1 + normal(D, std=0.2, dtype=torch.float32), bias=normal(D, std=0.2, dtype=torch.float32))
        if op == "norm_fwd":
            s["x"] = normal(R, D)
            s["residual"] = normal(R, D, std=3.0, dtype=torch.float32) if case["residual"] else None
        else:
            s["x"] = normal(R, D, std=2.0) + 0.25
            s["grad_y"] = normal(R, D)
            s["grad_residual"] = normal(R, D) if case["residual"] else None
        return s

    B = case["batch"]
    step = op.endswith("step")
    lead = (B,) if step else (B, case["tokens"])
    lengths = None
    if not step:
        if case["seqs"]:
            lengths = _lengths(case, host)
            s["cu_seqlens"] = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).cuda()
            s["offsets"] = s["cu_seqlens"]
        else:
            s["cu_seqlens"] = None
            s["offsets"] = torch.arange(B + 1, dtype=torch.int32, device="cuda") * case["tokens"]
    N = len(lengths) if lengths else B

    if op.startswith("conv"):
        W = case["width"]
        wide = normal(*lead, 2 * D if case.get("sliced") else D)
        s["x"] = wide[..., :D]
        s["weight"] = normal(D, W, std=W ** -0.5, dtype=torch.float32)
        s["bias"] = normal(D, std=0.1, dtype=torch.float32)
        s["state"] = normal(N, W - 1, D)
        if op == "conv_bwd":
            s["grad_y"] = normal(*lead, D)
        return s

    ds = case["ds"]
    if case.get("sliced"):
        wide = normal(*lead, 2 * D)
        s["u"], s["z"] = wide[..., :D], wide[..., D:]
        low = normal(*lead, RANK + 2 * ds)
        s["B"], s["C"] = low[..., RANK:RANK + ds], low[..., RANK + ds:]
    else:
        s["u"], s["z"] = normal(*lead, D), normal(*lead, D)
        s["B"], s["C"] = normal(*lead, ds), normal(*lead, ds)
    if not case["gate"]:
        s["z"] = None
    s["dt"] = normal(*lead, D, std=0.5)
    # step sizes spread over 0.001 .. 0.1 at a zero logit: the bias is softplus's inverse of them
    size = torch.exp(torch.rand(D, generator=gen, device="cuda") * math.log(100.0) + math.log(0.001))
    s["dt_bias"] = size + torch.log(-torch.expm1(-size))
    n = torch.arange(1, ds + 1, device="cuda", dtype=torch.float32)
    s["A"] = -n * torch.exp(0.1 * torch.randn(D, ds, generator=gen, device="cuda"))
    s["D"] = 1 + normal(D, std=0.1, dtype=torch.float32)
    s["state"] = normal(N, D, ds, std=0.5, dtype=torch.float32)
    if op == "scan_bwd":
        s["grad_y"] = normal(*lead, D)
        s["grad_state"] = normal(N, D, ds, std=0.5, dtype=torch.float32)
    return s


# ---- the plain form -------------------------------------------------------------------------------------------------

def _f(x):
    return None if x is None else x.float()


def _flat(x):
    return None if x is None else x.reshape(-1, x.shape[-1]).float()


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _places(offsets, tokens):
    """(sequence of each token, whether the token is its sequence's first, whether its last)"""
    t = torch.arange(tokens, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(offsets[1:].contiguous(), t, right=True)
    return seq, t == offsets[seq], t + 1 == offsets[seq + 1]


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t over the first axis from zero, by doubling."""
    k = 1
    while k < len(a):
        b = torch.cat([b[:k], b[k:] + a[k:] * b[:-k]])
        a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    return b


def _of_sequences(per_token, offsets, otherwise):
    """Each sequence's row of per_token at its given token; the empty ones' from `otherwise`."""
    empty = (offsets[1:] == offsets[:-1]).view(-1, 1, 1)
    return empty, torch.where(empty, otherwise, per_token)


def _states(s):
    u, delta = _flat(s["u"]), _softplus(_flat(s["dt"]) + s["dt_bias"])
    Bm, Cm, z = _flat(s["B"]), _flat(s["C"]), _flat(s["z"])
    seq, first, last = _places(s["offsets"], len(u))
    decay = torch.exp(delta[:, :, None] * s["A"])
    enter = torch.where(first[:, None, None], s["state"][seq], 0.0)
    b = (delta * u)[:, :, None] * Bm[:, None, :] + decay * enter
    a = torch.where(first[:, None, None], 0.0, decay)
    return u, delta, Bm, Cm, z, seq, first, last, decay, enter, _scan(a, b)


def _plain_scan_fwd(s):
    u, delta, Bm, Cm, z, seq, first, last, decay, enter, h = _states(s)
    y = (h * Cm[:, None, :]).sum(-1) + s["D"] * u
    if z is not None:
        y = y * z * torch.sigmoid(z)
    end = (s["offsets"][1:] - 1).clamp(min=0)
    final = _of_sequences(h[end], s["offsets"], s["state"])[1]
    return dict(y=y.view(s["u"].shape).to(s["u"].dtype), state=final)


def _plain_scan_step(s):
    u, delta, z = _f(s["u"]), _softplus(_f(s["dt"]) + s["dt_bias"]), _f(s["z"])
    h = torch.exp(delta[:, :, None] * s["A"]) * s["state"] + (delta * u)[:, :, None] * _f(s["B"])[:, None, :]
    y = (h * _f(s["C"])[:, None, :]).sum(-1) + s["D"] * u
    if z is not None:
        y = y * z * torch.sigmoid(z)
    return dict(y=y.to(s["u"].dtype), state=h)


def _plain_scan_bwd(s):
    u, delta, Bm, Cm, z, seq, first, last, decay, enter, h = _states(s)
    gy = _flat(s["grad_y"])
    out, kind = {}, s["u"].dtype
    if z is not None:
        sig = torch.sigmoid(z)
        yp = (h * Cm[:, None, :]).sum(-1) + s["D"] * u
        out["dz"] = (gy * yp * sig * (1 + z * (1 - sig))).view(s["u"].shape).to(kind)
        gy = gy * z * sig
    c = gy[:, :, None] * Cm[:, None, :] + torch.where(last[:, None, None], s["grad_state"][seq], 0.0)
    after = torch.where(last[:, None, None], 0.0, torch.cat([decay[1:], decay[:1]]))
    G = _scan(after.flip(0), c.flip(0)).flip(0)
    carried = decay * torch.where(first[:, None, None], enter, torch.cat([h[:1], h[:-1]]))
    P = (G * Bm[:, None, :]).sum(-1)
    ddelta = u * P + (G * carried * s["A"]).sum(-1)
    ddt = ddelta * torch.sigmoid(_flat(s["dt"]) + s["dt_bias"])
    begin = s["offsets"][:-1].clamp(max=len(u) - 1)
    out["du"] = (gy * s["D"] + delta * P).view(s["u"].shape).to(kind)
    out["ddt"] = ddt.view(s["u"].shape).to(kind)
    out["dA"] = (G * carried * delta[:, :, None]).sum(0)
    out["dB"] = (G * (delta * u)[:, :, None]).sum(1).view(s["B"].shape).to(kind)
    out["dC"] = (h * gy[:, :, None]).sum(1).view(s["B"].shape).to(kind)
    out["dD"] = (gy * u).sum(0)
    out["ddt_bias"] = ddt.sum(0)
    out["dh0"] = _of_sequences((decay * G)[begin], s["offsets"], s["grad_state"])[1]
    return out


def _taps(x, state, offsets, W):
    """[W, tokens, D]: tap j holds each token's input W-1-j tokens ago, from its sequence's state before the start."""
    T = len(x)
    seq = _places(offsets, T)[0]
    at = torch.arange(T, device="cuda")
    since = at - offsets[seq]
    taps = []
    for back in range(W - 1, -1, -1):
        inside = x[(at - back).clamp(min=0)]
        row = (W - 1 + since - back).clamp(min=0, max=max(0, W - 2))
        taps.append(torch.where((since >= back)[:, None], inside, state[seq, row]) if back else inside)
    return torch.stack(taps), seq, since


def _conv_pre(s, taps):
    return (taps * s["weight"].t()[:, None, :]).sum(0) + s["bias"]


def _plain_conv_fwd(s):
    W = s["case"]["width"]
    x, state, offsets = _flat(s["x"]), _f(s["state"]), s["offsets"]
    p = _conv_pre(s, _taps(x, state, offsets, W)[0])
    if s["case"]["silu"]:
        p = p * torch.sigmoid(p)
    back = torch.arange(W - 1, 0, -1, device="cuda")
    at = offsets[1:, None] - back
    rows = (W - 1 + offsets[1:, None] - offsets[:-1, None] - back).clamp(min=0, max=W - 2)
    old = torch.gather(state, 1, rows.long()[:, :, None].expand(-1, -1, x.shape[1]))
    final = torch.where((at >= offsets[:-1, None])[:, :, None], x[at.clamp(min=0)], old)
    return dict(y=p.view(s["x"].shape).to(s["x"].dtype), state=final.to(s["x"].dtype))


def _plain_conv_step(s):
    window = torch.cat([_f(s["state"]), _f(s["x"])[:, None]], 1)
    p = (window * s["weight"].t()).sum(1) + s["bias"]
    if s["case"]["silu"]:
        p = p * torch.sigmoid(p)
    return dict(y=p.to(s["x"].dtype), state=window[:, 1:].to(s["x"].dtype))


def _plain_conv_bwd(s):
    W = s["case"]["width"]
    x, state, offsets, gp = _flat(s["x"]), _f(s["state"]), s["offsets"], _flat(s["grad_y"])
    taps, seq, since = _taps(x, state, offsets, W)
    if s["case"]["silu"]:
        p = _conv_pre(s, taps)
        sig = torch.sigmoid(p)
        gp = gp * sig * (1 + p * (1 - sig))
    T, D = x.shape
    at = torch.arange(T, device="cuda")
    left = offsets[seq + 1] - 1 - at
    dx, dh0 = torch.zeros_like(gp), torch.zeros_like(state)
    for back in range(W):  # token t's input meets weight W-1-back in token t+back's output
        w = s["weight"][:, W - 1 - back]
        dx = dx + torch.where((left >= back)[:, None], gp[(at + back).clamp(max=T - 1)] * w, 0.0)
        for row in range(W - 1):  # state row `row` is W-1-row tokens before the start, so back-(W-1-row) after it
            t = offsets[:-1] + back - (W - 1 - row)
            met = (t >= offsets[:-1]) & (t < offsets[1:])
            dh0[:, row] += torch.where(met[:, None], gp[t.clamp(0, T - 1)] * w, 0.0)
    return dict(dx=dx.view(s["x"].shape).to(s["x"].dtype), dweight=(taps * gp).sum(1).t(), dbias=gp.sum(0), dh0=dh0)


def _plain_norm_fwd(s):
    x = _f(s["x"])
    out = {}
    if s["residual"] is not None:
        x = x + s["residual"]
        out["residual"] = x
    x = x - x.mean(-1, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5) * s["weight"] + s["bias"]
    return dict(out, y=y.to(s["x"].dtype))


def _plain_norm_bwd(s):
    x, gy = _f(s["x"]), _f(s["grad_y"])
    x = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5)
    xh, g = x * rstd, gy * s["weight"]
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    if s["grad_residual"] is not None:
        dx = dx + _f(s["grad_residual"])
    return dict(dx=dx.to(s["x"].dtype), dweight=(gy * xh).sum(0), dbias=gy.sum(0))


# ---- the framework's calls ------------------------------------------------------------------------------------------

def _own(s):
    import gated_delta_rule_52_amd as kda

    op, case = s["op"], s["case"]
    if op == "scan_fwd":
        y, state = kda.selective_scan_fwd(s["u"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"],
                                          initial_state=s["state"], cu_seqlens=s["cu_seqlens"], dt_softplus=True)
        return dict(y=y, state=state)
    if op == "scan_step":
        # the cached state is kept for the next pass: the new one goes to a buffer of its own
        state = torch.empty_like(s["state"])
        y = kda.selective_scan_step(s["u"], s["dt"], s["A"], s["B"], s["C"], s["state"], s["D"], s["z"], s["dt_bias"],
                                    dt_softplus=True, final_state=state)
        return dict(y=y, state=state)
    if op == "scan_bwd":
        got = kda.selective_scan_bwd(s["u"], s["dt"], s["A"], s["B"], s["C"], s["grad_y"], s["D"], s["z"], s["dt_bias"],
                                     initial_state=s["state"], grad_final_state=s["grad_state"],
                                     cu_seqlens=s["cu_seqlens"], dt_softplus=True, grad_dtype=s["u"].dtype)
        return {k: v for k, v in got.items() if v is not None}
    if op == "conv_fwd":
        y, state = kda.short_conv_fwd(s["x"], s["weight"], s["bias"], initial_state=s["state"],
                                      cu_seqlens=s["cu_seqlens"], silu=case["silu"])
        return dict(y=y, state=state)
    if op == "conv_step":
        state = torch.empty_like(s["state"])
        y = kda.short_conv_step(s["x"], s["weight"], s["state"], s["bias"], silu=case["silu"], final_state=state)
        return dict(y=y, state=state)
    if op == "conv_bwd":
        return kda.short_conv_bwd(s["x"], s["weight"], s["grad_y"], s["bias"], initial_state=s["state"],
                                  cu_seqlens=s["cu_seqlens"], silu=case["silu"], grad_dtype=s["x"].dtype)
    if op == "norm_fwd":
        got = kda.layer_norm_fwd(s["x"], s["weight"], s["bias"], residual=s["residual"])
        return dict(y=got) if s["residual"] is None else dict(y=got[0], residual=got[1])
    return kda.layer_norm_bwd(s["x"], s["grad_y"], s["weight"], s["bias"], grad_residual=s["grad_residual"],
                              grad_dtype=s["x"].dtype)


def run(state):
    return _own(state) if own else globals()["_plain_" + state["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------------------------------------------

def work(case):
    e = 2 if case["dtype"] == BF16 else 4
    op, D = case["op"], case["dim"]
    if op == "norm_fwd":
        n = case["rows"] * D
        return dict(bytes=n * (2 * e + (8 if case["residual"] else 0)) + 8 * D, flops=8 * n)
    if op == "norm_bwd":
        n = case["rows"] * D
        return dict(bytes=n * (3 * e + (e if case["residual"] else 0)) + 12 * D, flops=14 * n)
    rows = case["batch"] * case.get("tokens", 1)
    N = case["seqs"] if case.get("seqs") else case["batch"]
    n = rows * D
    if op.startswith("conv"):
        W = case["width"]
        state = N * (W - 1) * D
        act = 4 if case["silu"] else 0
        if op == "conv_bwd":
            return dict(bytes=3 * e * n + (e + 4) * state + 8 * (W + 1) * D, flops=n * (6 * W + act + 4))
        return dict(bytes=2 * e * n + 2 * e * state + 4 * (W + 1) * D, flops=n * (2 * W + act))
    ds, gate = case["ds"], 1 if case["gate"] else 0
    state, weights = 4 * N * D * ds, 4 * D * (ds + 2)
    if op == "scan_bwd":
        return dict(bytes=e * n * (5 + 2 * gate) + 4 * e * rows * ds + 3 * state + 2 * weights,
                    flops=n * (20 * ds + 12 + 8 * gate))
    return dict(bytes=e * n * (3 + gate) + 2 * e * rows * ds + 2 * state + weights, flops=n * (7 * ds + 6 + 4 * gate))


# ---- the operators' definitions in 64 bits --------------------------------------------------------------------------

def _groups(s, lead):
    """Token numbers [time, members] of sequences that are walked together, with their sequence numbers."""
    B, T = lead
    if s["cu_seqlens"] is None:
        yield torch.arange(B * T, device="cuda").view(B, T).t(), torch.arange(B, device="cuda")
        return
    ends = s["cu_seqlens"].tolist()
    for n, (a, b) in enumerate(zip(ends, ends[1:])):
        if b > a:
            yield torch.arange(a, b, device="cuda")[:, None], torch.tensor([n], device="cuda")


def _exact_scan(s):
    d = lambda x: None if x is None else x.double().reshape(-1, x.shape[-1])  # noqa: E731
    u, raw, Bm, Cm, z = d(s["u"]), d(s["dt"]) + s["dt_bias"].double(), d(s["B"]), d(s["C"]), d(s["z"])
    A, skip, h0 = s["A"].double(), s["D"].double(), s["state"].double()
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    silu = 1.0 if z is None else z / (1 + torch.exp(-z))
    back = s["op"] == "scan_bwd"
    y, final = torch.empty_like(u), h0.clone()
    if back:
        gy = d(s["grad_y"])
        gp = gy * silu
        du, ddelta, dh0 = torch.empty_like(u), torch.empty_like(u), s["grad_state"].double().clone()
        dB, dC, dA = torch.empty_like(Bm), torch.empty_like(Bm), torch.zeros_like(A)
    for at, seq in _groups(s, s["u"].shape[:2]):
        T = len(at)
        block = max(1, (1 << 27) // (at.shape[1] * A.numel()))
        h, kept = h0[seq], []
        for t0 in range(0, T, block):
            i = at[t0:t0 + block]
            decay = torch.exp(delta[i][..., None] * A)
            add = (delta[i] * u[i])[..., None] * Bm[i][:, :, None, :]
            hs = torch.empty_like(add)
            before = h
            for k in range(len(i)):
                h = torch.addcmul(add[k], decay[k], h, out=hs[k])
            y[i] = (hs * Cm[i][:, :, None, :]).sum(-1)
            kept.append((t0, before.clone(), hs if back else None))
        final[seq] = h
        if not back:
            continue
        G = s["grad_state"].double()[seq]
        for t0, before, hs in reversed(kept):
            i = at[t0:t0 + block]
            decay = torch.exp(delta[i][..., None] * A)
            Gs = gp[i][..., None] * Cm[i][:, :, None, :]
            for k in range(len(i) - 1, -1, -1):
                Gs[k] += G
                G = decay[k] * Gs[k]
            carried = torch.cat([before[None], hs[:-1]]) * decay * Gs
            P = (Gs * Bm[i][:, :, None, :]).sum(-1)
            du[i] = gp[i] * skip + delta[i] * P
            ddelta[i] = u[i] * P + (carried * A).sum(-1)
            dA += (carried * delta[i][..., None]).sum((0, 1))
            dB[i] = ((delta[i] * u[i])[..., None] * Gs).sum(2)
            dC[i] = (gp[i][..., None] * hs).sum(2)
        dh0[seq] = G
    yp = y + skip * u
    if not back:
        return dict(y=(yp * silu).view(s["u"].shape), state=final)
    ddt = ddelta / (1 + torch.exp(-raw))
    shape = s["u"].shape
    out = dict(du=du.view(shape), ddt=ddt.view(shape), dA=dA, dB=dB.view(s["B"].shape), dC=dC.view(s["B"].shape),
               dD=(gp * u).sum(0), ddt_bias=ddt.sum(0), dh0=dh0)
    if z is not None:
        sig = 1 / (1 + torch.exp(-z))
        out["dz"] = (gy * yp * (sig + z * sig * (1 - sig))).view(shape)
    return out


def _exact_conv(s):
    """Sequence by sequence on its inputs with the state in front; the gradients by differentiating that."""
    W, silu = s["case"]["width"], s["case"]["silu"]
    x, h0, shape = s["x"].double(), s["state"].double(), s["x"].shape
    x = x.reshape(-1, shape[-1])
    w, b = s["weight"].double(), s["bias"].double()
    back = s["op"] == "conv_bwd"
    gy = s["grad_y"].double().reshape(x.shape) if back else None
    y, final, dx, dh0 = torch.empty_like(x), torch.empty_like(h0), torch.empty_like(x), torch.zeros_like(h0)
    dw, db = torch.zeros_like(w), torch.zeros_like(b)
    ends = s["offsets"].tolist()
    for n, (i, j) in enumerate(zip(ends, ends[1:])):
        line = torch.cat([h0[n], x[i:j]])
        final[n] = line[len(line) - (W - 1):]
        if i == j:
            continue
        windows = line.unfold(0, W, 1)  # [tokens, D, W]
        p = (windows * w).sum(-1) + b
        sig = 1 / (1 + torch.exp(-p))
        y[i:j] = p * sig if silu else p
        if back:
            g = gy[i:j] * (sig + p * sig * (1 - sig)) if silu else gy[i:j]
            dw += (windows * g[..., None]).sum(0)
            db += g.sum(0)
            dline = torch.zeros_like(line)
            for k in range(W):
                dline[k:k + j - i] += g * w[:, k]
            dh0[n], dx[i:j] = dline[:W - 1], dline[W - 1:]
    if back:
        return dict(dx=dx.view(shape), dweight=dw, dbias=db, dh0=dh0)
    return dict(y=y.view(shape), state=final)


def _exact_norm(s):
    x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
    if s["op"] == "norm_fwd":
        out = {}
        if s["residual"] is not None:
            x = out["residual"] = x + s["residual"].double()
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        return dict(out, y=(x - mean) / torch.sqrt(var + 1e-5) * w + b)
    gy = s["grad_y"].double()
    var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
    std = torch.sqrt(var + 1e-5)
    xh = (x - mean) / std
    g = gy * w
    dx = (g - (g.sum(-1, keepdim=True) + xh * (g * xh).sum(-1, keepdim=True)) / x.shape[-1]) / std
    if s["grad_residual"] is not None:
        dx = dx + s["grad_residual"].double()
    return dict(dx=dx, dweight=(gy * xh).sum(0), dbias=gy.sum(0))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm"):
        return _exact_norm(s)
    if op.endswith("step"):  # one token of each sequence
        one = {k: v[:, None] if k in ("u", "dt", "z", "B", "C", "x") and v is not None else v for k, v in s.items()}
        one.update(cu_seqlens=None, offsets=torch.arange(case["batch"] + 1, device="cuda"))
        got = (_exact_scan if op.startswith("scan") else _exact_conv)(one)
        return dict(got, y=got["y"][:, 0])
    return (_exact_scan if op.startswith("scan") else _exact_conv)(s)
