"""64-bit references of the layer operators (selective scan, short convolution, layer norm) and the error bounds
that their GPU tests use.

The references follow the definitions sequence by sequence and token by token in numpy.  Each also runs in
`absolute` terms: the same sums with every term's absolute value.  A result computed in fp32 with n roundings on
the way to it is off by at most about n * 2^-24 of that absolute sum; `check` holds every element to it, and the
2-norm to 4 sqrt(n) * 2^-24, which independent roundings stay under.  A result rounded to bf16 at the end adds
half a bf16 step, 2^-8 relative.
"""
import numpy as np

EPS = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def check(name, got, ref, scale, roundings, out="fp32"):
    """got within the bound of ref; scale: the absolute sum.  Values below 2^-100 count as zero."""
    got, ref, scale = (np.asarray(a, dtype=np.float64) for a in (got, ref, scale))
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.isfinite(got).all(), f"{name}: not finite"
    err = np.abs(got - ref)
    bound = roundings * EPS * scale + HALF_STEP[out] * np.abs(ref) * (1 + roundings * EPS) + 2.0 ** -100
    worst = float((err / bound).max()) if err.size else 0.0
    norm = 4 * np.sqrt(roundings) * EPS * np.linalg.norm(scale) + HALF_STEP[out] * np.linalg.norm(ref) + 2.0 ** -100
    share = float(np.linalg.norm(err) / norm)
    print(f"    {name}: {worst:.3f} of the element bound, {share:.3f} of the norm's", flush=True)
    assert worst <= 1, f"{name}: {worst:.3g} times its bound"
    assert share <= 1, f"{name}: {share:.3g} times the bound of its norm"


def softplus(x):
    return np.logaddexp(x, 0.0)


def sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1, e) / (1 + e)


def spans(offsets):
    return list(enumerate(zip(offsets, offsets[1:])))


# ---- selective scan ----------------------------------------------------------------------------------------

def scan_forward(x, offsets, absolute=False):
    """x: dict of arrays u, dt, B, C [rows, .], A, and D, z, dt_bias, h0 or None, softplus.  Returns a dict with y,
    final, and what the gradients need."""
    ab = np.abs if absolute else (lambda a: a)
    u, B, C = ab(x["u"]), ab(x["B"]), ab(x["C"])
    raw = x["dt"] + (0 if x["dt_bias"] is None else x["dt_bias"])
    delta = softplus(raw) if x["softplus"] else raw
    D = np.zeros(u.shape[1]) if x["D"] is None else ab(x["D"])
    N, dim, ds = len(offsets) - 1, u.shape[1], B.shape[1]
    h0 = np.zeros((N, dim, ds)) if x["h0"] is None else ab(x["h0"])
    yp = np.zeros_like(u)
    h = np.zeros((len(u), dim, ds))
    carried = np.zeros_like(h)
    final = h0.copy()
    decay = np.exp(delta[:, :, None] * x["A"])
    for n, (s, e) in spans(offsets):
        state = h0[n]
        for t in range(s, e):
            carried[t] = decay[t] * state
            state = carried[t] + ab(delta[t] * u[t])[:, None] * B[t]
            h[t] = state
            yp[t] = state @ C[t] + D * u[t]
        final[n] = state
    gate = 1.0 if x["z"] is None else ab(x["z"] * sigmoid(x["z"]))
    return dict(y=yp * gate, final=final, yp=yp, h=h, carried=carried, decay=decay, delta=delta, raw=raw, gate=gate)


def scan_backward(x, offsets, grad_y, grad_final=None, absolute=False):
    ab = np.abs if absolute else (lambda a: a)
    f = scan_forward(x, offsets, absolute)
    u, B, C, A, delta = ab(x["u"]), ab(x["B"]), ab(x["C"]), ab(x["A"]), ab(f["delta"])
    D = np.zeros(u.shape[1]) if x["D"] is None else ab(x["D"])
    gy = ab(grad_y)
    gp = gy * f["gate"]
    N, dim, ds = len(offsets) - 1, u.shape[1], B.shape[1]
    G = np.zeros_like(f["h"])
    dh0 = np.zeros((N, dim, ds)) if grad_final is None else ab(grad_final).copy()
    for n, (s, e) in spans(offsets):
        g = dh0[n]
        for t in range(e - 1, s - 1, -1):
            G[t] = g + gp[t][:, None] * C[t]
            g = f["decay"][t] * G[t]
        dh0[n] = g
    P = (G * B[:, None, :]).sum(-1)
    slope = sigmoid(f["raw"]) if x["softplus"] else 1.0
    inside = np.zeros(len(u), bool)
    inside[offsets[0]:offsets[-1]] = True
    gc = G * f["carried"]
    ddt = slope * (u * P + (gc * A).sum(-1))
    out = dict(du=D * gp + delta * P, ddt=ddt, dA=(gc * delta[:, :, None]).sum(0),
               dB=(G * (delta * u)[:, :, None]).sum(1), dC=(f["h"] * gp[:, :, None]).sum(1), dh0=dh0,
               dD=None if x["D"] is None else (gp * u)[inside].sum(0),
               ddt_bias=None if x["dt_bias"] is None else ddt[inside].sum(0), dz=None)
    if x["z"] is not None:
        sg = sigmoid(x["z"])
        # in absolute terms the slope's sum is 1 + |z| (1 - s): near z = -1.28 it cancels, and each rounding of its
        # terms is relative to them, not to the sum
        out["dz"] = gy * f["yp"] * sg * (1 + ab(x["z"]) * (1 - sg))
    return out


def scan_roundings(x, offsets):
    """Roundings behind a state: per token the decay's (its exponent X = |delta A| log2 e carries 8 of its own: the
    step size's 6, the product's and A log2 e's; exp2 two), the carried product, the added term's three and the
    sum; the same again on the way out."""
    f = softplus(x["dt"] + (0 if x["dt_bias"] is None else x["dt_bias"])) if x["softplus"] else np.abs(x["dt"])
    X = float((f[:, :, None] * np.abs(x["A"])).max()) * 1.4427 if f.size else 0.0
    longest = max([e - s for _, (s, e) in spans(offsets)] + [1])
    return (8 * X + 8) * longest + 24 + x["B"].shape[1]


# ---- short convolution -------------------------------------------------------------------------------------

def conv_forward(x, w, b, h0, offsets, silu, absolute=False):
    ab = np.abs if absolute else (lambda a: a)
    W, N, dim = w.shape[1], len(offsets) - 1, x.shape[1]
    h0 = np.zeros((N, W - 1, dim)) if h0 is None else h0
    p, final = np.zeros_like(x), h0.copy()
    for n, (s, e) in spans(offsets):
        line = np.concatenate([h0[n], x[s:e]])
        for t in range(s, e):
            p[t] = (ab(line[t - s:t - s + W]) * ab(w.T)).sum(0) + (0 if b is None else ab(b))
        final[n] = line[len(line) - (W - 1):]
    return (p * sigmoid(p) if silu and not absolute else p), final, p


def conv_backward(x, w, b, h0, offsets, silu, grad_y, grad_final=None, absolute=False):
    ab = np.abs if absolute else (lambda a: a)
    W, N, dim = w.shape[1], len(offsets) - 1, x.shape[1]
    p = conv_forward(x, w, b, h0, offsets, silu)[2]
    sg = sigmoid(p)
    gp = ab(grad_y) * (ab(sg * (1 + p * (1 - sg))) if silu else 1.0)
    if absolute and silu:  # the slope's own error: its derivative (at most 1/2) times p's absolute sum
        gp = gp + ab(grad_y) * conv_forward(x, w, b, h0, offsets, silu, True)[2]
    h0 = np.zeros((N, W - 1, dim)) if h0 is None else h0
    dx, dw, db, dh0 = np.zeros_like(x), np.zeros_like(w), np.zeros(dim), np.zeros((N, W - 1, dim))
    for n, (s, e) in spans(offsets):
        line, d = np.concatenate([h0[n], x[s:e]]), np.zeros((W - 1 + e - s, dim))
        for t in range(e - s):
            for j in range(W):
                d[t + j] += gp[s + t] * ab(w[:, j])
                dw[:, j] += gp[s + t] * ab(line[t + j])
            db += gp[s + t]
        if grad_final is not None:
            d[len(d) - (W - 1):] += ab(grad_final[n])
        dh0[n], dx[s:e] = d[:W - 1], d[W - 1:]
    return dict(dx=dx, dweight=dw, dbias=None if b is None else db, dh0=dh0)


# ---- layer norm --------------------------------------------------------------------------------------------

def norm_forward(x, w, b, eps):
    mean, var = x.mean(-1, keepdims=True), x.var(-1, keepdims=True)
    rstd = 1 / np.sqrt(var + eps)
    return (x - mean) * rstd * (1 if w is None else w) + (0 if b is None else b), (x - mean) * rstd, rstd


def norm_backward(x, w, gy, eps, grad_residual=None):
    _, xh, rstd = norm_forward(x, w, None, eps)
    g = gy * (1 if w is None else w)
    dx = rstd * (g - g.mean(-1, keepdims=True) - xh * (g * xh).mean(-1, keepdims=True))
    return dict(dx=dx + (0 if grad_residual is None else grad_residual), dweight=(gy * xh).sum(0), dbias=gy.sum(0))


def norm_scales(x, w, b, gy, eps, grad_residual=None):
    """Absolute sums of y, dx, dweight and dbias.  x - mean is off by roundings of |x| + mean |x|; rstd's relative
    error is that of the variance, which a deviation's error reaches through 2 |x - mean|."""
    _, xh, rstd = norm_forward(x, w, b, eps)
    aw = 1 if w is None else np.abs(w)
    dev = rstd * (np.abs(x) + np.abs(x).mean(-1, keepdims=True))  # error unit of (x - mean) rstd from x - mean
    rel = (2 * np.abs(xh) * dev).mean(-1, keepdims=True) + 1      # and of rstd
    c = dev + np.abs(xh) * rel
    y = aw * c + (0 if b is None else np.abs(b))
    if gy is None:
        return dict(y=y)
    g = np.abs(gy) * aw
    m2 = (g * np.abs(xh)).mean(-1, keepdims=True)
    dx = rstd * rel * (g + g.mean(-1, keepdims=True) + np.abs(xh) * m2) + rstd * (c * m2 + np.abs(xh) * (g * c).mean(-1, keepdims=True))
    return dict(y=y, dx=dx + (0 if grad_residual is None else np.abs(grad_residual)),
                dweight=(np.abs(gy) * c).sum(0), dbias=np.abs(gy).sum(0))
