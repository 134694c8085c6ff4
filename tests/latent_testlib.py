"""64-bit references of latent attention (rotary positions, attention over expanded keys and values, its gradients, the
absorbed form over a cache) in numpy, and the error bounds that their GPU tests use.

A bound is a sum over the roundings behind a result, each half a step of its type (`U`) relative to the value rounded:

- a score is a sum of d products in fp32, scaled, off by at most (d + 4) U32 of the same sum in absolute terms; that is an
  absolute error of the exponent, so a relative one of the weight.  exp2 and the product in front of it add 4 U32 and 2 U32
  of the exponent's size;
- a weight is rounded to the operand's type where a matrix product takes it (bf16: U16 of it; fp32: exact);
- a sum of n products in fp32 is off by at most (n + 4) U32 of its absolute sum;
- the result is rounded once to its own type.

`check` holds every element to the sum of these, and the 2-norm of all errors to what independent roundings stay under:
the weights' roundings add up like the root of their squares' sum.
"""
import numpy as np

U32, U16 = 2.0 ** -24, 2.0 ** -8
U = {"bf16": U16, "fp32": U32}


def check(name, got, ref, bound, norm_bound):
    """got within `bound` of ref element by element, and within `norm_bound` (an array of the same shape) in the norm."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), f"{name}: infinities differ"
    got, ref, bound, norm_bound = (np.where(inf, 0.0, np.broadcast_to(a, inf.shape)) for a in (got, ref, bound, norm_bound))
    assert np.isfinite(got).all(), f"{name}: not finite"
    err = np.abs(got - ref)
    tiny = 2.0 ** -100
    worst = float((err / (bound + tiny)).max()) if err.size else 0.0
    share = float(np.linalg.norm(err) / (np.linalg.norm(norm_bound) + tiny))
    print(f"    {name}: {worst:.3f} of the element bound, {share:.3f} of the norm's", flush=True)
    assert worst <= 1, f"{name}: {worst:.3g} times its bound"
    assert share <= 1, f"{name}: {share:.3g} times the bound of its norm"


def sequences(off_q, off_k):
    return [(slice(a, b), slice(c, d)) for a, b, c, d in zip(off_q, off_q[1:], off_k, off_k[1:])]


def seen(nq, nk, causal):
    """[nq, nk]: whether a query sees a key."""
    if not causal:
        return np.ones((nq, nk), bool)
    return np.arange(nk)[None, :] <= np.arange(nq)[:, None] + nk - nq


def softmax(s, see):
    """(weights, lse) of scores [nq, nk]; rows that see nothing get zeros and -inf."""
    s = np.where(see, s, -np.inf)
    top = s.max(-1, initial=-np.inf)
    at = np.where(np.isfinite(top), top, 0.0)
    e = np.exp(s - at[:, None])
    total = e.sum(-1)
    with np.errstate(divide="ignore"):
        lse = at + np.log(total)
    return e / np.where(total == 0, 1, total)[:, None], lse


def attend(q, k, kr, v, off_q, off_k, scale, causal, kind="fp32", out="fp32"):
    """q [Tq,H,dn+dr], k [Tk,H,dn], kr [Tk,dr], v [Tk,H,dv] -> dict of o, lse, and their bounds."""
    Tq, H, d = q.shape
    o, lse = np.zeros((Tq, H, v.shape[-1])), np.full((Tq, H), -np.inf)
    eo, no, el = np.zeros_like(o), np.zeros_like(o), np.zeros_like(lse)
    for sq, sk in sequences(off_q, off_k):
        for h in range(H):
            kk = np.concatenate([k[sk, h], kr[sk]], -1)
            see = seen(sq.stop - sq.start, sk.stop - sk.start, causal)
            if not see.size:
                continue
            p, l = softmax(q[sq, h] @ kk.T * scale, see)
            x = np.abs(q[sq, h]) @ np.abs(kk).T * scale  # in absolute terms
            ex = np.where(see, (d + 6) * U32 * x + 4 * U32, 0.0).max(-1, initial=0.0)[:, None]
            n = see.sum(-1)[:, None]
            u = U16 if kind == "bf16" else 0.0
            a = p @ np.abs(v[sk, h])
            o[sq, h], lse[sq, h] = p @ v[sk, h], l
            rest = (2 * ex + 2 * (n + 6) * U32) * a + U[out] * np.abs(o[sq, h])
            eo[sq, h] = u * a + rest
            no[sq, h] = u * np.sqrt((p * p) @ (v[sk, h] ** 2)) + rest
            el[sq, h] = (ex + (n + 8) * U32)[:, 0] + 8 * U32 * np.abs(np.where(np.isfinite(l), l, 0))
    return dict(o=o, lse=lse, eo=eo, no=no, el=el)


def attend_grads(q, k, kr, v, o, lse, go, off_q, off_k, scale, causal, kind="fp32", out="fp32"):
    """The gradients from given o and lse, as the entry point takes them, and their bounds: name -> (value, element bound,
    norm bound).

    delta_i = grad_o_i . o_i = sum_j p_ij dp_ij.  Where o is bf16 the two differ by what o's roundings make of it, a number
    that is known here.  A kernel may take either, or what lies between: ds is linear in delta, so with the second as the
    value the bound of ds has that number times p.  The second is a sum over weights that are each off by ep, so it is off
    by at most sum_j p_ij ep_ij (|dp_ij| + |delta_i|)."""
    H, d = q.shape[1:]
    dn = k.shape[-1]
    z = np.zeros_like
    g = dict(dq=z(q), dk=np.zeros((len(k), H, d)), dv=z(v))
    e, m = {n: z(a) for n, a in g.items()}, {n: z(a) for n, a in g.items()}
    u = U16 if kind == "bf16" else 0.0
    for sq, sk in sequences(off_q, off_k):
        for h in range(H):
            kk = np.concatenate([k[sk, h], kr[sk]], -1)
            see = seen(sq.stop - sq.start, sk.stop - sk.start, causal)
            if not see.size:
                continue
            qh, vh, gh, oh = q[sq, h], v[sk, h], go[sq, h], o[sq, h]
            l = np.where(np.isfinite(lse[sq, h]), lse[sq, h], 0.0)[:, None]
            s = qh @ kk.T * scale
            p = np.where(see, np.exp(np.where(see, s - l, 0.0)), 0.0)
            x = np.abs(qh) @ np.abs(kk).T * scale
            ep = (d + 8) * U32 * x + 4 * U32 * np.abs(l) + 6 * U32  # relative, of a weight
            dp, delta = gh @ vh.T, (gh * oh).sum(-1)[:, None]
            between = 0.0
            if kind == "bf16":
                given, delta = delta, (p * dp).sum(-1)[:, None]
                between = np.abs(given - delta) + (p * ep * (np.abs(dp) + np.abs(delta))).sum(-1)[:, None]
            ds = p * (dp - delta)
            eds = p * between + p * (v.shape[-1] + 6) * U32 * (np.abs(gh) @ np.abs(vh).T + (np.abs(gh) * np.abs(oh)).sum(-1)[:, None]) + np.abs(ds) * (ep + 2 * U32)
            for name, a, ea, b, f, at in (("dv", p.T, (p * ep).T, gh, 1.0, sk), ("dk", ds.T, eds.T, qh, scale, sk), ("dq", ds, eds, kk, scale, sq)):
                ab, n = np.abs(b), a.shape[1]
                g[name][at, h] = f * (a @ b)
                rest = f * ((ea + (n + 6) * U32 * np.abs(a)) @ ab)
                e[name][at, h] = rest + f * u * (np.abs(a) @ ab)
                m[name][at, h] = rest + f * u * np.sqrt((a * a) @ (b * b))
    got = {n: (g[n], e[n], m[n]) for n in ("dq", "dv")}
    got["dk"] = tuple(t["dk"][..., :dn] for t in (g, e, m))
    r, er, mr = (t["dk"][..., dn:] for t in (g, e, m))
    got["dk_rope"] = (r.sum(1), er.sum(1) + (H + 2) * U32 * np.abs(r).sum(1), np.sqrt((mr ** 2).sum(1)) + (H + 2) * U32 * np.abs(r).sum(1))
    return {n: (val, eb + U[out] * np.abs(val), nb + U[out] * np.abs(val)) for n, (val, eb, nb) in got.items()}


def cached_rows(cache, table, length):
    """The rows of a sequence that exist: cache [blocks, page, W], table [max_blocks]."""
    page = cache.shape[1]
    rows = []
    for pos in range(max(0, min(length, len(table) * page))):
        b = table[pos // page]
        if 0 <= b < len(cache):
            rows.append(cache[b, pos % page])
    return np.array(rows).reshape(len(rows), cache.shape[2])


def step(ql, qr, cache, table, lengths, scale, kind="fp32", out="fp32"):
    """ql [N,H,dl], qr [N,H,dr] -> dict as attend's: every head's key is a cached row, its value the row's first dl."""
    N, H, dl = ql.shape
    got = dict(o=np.zeros((N, H, dl)), lse=np.full((N, H), -np.inf), eo=np.zeros((N, H, dl)), no=np.zeros((N, H, dl)), el=np.zeros((N, H)))
    for n in range(N):
        rows = cached_rows(cache, table[n], lengths[n])
        if not len(rows):
            continue
        q = np.concatenate([ql[n], qr[n]], -1)[None]
        one = attend(q.transpose(1, 0, 2), rows[:, None, :dl], rows[:, dl:], rows[:, None, :dl], [0, H], [0, len(rows)], scale, False, kind, out)
        for key in got:
            got[key][n] = one[key][:, 0]
    return got


def rotate(x, positions, inv_freq, interleaved, offset, scale, sign=1):
    """x [rows, H, D] turned; inv_freq as float64 of the fp32 values."""
    y = np.array(x, np.float64)
    half = len(inv_freq)
    a = positions.astype(np.float64)[:, None, None] * inv_freq
    c, s = np.cos(a) * scale, np.sin(a) * scale * sign
    part = x[..., offset:offset + 2 * half]
    p, q = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :half], part[..., half:])
    t, w = p * c - q * s, q * c + p * s
    y[..., offset:offset + 2 * half] = np.stack([t, w], -1).reshape(part.shape) if interleaved else np.concatenate([t, w], -1)
    return y


def rotate_bound(x, half, interleaved, offset, scale, out):
    """Angles: 2^-25 turns from the fraction's rounding (pi 2^-24 of the radius), 4 U32 from sine and cosine, 4 from the products
    and the sum; and the result's rounding (added by the caller relative to its value)."""
    b = np.zeros_like(x)
    part = np.abs(x[..., offset:offset + 2 * half])
    p, q = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :half], part[..., half:])
    r = (p + q) * abs(scale) * (np.pi + 8) * U32
    b[..., offset:offset + 2 * half] = np.stack([r, r], -1).reshape(part.shape) if interleaved else np.concatenate([r, r], -1)
    return b
