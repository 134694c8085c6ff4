"""The selective scan where it cuts sequences into tiles, and its step where a workgroup takes two sequences, against
references in 64 bits: every tile length, every size of state, sequences as long as 32-bit sizes hold."""
import numpy as np
import pytest

import layer_testlib as ref
import test_gpu_layer as base
from test_gpu_layer import dev, host, kda, layout, scan_inputs  # noqa: F401  (kda is the fixture)

pytestmark = pytest.mark.gpu


def test_scan_of_the_longest_sequences(kda):
    """One channel of one state over 2^31 - 200 tokens, packed and fixed: a length to which no tile can be added in 32
    bits.  Every row is written, and windows of rows, the sequence's two ends among them, equal the definition.  A token's decay
    is at most exp(-1/2), so 250 tokens around a window hold all that reaches it (exp(-125) of the rest)."""
    import torch
    T, around, size = 2 ** 31 - 200, 250, 400
    g = torch.Generator("cuda").manual_seed(1)
    token = lambda: torch.empty(1, T, 1, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    u, B, C, gy = (token().normal_(generator=g) for _ in range(4))
    dt = token().uniform_(generator=g).mul_(0.5).add_(0.5)
    A, h0, gf = torch.full((1, 1), -1.0, device="cuda"), torch.full((1, 1, 1), 0.7, device="cuda"), torch.full((1, 1, 1), -0.3, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    at = [0, T - size, 2 ** 30 - size // 2] + np.random.default_rng(2).integers(around, T - 2 * size, 20).tolist()

    def window(w):
        """(the reference's inputs around rows w to w + size, the first of them, the initial and final gradient's place)"""
        a, b = max(0, w - around), min(T, w + size + around)
        f = lambda t: host(t[0, a:b])  # noqa: E731
        return dict(u=f(u), dt=f(dt), B=f(B), C=f(C), A=np.full((1, 1), -1.0), D=None, z=None, dt_bias=None, softplus=False,
                    h0=np.full((1, 1, 1), float(np.float32(0.7))) if a == 0 else None), a, b

    def written(t):
        return not any(bool(part.isnan().any()) for part in t.view(-1).split(1 << 28))

    print("forward", flush=True)
    y = token().fill_(float("nan"))
    _, final = kda.selective_scan_fwd(u, dt, A, B, C, initial_state=h0, cu_seqlens=cu, y=y)
    torch.cuda.synchronize()
    assert written(y)
    for w in at:
        x, a, b = window(w)
        want, scale = ref.scan_forward(x, [0, b - a]), ref.scan_forward(x, [0, b - a], absolute=True)
        n = ref.scan_roundings(x, [0, b - a])
        part = slice(w - a, w - a + size)
        ref.check(f"y at {w}", host(y[0, w:w + size]), want["y"][part], scale["y"][part], n, "bf16")
        if b == T:
            ref.check("state", host(final), want["final"], scale["final"], n)
    y2, final2 = kda.selective_scan_fwd(u, dt, A, B, C, initial_state=h0)
    assert all(torch.equal(p, q) for p, q in zip(y.view(-1).split(1 << 28), y2.view(-1).split(1 << 28))) and torch.equal(final, final2)
    del y, y2

    print("gradients", flush=True)
    out = {k: token().fill_(float("nan")) for k in ("du", "ddt", "dB", "dC")}
    got = kda.selective_scan_bwd(u, dt, A, B, C, gy, initial_state=h0, grad_final_state=gf, cu_seqlens=cu,
                                 grad_dtype=torch.bfloat16, out=out)
    torch.cuda.synchronize()
    assert all(written(v) for v in out.values()) and bool(got["dA"].isfinite().all())
    for w in at:
        x, a, b = window(w)
        end = host(gf) if b == T else None
        want = ref.scan_backward(x, [0, b - a], host(gy[0, a:b]), end)
        scale = ref.scan_backward(x, [0, b - a], host(gy[0, a:b]), end, absolute=True)
        n = 2 * ref.scan_roundings(x, [0, b - a])
        part = slice(w - a, w - a + size)
        for k in out:
            ref.check(f"{k} at {w}", host(out[k][0, w:w + size]), want[k][part], scale[k][part], n, "bf16")
        if a == 0:
            ref.check("dh0", host(got["dh0"]), want["dh0"], scale["dh0"], n)


# (sequences, ds, input, output): a state of every arrangement of lanes, some of them padded, in tiles of 64 tokens
STATES = [((1, 300), 12, "bf16", "fp32"), ((1, 300), 20, "fp32", "fp32"), ((1, 300), 32, "bf16", "bf16"),
          ((1, 300), 40, "fp32", "fp32"), ((1, 300), 64, "bf16", "fp32"), ((2, 129), 3, "fp32", "fp32"),
          ([200, 0, 1, 131], 8, "bf16", "fp32"), ([200, 0, 1, 131], 20, "bf16", "fp32"), ([200, 0, 1, 131], 64, "fp32", "fp32"),
          ([65, 0, 64, 1, 63, 190], 33, "bf16", "fp32")]


@pytest.mark.parametrize("seqs,ds,dtype,out", STATES)
@pytest.mark.parametrize("gate", [True, False])
def test_tiles_of_every_state_size(kda, seqs, ds, dtype, out, gate):
    base.test_scan_forward(kda, seqs, 70, ds, dtype, out, dict(gate=gate))
    base.test_scan_gradients(kda, seqs, 70, ds, dtype, out, dict(gate=gate))


def walk(offsets, u, dt, A, B, C, D, z, bias, h0, gy, gf):
    """The definition in 64 bits on the GPU, token by token: outputs, final states and gradients."""
    import torch
    d = lambda t: t.double().reshape(-1, t.shape[-1])  # noqa: E731
    u, B, C, z, gy, A, D, h0, gf = d(u), d(B), d(C), d(z), d(gy), A.double(), D.double(), h0.double(), gf.double()
    raw = d(dt) + bias.double()
    delta, sg = torch.logaddexp(raw, torch.zeros_like(raw)), 1 / (1 + torch.exp(-z))
    gate = z * sg
    gp, xl = gy * gate, delta * u
    rows, dim, ds = len(u), *A.shape
    h, carried = (torch.empty(rows, dim, ds, dtype=torch.float64, device="cuda") for _ in range(2))
    final, dh0, dA = h0.clone(), gf.clone(), torch.zeros_like(A)
    dB, dC, P, S = torch.empty_like(B), torch.empty_like(C), torch.empty_like(u), torch.empty_like(u)
    for n, (s, e) in ref.spans(offsets):
        state = h0[n]
        for t in range(s, e):
            torch.mul(torch.exp(delta[t, :, None] * A), state, out=carried[t])
            state = torch.addcmul(carried[t], xl[t, :, None], B[t], out=h[t])
        if e > s:
            final[n] = state
        g = gf[n]
        for t in range(e - 1, s - 1, -1):
            G = torch.addcmul(g, gp[t, :, None], C[t])
            c = G * carried[t]
            dC[t], dB[t], P[t], S[t] = gp[t] @ h[t], xl[t] @ G, G @ B[t], (c * A).sum(-1)
            dA.addcmul_(c, delta[t, :, None])
            g = torch.exp(delta[t, :, None] * A) * G
        dh0[n] = g
    yp = (h * C[:, None]).sum(-1) + D * u
    ddt = (u * P + S) / (1 + torch.exp(-raw))
    return dict(y=yp * gate, final=final, du=D * gp + delta * P, ddt=ddt, dz=gy * yp * sg * (1 + z * (1 - sg)), dB=dB, dC=dC,
                dA=dA, dD=(gp * u).sum(0), ddt_bias=ddt.sum(0), dh0=dh0)


@pytest.mark.parametrize("seqs,ds,dtype,tile", [
    ((1, 4499), 16, "bf16", 144), ((1, 8200), 16, "bf16", 256), ((3, 1500), 16, "fp32", 144),
    ([700, 0, 1, 1500, 144, 0, 998], 16, "fp32", 112), ((1, 2400), 24, "bf16", 80), ((1, 2400), 40, "fp32", 80),
    ([3000, 1, 0, 2000], 8, "bf16", 160)])
def test_long_tiles(kda, seqs, ds, dtype, tile):
    """Tiles above the shortest, of lengths that are no powers of two, the last of a sequence shorter.  Every token's row
    is held by itself: a state's roundings, some 20 a token, add up independently over the tokens that it remembers, at
    most the longest sequence; the gradients have them on both ways, and sums over channels or tokens some more."""
    import torch
    dim = 2048
    offsets, B, T, cu = layout(seqs)
    N, rows = len(offsets) - 1, offsets[-1]
    g = torch.Generator("cuda").manual_seed(ds + rows)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    tokens = lambda d: n(B, T, d).to(base.tdtype(dtype))  # noqa: E731
    u, dt, z, gy, Bm, Cm = tokens(dim), tokens(dim), tokens(dim), tokens(dim), tokens(ds), tokens(ds)
    A, D, bias, h0, gf = -torch.exp(n(dim, ds)), n(dim), n(dim) - 3, n(N, dim, ds), n(N, dim, ds)
    slots = N * -(-T // tile) if cu is None else T // tile + N
    assert kda.selective_scan_fwd_workspace_bytes(u, ds, cu) == slots * dim * (ds + 1) * 4, "another tile length"
    kw = dict(initial_state=h0, cu_seqlens=cu, dt_softplus=True)
    y, final = kda.selective_scan_fwd(u, dt, A, Bm, Cm, D, z, bias, out_dtype=torch.float32, **kw)
    got = kda.selective_scan_bwd(u, dt, A, Bm, Cm, gy, D, z, bias, grad_final_state=gf, **kw)
    got.update(y=y, final=final)
    want = walk(offsets, u, dt, A, Bm, Cm, D, z, bias, h0, gy, gf)
    longest = max(b - a for a, b in zip(offsets, offsets[1:]))
    bound = 2 * (20 * longest) ** .5 * 2 ** -24
    for k, v in want.items():
        v = v.reshape(-1, v.shape[-1]) if k not in ("final", "dh0") else v.reshape(N, -1)
        v = v if k not in ("dD", "ddt_bias") else v.reshape(1, -1)
        err = (got[k].double().reshape(v.shape) - v).norm(dim=1) / v.norm(dim=1)
        most = bound if k in ("y", "final") else 2 * bound if k in ("du", "ddt", "dz", "dB", "dC", "dh0") else 8 * bound
        print(f"    {k}: worst row {float(err.max() / most):.3f} of its bound", flush=True)
        assert float(err.max()) < most, k


@pytest.mark.parametrize("N,dim,ds,dtype", [(65, 4096, 16, "bf16"), (129, 2050, 13, "fp32"), (67, 4096, 40, "fp32"),
                                            (131, 2100, 32, "bf16")])
@pytest.mark.parametrize("gate", [True, False])
def test_steps_of_a_full_batch(kda, N, dim, ds, dtype, gate):
    """Batches from which on a workgroup takes two sequences, odd ones: in place, against the definition and bit for bit
    against smaller batches, of which it takes one each."""
    import torch
    assert N * -(-dim // 64) >= 4096 and (N - N // 2) * -(-dim // 64) < 4096
    offsets = list(range(N + 1))
    x = scan_inputs(4, offsets, N, dim, ds, dtype, gate=gate)
    s = {k: None if x[k] is None else dev(x[k], dtype, sliced=k == "B") for k in ("u", "dt", "B", "C", "z")}
    p = {k: dev(x[k]) for k in ("A", "D", "dt_bias")}

    def step(a, b, state):
        t = {k: None if v is None else v[a:b] for k, v in s.items()}
        return kda.selective_scan_step(t["u"], t["dt"], p["A"], t["B"], t["C"], state, p["D"], t["z"], p["dt_bias"],
                                       dt_softplus=True, out_dtype=torch.float32)

    state, half = dev(x["h0"]), N // 2
    parts = dev(x["h0"][:half]), dev(x["h0"][half:])
    y = step(0, N, state)
    y0, y1 = step(0, half, parts[0]), step(half, N, parts[1])
    assert torch.equal(y, torch.cat([y0, y1])) and torch.equal(state, torch.cat(parts))
    want, size = ref.scan_forward(x, offsets), ref.scan_forward(x, offsets, absolute=True)
    n = ref.scan_roundings(x, offsets)
    ref.check("y", host(y), want["y"], size["y"], n)
    ref.check("state", host(state), want["final"], size["final"], n)
    other = torch.full_like(state, 7.0)  # to memory of its own, the old state kept
    old = dev(x["h0"])
    t = {k: v for k, v in s.items() if v is not None}
    y2 = kda.selective_scan_step(t["u"], t["dt"], p["A"], t["B"], t["C"], old, p["D"], t.get("z"), p["dt_bias"], dt_softplus=True,
                                 out_dtype=torch.float32, final_state=other)
    assert torch.equal(y2, y) and torch.equal(other, state) and torch.equal(old, dev(x["h0"]))
