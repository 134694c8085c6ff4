"""The selective scan where it cuts sequences into tiles, against references in 64 bits: sequences as long as 32-bit
sizes hold."""
import numpy as np
import pytest

import layer_testlib as ref
from test_gpu_layer import host, kda  # noqa: F401  (kda is the fixture)

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
