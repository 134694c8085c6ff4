"""Layer operators on one position of every sequence of a long batch, as it lies: rows a whole sequence apart."""
import pytest

from test_gpu_layer import kda  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def test_one_position_of_a_long_batch(kda):
    """Strides from 2^22 elements on: the same bits as with dense copies, in and out."""
    import torch
    B, T, dim, ds, t = 3, 2100, 2048, 16, 1733
    assert T * dim >= 1 << 22
    g = torch.Generator("cuda").manual_seed(1)
    n = lambda *s, dtype=torch.bfloat16: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    f = torch.float32
    far = [n(B, T, dim)[:, t] for _ in range(4)]
    u, dt, z, gy = far
    low = n(B, T * dim)[:, 7:7 + 2 * ds]
    Bm, Cm = low[:, :ds], low[:, ds:]
    A, D, bias, h0 = -torch.exp(n(dim, ds, dtype=f)), n(dim, dtype=f), n(dim, dtype=f) - 3, n(B, dim, ds, dtype=f)
    assert all(v.stride(0) >= 1 << 22 for v in far + [Bm, Cm])
    dense = lambda *v: [x.contiguous() for x in v]  # noqa: E731
    place = lambda: torch.full((B, T, dim), 5.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731

    def same(a, b):
        assert torch.equal(a, b)

    def alone(whole):
        assert bool((whole[:, :t] == 5).all()) and bool((whole[:, t + 1:] == 5).all())

    # the scan: step, one-token prompt with and without its state, gradients
    s0, s1, out = h0.clone(), h0.clone(), place()
    du, ddt, dB, dC, dz = dense(u, dt, Bm, Cm, z)
    y = kda.selective_scan_step(du, ddt, A, dB, dC, s0, D, dz, bias, dt_softplus=True)
    kda.selective_scan_step(u, dt, A, Bm, Cm, s1, D, z, bias, dt_softplus=True, y=out[:, t])
    same(s0, s1), same(out[:, t], y), alone(out)
    one = lambda *v: [x[:, None] for x in v]  # noqa: E731
    for state in (True, False):
        kw = dict(initial_state=h0, dt_softplus=True, output_final_state=state)
        w = [*one(u, dt), A, *one(Bm, Cm), D, *one(z), bias]
        got = kda.selective_scan_fwd(*w, **kw)
        same(got[0][:, 0], y)
        if state:
            same(got[1], s0)
    want = kda.selective_scan_bwd(*one(du, ddt), A, *one(dB, dC), *one(gy.contiguous()), D, *one(dz), bias, initial_state=h0,
                                  dt_softplus=True, grad_dtype=torch.bfloat16)
    out = {k: place()[:, t:t + 1] for k in ("du", "ddt", "dz")}
    out.update({k: n(B, T * dim)[:, None, 9:9 + ds] for k in ("dB", "dC")})
    got = kda.selective_scan_bwd(*one(u, dt), A, *one(Bm, Cm), *one(gy), D, *one(z), bias, initial_state=h0, dt_softplus=True,
                                 grad_dtype=torch.bfloat16, out=out)
    for k, v in want.items():
        same(got[k], v)

    # the convolution: step, one-token prompt, gradients
    w, b, c0 = n(dim, 4, dtype=f), n(dim, dtype=f), n(B, 3, dim)
    s0, s1, out = c0.clone(), c0.clone(), place()
    y = kda.short_conv_step(du, w, s0, b, silu=True)
    kda.short_conv_step(u, w, s1, b, silu=True, y=out[:, t])
    same(s0, s1), same(out[:, t], y), alone(out)
    same(kda.short_conv_fwd(u[:, None], w, b, initial_state=c0, silu=True)[0][:, 0], y)
    want = kda.short_conv_bwd(du[:, None], w, gy.contiguous()[:, None], b, initial_state=c0, silu=True, grad_dtype=torch.bfloat16)
    got = kda.short_conv_bwd(u[:, None], w, gy[:, None], b, initial_state=c0, silu=True, out=dict(dx=place()[:, t:t + 1]),
                             grad_dtype=torch.bfloat16)
    for k, v in want.items():
        same(got[k], v)

    # layer norm, with rows of a head and of the model's width
    for width in (2048, 128, 5):
        x, r, gx = u[:, :width], z[:, :width], gy[:, :width]
        w = 1 + 0.1 * n(width, dtype=f)
        out = place()
        y, s = kda.layer_norm_fwd(x, w, w, residual=r, y=out[:, t, :width])
        y0, s0 = kda.layer_norm_fwd(x.contiguous(), w, w, residual=r.contiguous())
        same(y, y0), same(s, s0)
        assert bool((out[:, t, width:] == 5).all())
        alone(out)
        got = kda.layer_norm_bwd(x, gx, w, w, grad_residual=r, grad_dtype=torch.bfloat16, out=dict(dx=place()[:, t, :width]))
        want = kda.layer_norm_bwd(x.contiguous(), gx.contiguous(), w, w, grad_residual=r.contiguous(), grad_dtype=torch.bfloat16)
        for k, v in want.items():
            same(got[k], v)


@pytest.mark.parametrize("dim,stride", [(100, (1 << 26) - 1), (2048, (1 << 26) - 1), (4096, 1 << 27)])
def test_norm_of_rows_far_apart(kda, dim, stride):
    """At the limit of its strides, over more rows than a workgroup has: the same bits as dense rows."""
    import torch
    rows = 21
    g = torch.Generator("cuda").manual_seed(2)
    wide = torch.empty(rows, stride, dtype=torch.bfloat16, device="cuda")
    x, y = wide[:, :dim], wide[:, 5000:5000 + dim]
    x.copy_(torch.randn(rows, dim, generator=g, device="cuda"))
    gy, w = torch.randn(rows, dim, generator=g, device="cuda"), torch.randn(dim, generator=g, device="cuda")
    kda.layer_norm_fwd(x, w, y=y)
    assert torch.equal(y, kda.layer_norm_fwd(x.contiguous(), w))
    got, want = (kda.layer_norm_bwd(v, gy, w, w, grad_dtype=torch.bfloat16, out=o) for v, o in ((x, dict(dx=y)), (x.contiguous(), None)))
    assert all(torch.equal(got[k], want[k]) for k in want)
