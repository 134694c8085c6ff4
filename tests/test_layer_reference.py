"""The layer operators' 64-bit references themselves: gradients against central differences of the forward
definitions, closed forms, and mistakes planted in the references, which the error bounds have to find (CPU)."""
import numpy as np
import pytest

import layer_testlib as ref


def scan_case(seed, offsets, dim=3, ds=4, gate=True, softplus=True):
    r = np.random.default_rng(seed)
    rows = offsets[-1]
    return dict(u=r.normal(size=(rows, dim)), dt=r.normal(size=(rows, dim)), A=-np.exp(r.normal(size=(dim, ds))),
                B=r.normal(size=(rows, ds)), C=r.normal(size=(rows, ds)), D=r.normal(size=dim),
                z=r.normal(size=(rows, dim)) if gate else None, dt_bias=r.normal(size=dim),
                h0=r.normal(size=(len(offsets) - 1, dim, ds)), softplus=softplus)


def differences(f, x, eps=1e-6):
    """Central differences of the number f() in every entry of x, which f reads."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + eps
        up = f()
        x[i] = keep - eps
        g[i] = (up - f()) / (2 * eps)
        x[i] = keep
    return g


@pytest.mark.parametrize("gate,softplus", [(True, True), (False, True), (True, False)])
def test_scan_gradients_against_differences(gate, softplus):
    offsets = [0, 3, 3, 4, 9]
    x = scan_case(1, offsets, gate=gate, softplus=softplus)
    if not softplus:
        x["dt"] = 0.3 * np.abs(x["dt"])
        x["dt_bias"] = np.abs(x["dt_bias"])
    r = np.random.default_rng(2)
    gy, gf = r.normal(size=x["u"].shape), r.normal(size=x["h0"].shape)

    def loss():
        f = ref.scan_forward(x, offsets)
        return (f["y"] * gy).sum() + (f["final"] * gf).sum()

    got = ref.scan_backward(x, offsets, gy, gf)
    for name, of in (("du", "u"), ("ddt", "dt"), ("dA", "A"), ("dB", "B"), ("dC", "C"), ("dD", "D"), ("dz", "z"),
                     ("ddt_bias", "dt_bias"), ("dh0", "h0")):
        if x[of] is None:
            assert got[name] is None
            continue
        want = differences(loss, x[of])
        # the differences' error: second order in 1e-6, and 1e-16 of the loss over 2e-6
        assert np.abs(got[name] - want).max() <= 1e-7 * (1 + np.abs(want).max()), name


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("silu", [True, False])
def test_conv_gradients_against_differences(W, silu):
    offsets, dim = [0, 1, 1, 6, 8], 2
    r = np.random.default_rng(W)
    x, w, b = r.normal(size=(8, dim)), r.normal(size=(dim, W)), r.normal(size=dim)
    h0 = r.normal(size=(4, W - 1, dim))
    gy, gf = r.normal(size=x.shape), r.normal(size=h0.shape)

    def loss():
        y, final, _ = ref.conv_forward(x, w, b, h0, offsets, silu)
        return (y * gy).sum() + (final * gf).sum()

    got = ref.conv_backward(x, w, b, h0, offsets, silu, gy, gf)
    for name, of in (("dx", x), ("dweight", w), ("dbias", b), ("dh0", h0)):
        assert np.abs(got[name] - differences(loss, of)).max() <= 1e-7, name


def test_norm_gradients_against_differences():
    r = np.random.default_rng(3)
    x, w, b, gy = r.normal(size=(4, 7)) + 2, r.normal(size=7), r.normal(size=7), r.normal(size=(4, 7))
    got = ref.norm_backward(x, w, gy, 1e-5)
    loss = lambda: (ref.norm_forward(x, w, b, 1e-5)[0] * gy).sum()  # noqa: E731
    for name, of in (("dx", x), ("dweight", w), ("dbias", b)):
        assert np.abs(got[name] - differences(loss, of)).max() <= 1e-7, name


def test_scan_closed_form():
    """Constant step, one state, unit inputs: a geometric series."""
    rows, d, a = 12, 0.25, np.exp(-0.25)
    x = dict(u=np.ones((rows, 1)), dt=np.full((rows, 1), d), A=-np.ones((1, 1)), B=np.ones((rows, 1)),
             C=np.ones((rows, 1)), D=None, z=None, dt_bias=None, h0=None, softplus=False)
    t = np.arange(1, rows + 1)
    assert np.allclose(ref.scan_forward(x, [0, rows])["y"][:, 0], d * (1 - a ** t) / (1 - a), rtol=1e-13)


@pytest.mark.parametrize("mistake", ["token", "boundary", "decay", "gate"])
def test_planted_scan_mistakes_break_the_bound(mistake):
    offsets = [0, 40, 77]
    x = scan_case(5, offsets, dim=6, ds=4)
    good = ref.scan_forward(x, offsets)
    wrong, cut = {k: np.array(v) if isinstance(v, np.ndarray) else v for k, v in x.items()}, offsets
    if mistake == "token":
        wrong["B"][[50, 51]] = wrong["B"][[51, 50]]
    elif mistake == "boundary":
        cut = [0, 41, 77]
    elif mistake == "decay":
        wrong["A"] = wrong["A"] * 1.01
    else:
        wrong["z"] = wrong["z"] * 1.01
    scale = ref.scan_forward(x, offsets, absolute=True)["y"]
    n = ref.scan_roundings(x, offsets)
    ref.check("unharmed", good["y"], good["y"], scale, n, "bf16")
    with pytest.raises(AssertionError, match="times"):
        ref.check(mistake, ref.scan_forward(wrong, cut)["y"], good["y"], scale, n)


@pytest.mark.parametrize("mistake", ["tap", "state", "slope"])
def test_planted_conv_mistakes_break_the_bound(mistake):
    r = np.random.default_rng(7)
    offsets, dim, W = [0, 20, 33], 5, 4
    x, w, b, h0 = r.normal(size=(33, dim)), r.normal(size=(dim, W)), r.normal(size=dim), r.normal(size=(2, W - 1, dim))
    gy = r.normal(size=x.shape)
    args = (offsets, True, gy)
    good, scale = ref.conv_backward(x, w, b, h0, *args), ref.conv_backward(x, w, b, h0, *args, absolute=True)
    if mistake == "tap":
        bad = ref.conv_backward(x, w[:, ::-1], b, h0, *args)
    elif mistake == "state":
        bad = ref.conv_backward(x, w, b, None, *args)
    else:
        bad = ref.conv_backward(x, w, b, h0, offsets, False, gy)
    with pytest.raises(AssertionError, match="times"):
        ref.check(mistake, bad["dx"], good["dx"], scale["dx"], 64, "bf16")
