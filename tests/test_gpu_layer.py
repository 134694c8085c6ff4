"""The layer operators (selective scan, short convolution, layer norm) against their 64-bit references: types,
odd sizes, strides, packed sequences with empty and one-token members, single tokens, gradients, rows behind the last
sequence, states in place, other streams, graphs, and a run of all of them as a layer uses them."""
import numpy as np
import pytest

import layer_testlib as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_delta_rule_52_amd as m
    from gated_delta_rule_52_amd import _lib
    _lib.load()
    return m


def tdtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def rounded(a, dtype):
    """The values of a in the dtype, as float64."""
    import torch
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(tdtype(dtype)).double().numpy()


def dev(a, dtype="fp32", shape=None, sliced=False):
    """a on the device; sliced: as columns of a wider buffer whose other columns are NaN, not 16-byte aligned."""
    import torch
    if a is None:
        return None
    t = torch.from_numpy(np.asarray(a, dtype=np.float32)).to(tdtype(dtype))
    t = t if shape is None else t.reshape(shape)
    if sliced:
        wide = torch.full((*t.shape[:-1], t.shape[-1] + 5), float("nan"), dtype=t.dtype)
        wide[..., 3:-2] = t
        return wide.cuda()[..., 3:-2]
    return t.cuda()


def host(t):
    return None if t is None else t.double().cpu().numpy()


def layout(case):
    """(offsets, batch, tokens, cu or None) of a case's sequences: an int pair (B, T) or a list of lengths."""
    import torch
    if isinstance(case, tuple):
        B, T = case
        return [b * T for b in range(B + 1)], B, T, None
    offsets = np.concatenate([[0], np.cumsum(case)]).tolist()
    return offsets, 1, offsets[-1], torch.tensor(offsets, dtype=torch.int32, device="cuda")


def scan_inputs(seed, offsets, rows, dim, ds, dtype, gate=True, params=True, state=True, step=0.05, positive=False):
    r = np.random.default_rng(seed)
    n = lambda *s: r.normal(size=s)  # noqa: E731
    x = dict(u=rounded(n(rows, dim), dtype), dt=rounded(0.5 * n(rows, dim), dtype), B=rounded(n(rows, ds), dtype),
             C=rounded(n(rows, ds), dtype), z=rounded(n(rows, dim), dtype) if gate else None,
             A=rounded(-np.arange(1, ds + 1) * np.exp(0.1 * n(dim, ds)), "fp32"), D=None, dt_bias=None, h0=None,
             softplus=True)
    if params:
        x["D"] = rounded(1 + 0.1 * n(dim), "fp32")
        x["dt_bias"] = rounded(np.log(np.expm1(step * np.exp(n(dim)))), "fp32")
    if state:
        x["h0"] = rounded(0.5 * n(len(offsets) - 1, dim, ds), "fp32")
    if positive:
        x["softplus"], x["dt"] = False, rounded(0.05 * np.abs(n(rows, dim)), dtype)
        x["dt_bias"] = None
    return x


def scan_device(x, B, T, dtype, sliced=False):
    s = {k: dev(x[k], dtype, (B, T, -1), sliced) for k in ("u", "dt", "B", "C", "z")}
    s.update({k: dev(x[k]) for k in ("A", "D", "dt_bias")})
    return s


SCAN = [  # sequences, dim, ds, input, output, extras
    ((1, 1), 1, 1, "fp32", "fp32", {}),
    ((2, 17), 5, 4, "fp32", "fp32", {}),
    ((3, 16), 64, 16, "bf16", "bf16", {}),
    ((1, 300), 70, 16, "bf16", "fp32", dict(sliced=True)),
    ((2, 33), 130, 12, "fp32", "bf16", dict(sliced=True, gate=False)),
    ((1, 50), 64, 17, "fp32", "fp32", dict(state=False)),
    ((1, 40), 33, 32, "bf16", "fp32", dict(params=False)),
    ((1, 37), 20, 40, "fp32", "fp32", {}),
    ((2, 31), 65, 64, "bf16", "fp32", {}),
    ([5, 0, 1, 64, 0, 33, 2], 66, 16, "fp32", "fp32", {}),
    ([0, 0, 100, 15, 16, 17, 0], 128, 16, "bf16", "bf16", dict(sliced=True)),
    ([1], 64, 16, "fp32", "fp32", {}),
    ([1] * 40, 10, 8, "fp32", "fp32", {}),
    ([700, 3, 1200], 24, 16, "fp32", "fp32", {}),
    ((2, 1500), 40, 16, "fp32", "fp32", dict(step=0.01)),
    ((1, 90), 16, 16, "fp32", "fp32", dict(positive=True)),
]


@pytest.mark.parametrize("seqs,dim,ds,dtype,out,extra", SCAN)
def test_scan_forward(kda, seqs, dim, ds, dtype, out, extra):
    print(f"case scan forward: {seqs} dim={dim} ds={ds} {dtype}->{out} {extra}", flush=True)
    import torch
    extra = dict(extra)
    sliced = extra.pop("sliced", False)
    offsets, B, T, cu = layout(seqs)
    x = scan_inputs(1, offsets, offsets[-1], dim, ds, dtype, **extra)
    s = scan_device(x, B, T, dtype, sliced)
    y, final = kda.selective_scan_fwd(**s, initial_state=dev(x["h0"]), cu_seqlens=cu, dt_softplus=x["softplus"],
                                      out_dtype=tdtype(out))
    torch.cuda.synchronize()
    want, size = ref.scan_forward(x, offsets), ref.scan_forward(x, offsets, absolute=True)
    n = ref.scan_roundings(x, offsets)
    ref.check("y", host(y).reshape(-1, dim), want["y"], size["y"], n, out)
    ref.check("state", host(final), want["final"], size["final"], n)


@pytest.mark.parametrize("seqs,dim,ds,dtype,out,extra", SCAN)
def test_scan_gradients(kda, seqs, dim, ds, dtype, out, extra):
    print(f"case scan gradients: {seqs} dim={dim} ds={ds} {dtype}->{out} {extra}", flush=True)
    import torch
    extra = dict(extra)
    sliced = extra.pop("sliced", False)
    offsets, B, T, cu = layout(seqs)
    x = scan_inputs(2, offsets, offsets[-1], dim, ds, dtype, **extra)
    r = np.random.default_rng(3)
    gy = rounded(r.normal(size=x["u"].shape), dtype)
    gf = rounded(r.normal(size=(len(offsets) - 1, dim, ds)), "fp32") if x["h0"] is not None else None
    s = scan_device(x, B, T, dtype, sliced)
    got = kda.selective_scan_bwd(s.pop("u"), s.pop("dt"), s.pop("A"), s.pop("B"), s.pop("C"),
                                 dev(gy, dtype, (B, T, dim), sliced), **s, initial_state=dev(x["h0"]),
                                 grad_final_state=dev(gf), cu_seqlens=cu, dt_softplus=x["softplus"],
                                 grad_dtype=tdtype(out))
    torch.cuda.synchronize()
    want = ref.scan_backward(x, offsets, gy, gf)
    size = ref.scan_backward(x, offsets, gy, gf, absolute=True)
    n = 2 * ref.scan_roundings(x, offsets)
    for name in ("du", "ddt", "dz", "dB", "dC", "dA", "dD", "ddt_bias", "dh0"):
        if want[name] is None:
            assert got[name] is None
            continue
        token = name in ("du", "ddt", "dz", "dB", "dC")
        more = dim if name in ("dB", "dC") else offsets[-1] if name in ("dA", "dD", "ddt_bias") else 0
        ref.check(name, host(got[name]).reshape(want[name].shape), want[name], size[name], n + more,
                  out if token else "fp32")


@pytest.mark.parametrize("N,dim,ds,dtype", [(1, 1, 1, "fp32"), (3, 70, 16, "bf16"), (5, 33, 13, "fp32"), (2, 64, 32, "bf16"),
                                            (2, 9, 64, "fp32"), (4, 64, 8, "bf16")])
@pytest.mark.parametrize("gate", [True, False])
def test_scan_step(kda, N, dim, ds, dtype, gate):
    """Steps in place, against the reference and bit for bit against one-token prompts."""
    import torch
    print(f"case scan step: N={N} dim={dim} ds={ds} {dtype} gate={gate}", flush=True)
    offsets = list(range(N + 1))
    x = scan_inputs(4, offsets, N, dim, ds, dtype, gate=gate)
    s = {k: None if x[k] is None else dev(x[k], dtype, sliced=k == "B") for k in ("u", "dt", "B", "C", "z")}
    p = {k: dev(x[k]) for k in ("A", "D", "dt_bias")}
    state = dev(x["h0"])
    y = kda.selective_scan_step(s["u"], s["dt"], p["A"], s["B"], s["C"], state, p["D"], s["z"], p["dt_bias"],
                                dt_softplus=True, out_dtype=torch.float32)
    one = {k: None if v is None else v[:, None] for k, v in s.items()}
    y1, final = kda.selective_scan_fwd(one["u"], one["dt"], p["A"], one["B"], one["C"], p["D"], one["z"], p["dt_bias"],
                                       initial_state=dev(x["h0"]), dt_softplus=True, out_dtype=torch.float32)
    y2, none = kda.selective_scan_fwd(one["u"], one["dt"], p["A"], one["B"], one["C"], p["D"], one["z"], p["dt_bias"],
                                      initial_state=dev(x["h0"]), dt_softplus=True, out_dtype=torch.float32,
                                      output_final_state=False)
    torch.cuda.synchronize()
    assert torch.equal(y, y1[:, 0]) and torch.equal(state, final) and torch.equal(y2, y1) and none is None
    want, size = ref.scan_forward(x, offsets), ref.scan_forward(x, offsets, absolute=True)
    n = ref.scan_roundings(x, offsets)
    ref.check("y", host(y), want["y"], size["y"], n)
    ref.check("state", host(state), want["final"], size["final"], n)


def test_scan_large_steps_and_extreme_logits(kda):
    """Decays that underflow, steps of softplus far out on both sides, gates far out: finite and right."""
    import torch
    rows, dim, ds = 40, 8, 16
    x = scan_inputs(5, [0, rows], rows, dim, ds, "fp32")
    x["dt"] = np.linspace(-90, 90, rows)[:, None] + np.zeros((1, dim))
    x["z"] = np.linspace(80, -80, rows)[:, None] + np.zeros((1, dim))
    x["dt"], x["z"], x["dt_bias"] = rounded(x["dt"], "fp32"), rounded(x["z"], "fp32"), np.zeros(dim)
    s = scan_device(x, 1, rows, "fp32")
    y, final = kda.selective_scan_fwd(**s, initial_state=dev(x["h0"]), dt_softplus=True)
    want, size = ref.scan_forward(x, [0, rows]), ref.scan_forward(x, [0, rows], absolute=True)
    # the exponent's own roundings are relative to |delta A|, at most 104 where the decay is not yet zero
    n = (8 * 104 * 1.45 + 8) * rows
    ref.check("y", host(y)[0], want["y"], size["y"], n)
    ref.check("state", host(final), want["final"], size["final"], n)


def test_scan_rows_behind_the_last_sequence_and_between_nan(kda):
    """Offsets that start late and end early: the other rows' inputs are NaN, their outputs stay as they were; and a
    NaN of one sequence stays in it."""
    import torch
    dim, ds, rows = 70, 16, 90
    offsets = [7, 30, 30, 61, 77]
    x = scan_inputs(6, offsets, rows, dim, ds, "bf16")
    r = np.random.default_rng(7)
    gy = rounded(r.normal(size=(rows, dim)), "bf16")
    for k in ("u", "dt", "B", "C", "z"):
        x[k][:7] = np.nan
        x[k][77:] = np.nan
    gy[:7] = gy[77:] = np.nan
    clean = {k: np.nan_to_num(v) if isinstance(v, np.ndarray) else v for k, v in x.items()}
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    s = scan_device(x, 1, rows, "bf16")
    y = torch.full((1, rows, dim), 5.0, device="cuda")
    _, final = kda.selective_scan_fwd(**s, initial_state=dev(x["h0"]), cu_seqlens=cu, dt_softplus=True, y=y)
    want, size = ref.scan_forward(clean, offsets), ref.scan_forward(clean, offsets, absolute=True)
    n = ref.scan_roundings(clean, offsets)
    assert bool((y[0, :7] == 5).all()) and bool((y[0, 77:] == 5).all())
    ref.check("y", host(y)[0, 7:77], want["y"][7:77], size["y"][7:77], n)
    ref.check("state", host(final), want["final"], size["final"], n)

    out = {k: torch.full((1, rows, ds if k in ("dB", "dC") else dim), 5.0, device="cuda")
           for k in ("du", "ddt", "dB", "dC", "dz")}
    a = dict(s)
    got = kda.selective_scan_bwd(a.pop("u"), a.pop("dt"), a.pop("A"), a.pop("B"), a.pop("C"), dev(gy, "bf16", (1, rows, dim)),
                                 **a, initial_state=dev(x["h0"]), cu_seqlens=cu, dt_softplus=True, out=out)
    gclean = np.nan_to_num(gy)
    want, size = ref.scan_backward(clean, offsets, gclean), ref.scan_backward(clean, offsets, gclean, absolute=True)
    for k in ("du", "ddt", "dB", "dC", "dz"):
        assert bool((got[k][0, :7] == 5).all()) and bool((got[k][0, 77:] == 5).all()), k
        ref.check(k, host(got[k])[0, 7:77], want[k][7:77], size[k][7:77], 2 * n + dim)
    for k in ("dA", "dD", "ddt_bias", "dh0"):
        ref.check(k, host(got[k]), want[k], size[k], 2 * n + rows)

    s["u"][0, 40] = float("nan")  # inside the third sequence
    y2, final2 = kda.selective_scan_fwd(**s, initial_state=dev(x["h0"]), cu_seqlens=cu, dt_softplus=True,
                                        out_dtype=torch.float32)
    assert torch.equal(y2[0, 7:40], y[0, 7:40]) and torch.equal(y2[0, 61:77], y[0, 61:77])
    assert torch.equal(final2[[0, 1, 3]], final[[0, 1, 3]]) and bool(final2[2].isnan().all())


def test_scan_wrong_offsets_stay_inside(kda):
    """Offsets outside the rows or falling are a broken precondition: unspecified numbers, no access outside."""
    import torch
    x = scan_inputs(8, [0, 20], 20, 16, 16, "fp32")
    s = scan_device(x, 1, 20, "fp32")
    for cu in ([0, 1 << 30], [-5, 20], [20, 3, 50], [9, 9, 2]):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        kda.selective_scan_fwd(**s, cu_seqlens=c, dt_softplus=True)
        a = dict(s)
        kda.selective_scan_bwd(a.pop("u"), a.pop("dt"), a.pop("A"), a.pop("B"), a.pop("C"), s["u"], **a, cu_seqlens=c,
                               dt_softplus=True)
        kda.short_conv_fwd(s["u"], s["A"][:, :4].contiguous(), cu_seqlens=c)
        kda.short_conv_bwd(s["u"], s["A"][:, :4].contiguous(), s["u"], cu_seqlens=c)
    torch.cuda.synchronize()


@pytest.mark.parametrize("seqs", [(2, 100), (1, 2100), [40, 0, 700, 3, 900]])
def test_states_in_place(kda, seqs):
    """The final state in the initial one's memory, and the initial-state gradient in either state's: the same bits
    as with memory of their own."""
    import torch
    offsets, B, T, cu = layout(seqs)
    dim, ds, W = 48, 16, 4
    x = scan_inputs(9, offsets, offsets[-1], dim, ds, "bf16")
    s = scan_device(x, B, T, "bf16")
    kw = dict(cu_seqlens=cu, dt_softplus=True)
    y, final = kda.selective_scan_fwd(**s, initial_state=dev(x["h0"]), **kw)
    state = dev(x["h0"])
    y1, _ = kda.selective_scan_fwd(**s, initial_state=state, final_state=state, **kw)
    assert torch.equal(y, y1) and torch.equal(state, final)
    a = dict(s)
    args = [a.pop(k) for k in ("u", "dt", "A", "B", "C")] + [s["u"]]
    gf = dev(np.random.default_rng(1).normal(size=x["h0"].shape))
    want = kda.selective_scan_bwd(*args, **a, initial_state=dev(x["h0"]), grad_final_state=gf.clone(), **kw)
    state = dev(x["h0"])
    got = kda.selective_scan_bwd(*args, **a, initial_state=state, grad_final_state=gf.clone(), grad_initial_state=state, **kw)
    assert all(torch.equal(got[k], want[k]) for k in want if want[k] is not None)
    g2 = gf.clone()
    got = kda.selective_scan_bwd(*args, **a, initial_state=dev(x["h0"]), grad_final_state=g2, grad_initial_state=g2, **kw)
    assert all(torch.equal(got[k], want[k]) for k in want if want[k] is not None)

    w = dev(np.random.default_rng(2).normal(size=(dim, W)))
    h0 = dev(np.random.default_rng(3).normal(size=(len(offsets) - 1, W - 1, dim)), "bf16")
    y, final = kda.short_conv_fwd(s["u"], w, initial_state=h0.clone(), cu_seqlens=cu, silu=True)
    state = h0.clone()
    y1, _ = kda.short_conv_fwd(s["u"], w, initial_state=state, final_state=state, cu_seqlens=cu, silu=True)
    assert torch.equal(y, y1) and torch.equal(state, final)
    g = dev(np.random.default_rng(4).normal(size=h0.shape))
    want = kda.short_conv_bwd(s["u"], w, s["u"], initial_state=h0, grad_final_state=g.clone(), cu_seqlens=cu, silu=True)
    got = kda.short_conv_bwd(s["u"], w, s["u"], initial_state=h0, grad_final_state=g, grad_initial_state=g, cu_seqlens=cu,
                             silu=True)
    assert all(torch.equal(got[k], want[k]) for k in want if want[k] is not None)


# ---- convolution ---------------------------------------------------------------------------------------

CONV = [  # sequences, dim, W, input, output, weights, extras
    ((1, 1), 1, 2, "fp32", "fp32", "fp32", {}),
    ((2, 3), 7, 4, "fp32", "fp32", "fp32", {}),
    ((3, 70), 64, 4, "bf16", "bf16", "bf16", {}),
    ((1, 200), 36, 3, "bf16", "fp32", "fp32", dict(sliced=True)),
    ((2, 65), 1030, 4, "fp32", "bf16", "fp32", dict(silu=False)),
    ((1, 64), 8, 2, "fp32", "fp32", "bf16", dict(bias=False, state=False)),
    ([5, 0, 1, 2, 64, 0, 33, 3], 260, 4, "bf16", "fp32", "fp32", {}),
    ([0, 1, 1, 1, 0, 130], 12, 4, "fp32", "fp32", "fp32", dict(sliced=True)),
    ([1] * 50, 16, 3, "fp32", "fp32", "fp32", {}),
]


def conv_case(seed, offsets, dim, W, dtype, wdtype, silu=True, bias=True, state=True):
    r = np.random.default_rng(seed)
    x = rounded(r.normal(size=(offsets[-1], dim)), dtype)
    w = rounded(r.normal(size=(dim, W)) / W ** 0.5, wdtype)
    b = rounded(0.1 * r.normal(size=dim), wdtype) if bias else None
    h0 = rounded(r.normal(size=(len(offsets) - 1, W - 1, dim)), dtype) if state else None
    return x, w, b, h0, silu


@pytest.mark.parametrize("seqs,dim,W,dtype,out,wdtype,extra", CONV)
def test_conv_forward(kda, seqs, dim, W, dtype, out, wdtype, extra):
    print(f"case conv forward: {seqs} dim={dim} W={W} {dtype}->{out} {extra}", flush=True)
    extra = dict(extra)
    sliced = extra.pop("sliced", False)
    offsets, B, T, cu = layout(seqs)
    x, w, b, h0, silu = conv_case(1, offsets, dim, W, dtype, wdtype, **extra)
    y, final = kda.short_conv_fwd(dev(x, dtype, (B, T, dim), sliced), dev(w, wdtype), dev(b, wdtype),
                                  initial_state=dev(h0, dtype), cu_seqlens=cu, silu=silu, out_dtype=tdtype(out))
    want, wfinal, _ = ref.conv_forward(x, w, b, h0, offsets, silu)
    size = ref.conv_forward(x, w, b, h0, offsets, silu, absolute=True)[0]
    # W + 1 roundings of p; with silu its slope is at most 1.1, and the sigmoid's 6 act on |y| <= |p|
    ref.check("y", host(y).reshape(-1, dim), want, size, 16, out)
    assert np.array_equal(host(final), wfinal)


@pytest.mark.parametrize("seqs,dim,W,dtype,out,wdtype,extra", CONV)
def test_conv_gradients(kda, seqs, dim, W, dtype, out, wdtype, extra):
    print(f"case conv gradients: {seqs} dim={dim} W={W} {dtype}->{out} {extra}", flush=True)
    extra = dict(extra)
    sliced = extra.pop("sliced", False)
    offsets, B, T, cu = layout(seqs)
    x, w, b, h0, silu = conv_case(2, offsets, dim, W, dtype, wdtype, **extra)
    r = np.random.default_rng(5)
    gy = rounded(r.normal(size=x.shape), dtype)
    gf = rounded(r.normal(size=(len(offsets) - 1, W - 1, dim)), "fp32")
    got = kda.short_conv_bwd(dev(x, dtype, (B, T, dim), sliced), dev(w, wdtype), dev(gy, dtype, (B, T, dim), sliced),
                             dev(b, wdtype), initial_state=dev(h0, dtype), grad_final_state=dev(gf), cu_seqlens=cu,
                             silu=silu, grad_dtype=tdtype(out))
    want = ref.conv_backward(x, w, b, h0, offsets, silu, gy, gf)
    size = ref.conv_backward(x, w, b, h0, offsets, silu, gy, gf, absolute=True)
    for name in ("dx", "dweight", "dbias", "dh0"):
        if want[name] is None:
            assert got[name] is None
            continue
        ref.check(name, host(got[name]).reshape(want[name].shape), want[name], size[name],
                  32 + (offsets[-1] if name in ("dweight", "dbias") else 0), out if name == "dx" else "fp32")


@pytest.mark.parametrize("N,dim,W,dtype", [(1, 1, 2, "fp32"), (3, 70, 4, "bf16"), (5, 64, 3, "fp32"), (2, 2052, 4, "bf16")])
def test_conv_step(kda, N, dim, W, dtype):
    import torch
    print(f"case conv step: N={N} dim={dim} W={W} {dtype}", flush=True)
    offsets = list(range(N + 1))
    x, w, b, h0, silu = conv_case(6, offsets, dim, W, dtype, "fp32")
    state = dev(h0, dtype)
    y = kda.short_conv_step(dev(x, dtype, sliced=True), dev(w), state, dev(b), silu=True, out_dtype=torch.float32)
    y1, final = kda.short_conv_fwd(dev(x, dtype)[:, None], dev(w), dev(b), initial_state=dev(h0, dtype), silu=True,
                                   out_dtype=torch.float32)
    assert torch.equal(y, y1[:, 0]) and torch.equal(state, final)
    want, wfinal, _ = ref.conv_forward(x, w, b, h0, offsets, True)
    ref.check("y", host(y), want, ref.conv_forward(x, w, b, h0, offsets, True, absolute=True)[0], 16)
    assert np.array_equal(host(state), wfinal)


def test_conv_rows_behind_the_last_sequence(kda):
    import torch
    dim, rows, offsets = 36, 150, [5, 40, 41, 41, 118]
    x, w, b, h0, silu = conv_case(7, offsets[:-1] + [rows], dim, 4, "bf16", "fp32")
    gy = rounded(np.random.default_rng(8).normal(size=x.shape), "bf16")
    for a in (x, gy):
        a[:5] = a[118:] = np.nan
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    y = torch.full((1, rows, dim), 5.0, device="cuda")
    dx = torch.full((1, rows, dim), 5.0, device="cuda")
    args = dev(x, "bf16", (1, rows, dim)), dev(w)
    _, final = kda.short_conv_fwd(*args, dev(b), initial_state=dev(h0, "bf16"), cu_seqlens=cu, silu=True, y=y)
    got = kda.short_conv_bwd(*args, dev(gy, "bf16", (1, rows, dim)), dev(b), initial_state=dev(h0, "bf16"), cu_seqlens=cu,
                             silu=True, out=dict(dx=dx))
    want, wfinal, _ = ref.conv_forward(x, w, b, h0, offsets, True)
    for t in (y, dx):
        assert bool((t[0, :5] == 5).all()) and bool((t[0, 118:] == 5).all())
    ref.check("y", host(y)[0, 5:118], want[5:118], ref.conv_forward(x, w, b, h0, offsets, True, True)[0][5:118], 16)
    assert np.array_equal(host(final), wfinal)
    want = ref.conv_backward(x, w, b, h0, offsets, True, gy)
    size = ref.conv_backward(x, w, b, h0, offsets, True, gy, absolute=True)
    ref.check("dx", host(dx)[0, 5:118], want["dx"][5:118], size["dx"][5:118], 32)
    for k in ("dweight", "dbias", "dh0"):
        ref.check(k, host(got[k]), want[k], size[k], 32 + rows)


# ---- layer norm ----------------------------------------------------------------------------------------

NORM = [  # rows, dim, x, residual or None, weights or None, output
    (1, 1, "fp32", None, "fp32", "fp32"), (5, 7, "fp32", "fp32", "fp32", "fp32"), (33, 128, "bf16", None, "fp32", "bf16"),
    (17, 100, "bf16", "fp32", "bf16", "fp32"), (9, 129, "fp32", None, None, "fp32"), (40, 256, "bf16", "bf16", "bf16", "bf16"),
    (6, 500, "fp32", "fp32", "fp32", "bf16"), (5, 512, "bf16", None, "fp32", "fp32"), (7, 1001, "bf16", "fp32", "fp32", "bf16"),
    (3, 1024, "fp32", None, "bf16", "fp32"), (6, 2048, "bf16", "fp32", "fp32", "bf16"), (3, 2049, "fp32", None, "fp32", "fp32"),
    (4, 4096, "bf16", "fp32", "fp32", "bf16"), (3, 5001, "fp32", "fp32", "fp32", "fp32"), (2, 8192, "bf16", None, "fp32", "fp32"),
    (3, 8193, "fp32", None, "fp32", "fp32"), (2, 16384, "bf16", "bf16", "bf16", "bf16"), (2500, 64, "bf16", None, "fp32", "fp32"),
    # several rounds of rows for every workgroup, the last one partly filled
    (40011, 24, "fp32", None, "fp32", "fp32"), (5003, 600, "bf16", "fp32", "fp32", "bf16"), (777, 5000, "bf16", None, "fp32", "fp32"),
    (600, 9000, "fp32", None, "fp32", "fp32"), (9001, 200, "bf16", "fp32", "bf16", "bf16"), (4501, 509, "fp32", "bf16", "fp32", "fp32"),
    (2503, 1500, "bf16", None, "fp32", "fp32"), (1101, 4001, "fp32", "bf16", "fp32", "bf16"),
    # around the smallest row that is read in whole units
    (37, 8, "bf16", "fp32", "fp32", "fp32"), (37, 9, "fp32", "bf16", "bf16", "fp32"), (20000, 6, "bf16", "fp32", "fp32", "bf16"),
]
# roundings behind a sum over a row: a lane's 64 at most, the lanes' 6 steps and the waves' 16, and a dozen around them
ROW = 100


@pytest.mark.parametrize("rows,dim,dtype,rdtype,wdtype,out", NORM)
@pytest.mark.parametrize("sliced", [False, True])
def test_norm_forward(kda, rows, dim, dtype, rdtype, wdtype, out, sliced):
    print(f"case norm forward: {rows} x {dim} {dtype} residual={rdtype} weight={wdtype}->{out} sliced={sliced}", flush=True)
    r = np.random.default_rng(dim)
    x = rounded(r.normal(size=(rows, dim)) + 0.5, dtype)
    res = rounded(3 * r.normal(size=(rows, dim)), rdtype) if rdtype else None
    w, b = (rounded(1 + 0.2 * r.normal(size=dim), wdtype), rounded(0.2 * r.normal(size=dim), wdtype)) if wdtype else (None, None)
    got = kda.layer_norm_fwd(dev(x, dtype, None, sliced), dev(w, wdtype or "fp32"), dev(b, wdtype or "fp32"),
                             residual=dev(res, rdtype or "fp32", None, sliced), out_dtype=tdtype(out))
    s = x if res is None else x + res
    y = got if res is None else got[0]
    ref.check("y", host(y), ref.norm_forward(s, w, b, 1e-5)[0], ref.norm_scales(s, w, b, None, 1e-5)["y"], ROW, out)
    if res is not None:
        ref.check("residual", host(got[1]), s, np.abs(s), 1, rdtype)


@pytest.mark.parametrize("rows,dim,dtype,rdtype,wdtype,out", NORM)
@pytest.mark.parametrize("sliced", [False, True])
def test_norm_gradients(kda, rows, dim, dtype, rdtype, wdtype, out, sliced):
    print(f"case norm gradients: {rows} x {dim} {dtype} residual={rdtype} weight={wdtype}->{out} sliced={sliced}", flush=True)
    r = np.random.default_rng(dim + 1)
    x = rounded(2 * r.normal(size=(rows, dim)) + 0.5, rdtype or dtype)
    gy = rounded(r.normal(size=(rows, dim)), dtype)
    res = rounded(r.normal(size=(rows, dim)), rdtype) if rdtype else None
    w, b = (rounded(1 + 0.2 * r.normal(size=dim), wdtype), rounded(0.2 * r.normal(size=dim), wdtype)) if wdtype else (None, None)
    got = kda.layer_norm_bwd(dev(x, rdtype or dtype, None, sliced), dev(gy, dtype, None, sliced), dev(w, wdtype or "fp32"),
                             dev(b, wdtype or "fp32"), grad_residual=dev(res, rdtype or "fp32"), grad_dtype=tdtype(out))
    want, size = ref.norm_backward(x, w, gy, 1e-5, res), ref.norm_scales(x, w, b, gy, 1e-5, res)
    ref.check("dx", host(got["dx"]), want["dx"], size["dx"], ROW, out)
    if wdtype:
        for k in ("dweight", "dbias"):
            ref.check(k, host(got[k]), want[k], size[k], ROW + rows)
    else:
        assert got["dweight"] is None and got["dbias"] is None


@pytest.mark.parametrize("dim", [64, 777, 5001])
def test_norm_of_a_denormal_variance(kda, dim):
    """eps = 0 and values of 2^-64: a variance near 2^-128.  Its summands and its own rounding are on the grid of
    2^-149, off by 2^-150 each, which is 2^-22 of it: 4 roundings of 2^-24 twice over, of which the root takes half;
    the gradient has the root three times."""
    x = rounded(np.random.default_rng(dim).normal(size=(5, dim)), "fp32") * 2.0 ** -64
    y = kda.layer_norm_fwd(dev(x), eps=0.0)
    want = ref.norm_forward(x, None, None, 0.0)[0]
    ref.check("y", host(y), want, ref.norm_scales(x, None, None, None, 0.0)["y"], ROW + 8)
    gy = rounded(np.random.default_rng(1).normal(size=(5, dim)), "fp32") * 2.0 ** -64
    got = kda.layer_norm_bwd(dev(x), dev(gy), eps=0.0)
    ref.check("dx", host(got["dx"]), ref.norm_backward(x, None, gy, 0.0)["dx"],
              ref.norm_scales(x, None, None, gy, 0.0)["dx"], ROW + 24)


def test_norm_of_heads_and_far_means(kda):
    """The recurrence's output [B,T,H,dv] row by row, and rows whose mean is far above their spread."""
    import torch
    r = np.random.default_rng(1)
    x = rounded(r.normal(size=(2, 5, 3, 128)), "bf16")
    y = kda.layer_norm_fwd(dev(x, "bf16"), out_dtype=torch.float32)
    assert y.shape == (2, 5, 3, 128)
    ref.check("heads", host(y), ref.norm_forward(x, None, None, 1e-5)[0], ref.norm_scales(x, None, None, None, 1e-5)["y"], ROW)
    far = rounded(1000 + r.normal(size=(6, 777)), "fp32")
    y = kda.layer_norm_fwd(dev(far))
    ref.check("far", host(y), ref.norm_forward(far, None, None, 1e-5)[0], ref.norm_scales(far, None, None, None, 1e-5)["y"], ROW)
    far = rounded(1000 + r.normal(size=(6, 5001)), "fp32")  # a row over several waves
    y = kda.layer_norm_fwd(dev(far))
    ref.check("far, wide", host(y), ref.norm_forward(far, None, None, 1e-5)[0], ref.norm_scales(far, None, None, None, 1e-5)["y"], ROW)
    far[:, 0] = 1e4  # one element far from its wave's others
    y = kda.layer_norm_fwd(dev(far))
    ref.check("outlier", host(y), ref.norm_forward(far, None, None, 1e-5)[0], ref.norm_scales(far, None, None, None, 1e-5)["y"], ROW)
    flat = np.full((3, 64), 7.0)
    assert bool((kda.layer_norm_fwd(dev(flat)) == 0).all())
    # the residual in place
    a, b = dev(r.normal(size=(20, 300)), "bf16"), dev(r.normal(size=(20, 300)))
    y, s = kda.layer_norm_fwd(a, residual=b.clone())
    c = b.clone()
    y1, s1 = kda.layer_norm_fwd(a, residual=c, residual_out=c)
    assert s1 is c and torch.equal(y, y1) and torch.equal(s, c)


@pytest.mark.parametrize("rows,dim", [(33, 5), (33, 13), (7, 700), (5, 5001), (3, 9003)])
def test_norm_residual_in_place(kda, rows, dim):
    """The sums take every lane's inputs before one of them is replaced, also where units of a row overlap."""
    import torch
    g = torch.Generator("cuda").manual_seed(dim)
    x, res = (torch.randn(rows, dim, generator=g, device="cuda") for _ in range(2))
    y, s = kda.layer_norm_fwd(x, residual=res)
    assert torch.equal(s, x + res)
    for _ in range(3):
        held = res.clone()
        z, out = kda.layer_norm_fwd(x, residual=held, residual_out=held)
        assert out is held and torch.equal(held, s) and torch.equal(z, y)


def test_no_rows(kda):
    """No tokens: states pass through, parameter gradients are zero, nothing else is written."""
    import torch
    h0 = dev(np.random.default_rng(1).normal(size=(2, 6, 16)))
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    A = -torch.ones(6, 16, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    for lead, c in (((2, 0), None), ((1, 0), cu)):
        args = e(*lead, 6), e(*lead, 6), A, e(*lead, 16), e(*lead, 16)
        y, final = kda.selective_scan_fwd(*args, initial_state=h0, cu_seqlens=c)
        assert y.shape == (*lead, 6) and torch.equal(final, h0)
        g = kda.selective_scan_bwd(*args, e(*lead, 6), torch.ones(6, device="cuda"), grad_final_state=h0, cu_seqlens=c)
        assert torch.equal(g["dh0"], h0) and not g["dA"].any() and not g["dD"].any()
        hc = h0[:, :3, :8].contiguous()
        y, final = kda.short_conv_fwd(e(*lead, 8), torch.ones(8, 4, device="cuda"), initial_state=hc, cu_seqlens=c)
        assert torch.equal(final, hc)
        g = kda.short_conv_bwd(e(*lead, 8), torch.ones(8, 4, device="cuda"), e(*lead, 8), grad_final_state=hc, cu_seqlens=c)
        assert torch.equal(g["dh0"], hc) and not g["dweight"].any()
    w = torch.ones(8, device="cuda")
    assert kda.layer_norm_fwd(e(0, 8), w).shape == (0, 8)
    g = kda.layer_norm_bwd(e(0, 8), e(0, 8), w, w)
    assert not g["dweight"].any() and not g["dbias"].any()
    # no sequences: a batch of none, and packed rows that belong to no sequence (a single offset)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    for lead, c in (((0, 4), None), ((1, 5), one)):
        y = torch.full((*lead, 6), 5.0, device="cuda")
        args = e(*lead, 6), e(*lead, 6), A, e(*lead, 16), e(*lead, 16)
        _, final = kda.selective_scan_fwd(*args, cu_seqlens=c, y=y)
        assert final.shape == (0, 6, 16) and bool((y == 5).all())
        out = {k: torch.full((*lead, 16 if k in ("dB", "dC") else 6), 5.0, device="cuda") for k in ("du", "ddt", "dB", "dC")}
        none = kda.selective_scan_bwd(*args, y, cu_seqlens=c, out=out)
        assert not none["dA"].any() and all(bool((v == 5).all()) for v in out.values())
        x = e(*lead, 8)
        y = torch.full((*lead, 8), 5.0, device="cuda")
        kda.short_conv_fwd(x, torch.ones(8, 4, device="cuda"), cu_seqlens=c, y=y)
        dx = torch.full((*lead, 8), 5.0, device="cuda")
        none = kda.short_conv_bwd(x, torch.ones(8, 4, device="cuda"), x, cu_seqlens=c, out=dict(dx=dx))
        assert not none["dweight"].any() and bool((y == 5).all()) and bool((dx == 5).all())


def test_refusals(kda):
    import torch
    x = torch.zeros(2, 8, 16, device="cuda")
    A, n = -torch.ones(16, 4, device="cuda"), torch.zeros(2, 8, 4, device="cuda")
    bad = [lambda: kda.selective_scan_fwd(x.half(), x.half(), A, n.half(), n.half()),
           lambda: kda.selective_scan_fwd(x, x[:, :7], A, n, n),
           lambda: kda.selective_scan_fwd(x, x.bfloat16(), A, n, n),
           lambda: kda.selective_scan_fwd(x.cpu(), x, A, n, n),
           lambda: kda.selective_scan_fwd(x.transpose(1, 2), x, A, n, n),
           lambda: kda.selective_scan_fwd(x, x, A.double(), n, n),
           lambda: kda.selective_scan_fwd(torch.zeros(2, 16, 16, device="cuda")[:, ::2][:, :8].transpose(0, 1), x, A, n, n),
           lambda: kda.selective_scan_step(x[0], x[0], A, n[0], n[0], None),
           lambda: kda.selective_scan_step(x, x, A, n, n, None),
           lambda: kda.short_conv_fwd(x, A, initial_state=torch.zeros(2, 3, 16, dtype=torch.bfloat16, device="cuda")),
           lambda: kda.short_conv_fwd(x, A, cu_seqlens=torch.zeros(3, dtype=torch.int64, device="cuda")),
           lambda: kda.layer_norm_fwd(x, A[:, 0].bfloat16(), A[:, 0].contiguous()),
           lambda: kda.layer_norm_fwd(x, eps=1e-5, residual=x[:1]),
           # rows that repeat inside a batch whose sequences do not: no spacing fits, and none may be made up
           lambda: kda.short_conv_fwd(x[:, :1].expand(2, 8, 16), A),
           lambda: kda.layer_norm_bwd(x, x, grad_dtype=torch.float16)]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("not refused:", i)
    for f in (lambda: kda.selective_scan_fwd(x, x, -torch.ones(16, 65, device="cuda"), *[torch.zeros(2, 8, 65, device="cuda")] * 2),
              lambda: kda.selective_scan_fwd(x, x, A, n, n, y=x),
              lambda: kda.short_conv_fwd(x, torch.zeros(16, 5, device="cuda")),
              lambda: kda.short_conv_fwd(x[:1].expand(1, 8, 16), A, y=x[:1]),
              lambda: kda.short_conv_fwd(x[:, :1].expand(2, 8, 16)[:1], A),
              lambda: kda.layer_norm_fwd(x[0, 0].expand(4, 16)),
              lambda: kda.layer_norm_fwd(torch.zeros(1, 16385, device="cuda"))):
        with pytest.raises(kda.KdaError):
            f()


def test_sizes_past_32_bits_are_refused(kda):
    """One element seen 2^31 times: the argument structs hold sizes in 32 bits."""
    import torch
    one, many = torch.zeros(1, 1, 1, device="cuda"), 2 ** 31
    w, A = torch.ones(1, 4, device="cuda"), -torch.ones(1, 4, device="cuda")
    for x in (one.expand(1, many, 1), one.expand(many, 1, 1), one.expand(1, 1, many)):
        n = one.expand(*x.shape[:2], 4)
        for call in (lambda: kda.selective_scan_fwd(x, x, A, n, n), lambda: kda.selective_scan_bwd(x, x, A, n, n, x),
                     lambda: kda.short_conv_fwd(x, w), lambda: kda.short_conv_bwd(x, w, x),
                     lambda: kda.selective_scan_fwd_workspace_bytes(x, 4), lambda: kda.short_conv_bwd_workspace_bytes(x, 4)):
            with pytest.raises(ValueError):
                call()
    with pytest.raises(ValueError):
        kda.layer_norm_fwd(one.expand(1, 1, many))


def test_rows_past_32_bits(kda):
    """Rows whose offsets pass 2^32 elements, as slices of a very wide buffer: the same bits as a dense copy."""
    import torch
    rows, wide, dim, ds = 1100, 4_000_003, 24, 16
    r = np.random.default_rng(12)
    x = scan_inputs(13, [0, rows], rows, dim, ds, "bf16")
    dense = scan_device(x, 1, rows, "bf16")
    buffer = torch.empty(rows, wide, dtype=torch.bfloat16, device="cuda")
    far, at = {}, 5
    for k in ("u", "dt", "B", "C", "z"):
        n = dense[k].shape[-1]
        buffer[:, at:at + n] = dense[k][0]
        far[k] = buffer[:, at:at + n][None]
        at += n
    p = {k: dense[k] for k in ("A", "D", "dt_bias")}
    h0 = dev(x["h0"])
    y, final = kda.selective_scan_fwd(**dense, initial_state=h0, dt_softplus=True)
    y1, final1 = kda.selective_scan_fwd(**far, **p, initial_state=h0, dt_softplus=True, y=buffer[:, at:at + dim][None])
    assert torch.equal(y, y1) and torch.equal(final, final1)
    call = lambda s, out: kda.selective_scan_bwd(s["u"], s["dt"], p["A"], s["B"], s["C"], s["z"], p["D"], s["z"],  # noqa: E731
                                                 p["dt_bias"], dt_softplus=True, grad_dtype=torch.bfloat16, out=out)
    out = {k: buffer[:, at + i * 32:at + i * 32 + (ds if k in ("dB", "dC") else dim)][None]
           for i, k in enumerate(("du", "ddt", "dB", "dC", "dz"))}
    want, got = call(dense, None), call(far, out)
    assert all(torch.equal(want[k], got[k]) for k in want if want[k] is not None)
    w = dev(r.normal(size=(dim, 4)))
    y, s = kda.short_conv_fwd(dense["u"], w, silu=True)
    y1, s1 = kda.short_conv_fwd(far["u"], w, silu=True, y=buffer[:, at:at + dim][None])
    assert torch.equal(y, y1) and torch.equal(s, s1)
    want = kda.short_conv_bwd(dense["u"], w, dense["z"], silu=True, grad_dtype=torch.bfloat16)
    got = kda.short_conv_bwd(far["u"], w, far["z"], silu=True, grad_dtype=torch.bfloat16, out=dict(dx=buffer[:, at:at + dim][None]))
    assert all(torch.equal(want[k], got[k]) for k in want if want[k] is not None)
    wt = w[:, 0].contiguous()
    assert torch.equal(kda.layer_norm_fwd(dense["u"], wt), kda.layer_norm_fwd(far["u"], wt, y=buffer[:, at:at + dim][None]))
    want = kda.layer_norm_bwd(dense["u"], dense["z"], wt, wt)
    got = kda.layer_norm_bwd(far["u"], far["z"], wt, wt)
    assert all(torch.equal(want[k], got[k]) for k in want)


@pytest.mark.parametrize("B,T,dim,W,dtype", [(4, 4096, 4096, 4, "bf16"), (3, 5000, 2051, 3, "fp32")])
def test_conv_full_size(kda, B, T, dim, W, dtype):
    """Sizes at which each thread walks its longest tile, against the definition in 64 bits on the GPU."""
    import torch
    g = torch.Generator("cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, gy, w, b = n(B, T, dim).to(tdtype(dtype)), n(B, T, dim).to(tdtype(dtype)), n(dim, W) / W ** .5, .1 * n(dim)
    y, _ = kda.short_conv_fwd(x, w, b, silu=True, out_dtype=torch.float32)
    got = kda.short_conv_bwd(x, w, gy, b, silu=True)
    worst = 0.0
    for c in range(0, dim, 512):
        xs = torch.nn.functional.pad(x[:, :, c:c + 512].double(), (0, 0, W - 1, 0))
        ws, gs = w[c:c + 512].double(), gy[:, :, c:c + 512].double()
        p = sum(xs[:, j:j + T] * ws[:, j] for j in range(W)) + b[c:c + 512].double()
        size = sum((xs[:, j:j + T] * ws[:, j]).abs() for j in range(W)) + b[c:c + 512].double().abs()
        sg = torch.sigmoid(p)
        # 16 roundings of the absolute sum, as in the small cases
        worst = max(worst, float(((y[:, :, c:c + 512].double() - p * sg).abs() / (16 * 2 ** -24 * size)).max()))
        gp = gs * sg * (1 + p * (1 - sg))
        pad = torch.nn.functional.pad(gp, (0, 0, 0, W - 1))
        dx = sum(pad[:, W - 1 - j:W - 1 - j + T] * ws[:, j] for j in range(W))
        dw = torch.stack([(gp * xs[:, j:j + T]).sum((0, 1)) for j in range(W)], 1)
        near = lambda a, v: float((a.double() - v).norm() / v.norm())  # noqa: E731
        # norms: some 40 independent roundings of terms that a sum of W (dx) or of B T (dweight) keeps up with
        assert near(got["dx"][:, :, c:c + 512], dx) < 40 * 2 ** -24
        assert near(got["dweight"][c:c + 512], dw) < 200 * 2 ** -24 and near(got["dbias"][c:c + 512], gp.sum((0, 1))) < 200 * 2 ** -24
    assert worst <= 1, worst


@pytest.mark.parametrize("B,T,dim,ds", [(16, 300, 2048, 16), (2, 2000, 1024, 16), (12, 130, 2900, 20)])
def test_scan_full_size(kda, B, T, dim, ds):
    """Sizes that take whole sequences and long tiles, against a walk over the tokens in 64 bits on the GPU; the
    gradients against autograd through that walk, on a part of the channels."""
    import torch
    g = torch.Generator("cuda").manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    u, dt, z, gy = (n(B, T, dim).bfloat16() for _ in range(4))
    Bm, Cm, A, D = n(B, T, ds).bfloat16(), n(B, T, ds).bfloat16(), -torch.exp(n(dim, ds)), n(dim)
    bias, h0, gf = -3 + n(dim), n(B, dim, ds), n(B, dim, ds)
    y, final = kda.selective_scan_fwd(u, dt, A, Bm, Cm, D, z, bias, initial_state=h0, dt_softplus=True, out_dtype=torch.float32)
    got = kda.selective_scan_bwd(u, dt, A, Bm, Cm, gy, D, z, bias, initial_state=h0, grad_final_state=gf, dt_softplus=True)
    some = torch.cat([torch.arange(40), torch.arange(dim - 40, dim)]).cuda()
    leaf = lambda t: t.double().requires_grad_()  # noqa: E731
    L = dict(u=leaf(u[..., some]), dt=leaf(dt[..., some]), z=leaf(z[..., some]), A=leaf(A[some]), D=leaf(D[some]),
             b=leaf(bias[some]), h0=leaf(h0[:, some]))
    Bd, Cd = Bm.double(), Cm.double()
    delta = torch.logaddexp(L["dt"] + L["b"], torch.zeros((), dtype=torch.float64, device="cuda"))
    h, ys = L["h0"], []
    for t in range(T):
        h = torch.exp(delta[:, t, :, None] * L["A"]) * h + (delta[:, t] * L["u"][:, t])[..., None] * Bd[:, t, None]
        ys.append((h * Cd[:, t, None]).sum(-1))
    want = (torch.stack(ys, 1) + L["D"] * L["u"]) * L["z"] * torch.sigmoid(L["z"])
    ((want * gy[..., some].double()).sum() + (h * gf[:, some].double()).sum()).backward()
    near = lambda a, v: float((a.double() - v).norm() / v.norm())  # noqa: E731
    # roundings add up independently over a state's memory of at most T tokens: some sqrt(20 T) of them
    bound = 2 * (20 * T) ** .5 * 2 ** -24
    assert near(y[..., some], want.detach()) < bound and near(final[:, some], h.detach()) < bound
    for k, v in (("du", "u"), ("ddt", "dt"), ("dz", "z"), ("dh0", "h0")):
        a = got[k][..., some] if k != "dh0" else got[k][:, some]
        assert near(a, L[v].grad) < 2 * bound, (k, near(a, L[v].grad), bound)
    for k, v in (("dA", "A"), ("dD", "D"), ("ddt_bias", "b")):
        assert near(got[k][some], L[v].grad) < 8 * bound, (k, near(got[k][some], L[v].grad), bound)


def test_streams_graphs_and_repeats(kda):
    """Every entry point on a side stream, captured once and replayed with other inputs in between, against eager
    calls on the default stream: the same bits each time."""
    import torch
    offsets, B, T, cu = layout([300, 0, 1, 211])
    dim, ds = 72, 16
    x = scan_inputs(11, offsets, T, dim, ds, "bf16")
    s = scan_device(x, B, T, "bf16")
    h0, gf = dev(x["h0"]), dev(np.random.default_rng(2).normal(size=x["h0"].shape))
    w, wb = dev(np.random.default_rng(3).normal(size=(dim, 4))), dev(np.random.default_rng(4).normal(size=dim))
    c0 = dev(np.random.default_rng(5).normal(size=(4, 3, dim)), "bf16")
    cur = {k: v[:, :4] for k, v in s.items() if k in ("u", "dt", "B", "C", "z")}

    def everything():
        p = s["A"], s["B"], s["C"]
        o = list(kda.selective_scan_fwd(s["u"], s["dt"], *p, s["D"], s["z"], s["dt_bias"], initial_state=h0, cu_seqlens=cu,
                                        dt_softplus=True))
        o += [v for v in kda.selective_scan_bwd(s["u"], s["dt"], *p, s["z"], s["D"], s["z"], s["dt_bias"], initial_state=h0,
                                                grad_final_state=gf, cu_seqlens=cu, dt_softplus=True).values()]
        st = torch.empty_like(h0)
        o += [kda.selective_scan_step(cur["u"][0], cur["dt"][0], s["A"], cur["B"][0], cur["C"][0], h0, s["D"], cur["z"][0],
                                      s["dt_bias"], dt_softplus=True, final_state=st), st]
        o += list(kda.short_conv_fwd(s["u"], w, wb, initial_state=c0, cu_seqlens=cu, silu=True))
        o += [v for v in kda.short_conv_bwd(s["u"], w, s["z"], wb, initial_state=c0, cu_seqlens=cu, silu=True).values()]
        sc = torch.empty_like(c0)
        o += [kda.short_conv_step(cur["u"][0], w, c0, wb, silu=True, final_state=sc), sc]
        o += list(kda.layer_norm_fwd(s["u"], wb, wb, residual=s["z"]))
        o += [v for v in kda.layer_norm_bwd(s["u"], s["z"], wb, wb).values()]
        return o

    side = torch.cuda.Stream()
    eager = everything()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = everything()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kept = everything()
    for rep in range(4):
        s["u"].mul_(0.75)
        h0.add_(0.125 * rep)
        eager = everything()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, kept)), rep


def test_layer_run(kda):
    """A layer as it is used: norm with residual, projections, convolution, scan, per-head norm; its gradients through
    every operator's backward pass against autograd of the same layer in 64 bits on the CPU; then decoding goes on from
    the prompt's states, token by token, as one longer prompt would."""
    import torch
    import torch.nn.functional as fn
    B, T, more, dim, inner, ds, heads, W = 2, 45, 5, 24, 64, 16, 4, 4
    g = torch.Generator().manual_seed(0)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std)  # noqa: E731
    P = dict(nw=1 + n(dim, std=.1), nb=n(dim, std=.1), win=n(dim, 2 * inner, std=dim ** -.5), cw=n(inner, W, std=.5),
             cb=n(inner, std=.1), wdt=n(inner, inner, std=.3 * inner ** -.5), wB=n(inner, ds, std=inner ** -.5),
             wC=n(inner, ds, std=inner ** -.5), A=-torch.arange(1., ds + 1).repeat(inner, 1), D=torch.ones(inner),
             db=torch.full((inner,), -3.), hw=1 + n(inner // heads, std=.1), hb=n(inner // heads, std=.1),
             wout=n(inner, dim, std=inner ** -.5))
    x, res, gy = n(B, T + more, dim), n(B, T + more, dim), n(B, T, dim)

    # 64 bits, on the CPU, by autograd
    R = {k: v.double().requires_grad_() for k, v in P.items()}

    def plain(x, res):
        s = x + res
        xz = fn.layer_norm(s, (dim,), R["nw"], R["nb"]) @ R["win"]
        u, z = xz.chunk(2, -1)
        u = fn.silu(fn.conv1d(fn.pad(u.transpose(1, 2), (W - 1, 0)), R["cw"][:, None], R["cb"], groups=inner).transpose(1, 2))
        delta, Bm, Cm = fn.softplus(u @ R["wdt"] + R["db"]), u @ R["wB"], u @ R["wC"]
        h, ys = torch.zeros(B, inner, ds, dtype=torch.float64), []
        for t in range(x.shape[1]):
            h = torch.exp(delta[:, t, :, None] * R["A"]) * h + (delta[:, t] * u[:, t])[..., None] * Bm[:, t, None]
            ys.append((h * Cm[:, t, None]).sum(-1) + R["D"] * u[:, t])
        y = torch.stack(ys, 1) * fn.silu(z)
        y = fn.layer_norm(y.view(*y.shape[:2], heads, -1), (inner // heads,), R["hw"], R["hb"]).reshape(y.shape)
        return y @ R["wout"] + s

    xd, rd = x[:, :T].double().requires_grad_(), res[:, :T].double().requires_grad_()
    want = plain(xd, rd)
    (want * gy).sum().backward()

    # the framework, fp32
    Q = {k: v.cuda() for k, v in P.items()}
    xs, rs = x.cuda(), res.cuda()
    nx, s = kda.layer_norm_fwd(xs[:, :T].contiguous(), Q["nw"], Q["nb"], residual=rs[:, :T].contiguous())
    xz = nx @ Q["win"]
    u0, z = xz[..., :inner], xz[..., inner:]
    u, conv_state = kda.short_conv_fwd(u0, Q["cw"], Q["cb"], silu=True)
    dt, Bm, Cm = u @ Q["wdt"], u @ Q["wB"], u @ Q["wC"]
    y, state = kda.selective_scan_fwd(u, dt, Q["A"], Bm, Cm, Q["D"], z, Q["db"], dt_softplus=True)
    yh = y.view(B, T, heads, -1)
    ny = kda.layer_norm_fwd(yh, Q["hw"], Q["hb"]).view(B, T, inner)
    out = ny @ Q["wout"] + s

    go = gy.cuda()
    flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
    grads = dict(wout=flat(ny).t() @ flat(go))
    gn = kda.layer_norm_bwd(yh, (go @ Q["wout"].t()).view_as(yh), Q["hw"], Q["hb"])
    grads.update(hw=gn["dweight"], hb=gn["dbias"])
    dxz = torch.empty_like(xz)
    gs = kda.selective_scan_bwd(u, dt, Q["A"], Bm, Cm, gn["dx"].view_as(y), Q["D"], z, Q["db"], dt_softplus=True,
                                out=dict(du=torch.empty_like(u), ddt=torch.empty_like(u), dB=torch.empty_like(Bm),
                                         dC=torch.empty_like(Cm), dz=dxz[..., inner:]))
    grads.update(A=gs["dA"], D=gs["dD"], db=gs["ddt_bias"], wdt=flat(u).t() @ flat(gs["ddt"]),
                 wB=flat(u).t() @ flat(gs["dB"]), wC=flat(u).t() @ flat(gs["dC"]))
    du = gs["du"] + gs["ddt"] @ Q["wdt"].t() + gs["dB"] @ Q["wB"].t() + gs["dC"] @ Q["wC"].t()
    gc = kda.short_conv_bwd(u0, Q["cw"], du, Q["cb"], silu=True, out=dict(dx=dxz[..., :inner]))
    grads.update(cw=gc["dweight"], cb=gc["dbias"], win=flat(nx).t() @ flat(dxz))
    g0 = kda.layer_norm_bwd(s, dxz @ Q["win"].t(), Q["nw"], Q["nb"], grad_residual=go)
    grads.update(nw=g0["dweight"], nb=g0["dbias"])
    # fp32 through a chain of about 10 operators of about 100 roundings each in the norm
    near = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    assert near(out, want.detach()) < 1000 * 2 ** -24
    assert near(g0["dx"], xd.grad) < 4000 * 2 ** -24 and near(g0["dx"], rd.grad) < 4000 * 2 ** -24
    for k, v in grads.items():
        assert near(v, R[k].grad) < 4000 * 2 ** -24, (k, near(v, R[k].grad))

    # decoding goes on from the two states
    full = plain(x.double(), res.double())
    for t in range(T, T + more):
        nx, s = kda.layer_norm_fwd(xs[:, t], Q["nw"], Q["nb"], residual=rs[:, t])
        xz = nx @ Q["win"]
        u = kda.short_conv_step(xz[:, :inner], Q["cw"], conv_state, Q["cb"], silu=True)
        y = kda.selective_scan_step(u, u @ Q["wdt"], Q["A"], u @ Q["wB"], u @ Q["wC"], state, Q["D"], xz[:, inner:], Q["db"],
                                    dt_softplus=True)
        out = kda.layer_norm_fwd(y.view(B, heads, -1), Q["hw"], Q["hb"]).view(B, inner) @ Q["wout"] + s
        assert near(out, full[:, t].detach()) < 1000 * 2 ** -24, t


def test_convolution_and_norm_around_the_delta_rule(kda):
    """The convolution in front of KDA's q, k, v and the per-head norm behind it: a packed prompt, then single tokens
    from the cached states, equal to the longer prompt."""
    import torch
    H, d, T, more = 2, 128, 70, 3
    g = torch.Generator("cuda").manual_seed(1)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
    x, w = n(1, T + more, 3 * H * d).bfloat16(), n(3 * H * d, 4, std=.5)
    gate, beta = -torch.rand(1, T + more, H, d, generator=g, device="cuda") * .1, torch.rand(1, T + more, H, generator=g, device="cuda").bfloat16()
    nw = 1 + n(d, std=.1)

    def prompt(T):
        qkv, cs = kda.short_conv_fwd(x[:, :T], w, silu=True)
        q, k, v = (t.contiguous().view(1, T, H, d) for t in qkv.chunk(3, -1))
        o, S = kda.recurrent_fwd(q, k, v, gate[:, :T].contiguous(), beta[:, :T].contiguous(), qk_l2norm=True,
                                 out_dtype=torch.float32, token_by_token=True)
        return kda.layer_norm_fwd(o, nw), cs, S

    whole, _, _ = prompt(T + more)
    part, cs, S = prompt(T)
    assert torch.equal(part, whole[:, :T])
    for t in range(T, T + more):
        q, k, v = (a.contiguous().view(1, H, d) for a in kda.short_conv_step(x[:, t], w, cs, silu=True).chunk(3, -1))
        o = kda.recurrent_step(q, k, v, gate[:, t].contiguous(), beta[:, t].contiguous(), S, qk_l2norm=True, out_dtype=torch.float32)
        got = kda.layer_norm_fwd(o, nw)
        assert float((got - whole[:, t]).abs().max()) < 1e-3, t
