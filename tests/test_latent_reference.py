"""CPU pins of latent attention's references: closed forms, agreement with differentiation and with differences, the absorbed
form against the expanded one, and mistakes planted in the references that the bounds have to find."""
import numpy as np
import pytest

import latent_testlib as ref


def inputs(seed, Tq, Tk, H=2, dn=8, dr=4, dv=8):
    r = np.random.default_rng(seed)
    n = lambda *s: r.normal(size=s)  # noqa: E731
    return dict(q=n(Tq, H, dn + dr), k=n(Tk, H, dn), kr=n(Tk, dr), v=n(Tk, H, dv)), n(Tq, H, dv)


def test_closed_forms():
    x, _ = inputs(0, 3, 3)
    one = ref.attend(**{n: a[:1] for n, a in x.items()}, off_q=[0, 1], off_k=[0, 1], scale=0.3, causal=True)
    assert np.allclose(one["o"], x["v"][:1]) and np.allclose(
        one["lse"], 0.3 * (np.einsum("thd,thd->th", x["q"][:1, :, :8], x["k"][:1]) + np.einsum("thd,td->th", x["q"][:1, :, 8:], x["kr"][:1])))
    x["k"][:], x["kr"][:] = x["k"][0], x["kr"][0]  # equal keys: means of what is seen
    got = ref.attend(**x, off_q=[0, 3], off_k=[0, 3], scale=0.3, causal=True)
    for i in range(3):
        assert np.allclose(got["o"][i], x["v"][:i + 1].mean(0))


def test_rows_that_see_nothing():
    x, go = inputs(1, 5, 3)
    got = ref.attend(**x, off_q=[0, 5], off_k=[0, 3], scale=0.3, causal=True)
    assert (got["o"][:2] == 0).all() and (got["lse"][:2] == -np.inf).all() and np.isfinite(got["lse"][2:]).all()
    g = ref.attend_grads(**x, o=got["o"], lse=got["lse"], go=go, off_q=[0, 5], off_k=[0, 3], scale=0.3, causal=True)
    assert (g["dq"][0][:2] == 0).all() and all(np.isfinite(v[0]).all() for v in g.values())


@pytest.mark.parametrize("causal", [True, False])
def test_gradients_against_autograd_and_differences(causal):
    import torch
    off_q, off_k = [0, 4, 4, 9], [0, 6, 8, 12]
    x, go = inputs(2, 9, 12)
    f = ref.attend(**x, off_q=off_q, off_k=off_k, scale=0.4, causal=causal)
    g = ref.attend_grads(**x, o=f["o"], lse=f["lse"], go=go, off_q=off_q, off_k=off_k, scale=0.4, causal=causal)
    t = {n: torch.from_numpy(a).requires_grad_() for n, a in x.items()}
    total = 0
    for sq, sk in ref.sequences(off_q, off_k):
        if sq.start == sq.stop or sk.start == sk.stop:
            continue
        see = torch.from_numpy(ref.seen(sq.stop - sq.start, sk.stop - sk.start, causal))
        some = see.any(-1)
        for h in range(2):
            s = (t["q"][sq, h] @ torch.cat([t["k"][sk, h], t["kr"][sk]], -1).t() * 0.4).masked_fill(~see, -1e300)
            o = torch.softmax(s, -1)[some] @ t["v"][sk, h]
            total = total + (o * torch.from_numpy(go[sq, h])[some]).sum()
    total.backward()
    for name, leaf in (("dq", "q"), ("dk", "k"), ("dk_rope", "kr"), ("dv", "v")):
        assert np.allclose(g[name][0], t[leaf].grad.numpy(), atol=1e-12), name
    # and by differences
    r = np.random.default_rng(3)
    for name, leaf in (("dq", "q"), ("dk", "k"), ("dk_rope", "kr"), ("dv", "v")):
        d = r.normal(size=x[leaf].shape)
        loss = [(ref.attend(**{**x, leaf: x[leaf] + e * d}, off_q=off_q, off_k=off_k, scale=0.4, causal=causal)["o"] * go).sum() for e in (1e-5, -1e-5)]
        assert abs((loss[0] - loss[1]) / 2e-5 - (g[name][0] * d).sum()) < 1e-6 * (1 + abs(loss[0])), name


def test_absorbed_form_is_the_expanded_one():
    """Keys and values expanded from cached rows by a head's projections, against queries and outputs taken through them."""
    r = np.random.default_rng(4)
    H, dn, dv, dl, dr, T = 3, 5, 6, 7, 4, 9
    cache, wk, wv = r.normal(size=(4, 3, dl + dr)), r.normal(size=(H, dl, dn)), r.normal(size=(H, dl, dv))
    table = np.array([[2, 0, 3, -1]])
    rows = ref.cached_rows(cache, table[0], T)
    q = r.normal(size=(1, H, dn + dr))
    k, v = np.einsum("tl,hld->thd", rows[:, :dl], wk), np.einsum("tl,hld->thd", rows[:, :dl], wv)
    want = ref.attend(q, k, rows[:, dl:], v, [0, 1], [0, T], 0.3, True)
    got = ref.step(np.einsum("nhd,hld->nhl", q[..., :dn], wk), q[..., dn:], cache, table, [T], 0.3)
    assert np.allclose(np.einsum("nhl,hld->nhd", got["o"], wv), want["o"]) and np.allclose(got["lse"], want["lse"])


def test_rotation_keeps_lengths_and_differences_of_positions():
    r = np.random.default_rng(5)
    x, f = r.normal(size=(2, 1, 8)), 10000.0 ** (-np.arange(4) / 4)
    for inter in (False, True):
        a = [ref.rotate(x, np.array(p), f, inter, 0, 1.0) for p in ([3, 10], [103, 110])]
        assert np.allclose(np.linalg.norm(a[0], axis=-1), np.linalg.norm(x, axis=-1))
        assert np.isclose(a[0][0, 0] @ a[0][1, 0], a[1][0, 0] @ a[1][1, 0])
        assert np.allclose(ref.rotate(a[0], np.array([3, 10]), f, inter, 0, 1.0, -1), x)


def test_page_lookup_of_the_reference():
    cache = np.arange(24.0).reshape(4, 3, 2)
    assert ref.cached_rows(cache, [1, 3], 5)[:, 0].tolist() == [6, 8, 10, 18, 20]
    assert ref.cached_rows(cache, [1, 7, -2, 0], 99)[:, 0].tolist() == [6, 8, 10, 0, 2, 4]
    assert ref.cached_rows(cache, [1], 0).shape == (0, 2)


@pytest.mark.parametrize("plant", ["mask", "scale", "rope", "value"])
def test_planted_mistakes_are_found(plant):
    x, _ = inputs(6, 40, 40)
    args = dict(off_q=[0, 40], off_k=[0, 40], scale=0.3, causal=True)
    good = ref.attend(**x, **args, kind="bf16", out="bf16")
    y = {n: a.copy() for n, a in x.items()}
    if plant == "mask":
        args["off_k"] = [0, 39]
    elif plant == "scale":
        args["scale"] = 0.33
    elif plant == "rope":
        y["kr"][17] *= -1
    else:
        y["v"][3] *= 1.1
    bad = ref.attend(**y, **args)
    with pytest.raises(AssertionError):
        ref.check("o", bad["o"], good["o"], good["eo"], good["no"])
