"""Latent attention (rotary positions, the paged cache, prompts with gradients, single tokens over the cache) against its
64-bit references: types, head layouts, lengths from none to several tiles, odd sizes, strides, rows that see nothing,
pages that do not exist or end inside a tile, rows outside the sequences, other streams, graphs, offsets past 32 bits, and
a run of all of them as a layer uses them."""
import numpy as np
import pytest

import latent_testlib as ref

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


def host(t):
    return t.double().cpu().numpy()


def ints(a):
    import torch
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def make(seed, shape, dtype, std=1.0, layout="dense", pad=8):
    """Random values on the device; layout: dense, sliced (columns of a wider buffer whose others are NaN), heads (the heads in
    front of the rows in memory; shape [..., rows, H, D])."""
    import torch
    g = torch.Generator().manual_seed(seed)
    t = (torch.randn(*shape, generator=g) * std).to(tdtype(dtype))
    if layout == "sliced":
        wide = torch.full((*shape[:-1], shape[-1] + 2 * pad), float("nan"), dtype=t.dtype)
        wide[..., pad:-pad] = t
        return wide.cuda()[..., pad:-pad]
    if layout == "heads":
        return t.transpose(-2, -3).contiguous().cuda().transpose(-2, -3)
    return t.cuda()


# ---- rotary positions and the cache ------------------------------------------------------------------------

def check_rotary(kda, seed, lead, H, D, rot, offset, interleaved, dtype, scale=1.0, start=0, layout="dense", pad=8, in_place=False, back=False):
    import torch
    x = make(seed, (*lead, H, D), dtype, layout=layout, pad=pad)
    rows = int(np.prod(lead))
    r = np.random.default_rng(seed)
    pos = (start + r.integers(0, 5000, rows)).clip(-2 ** 31, 2 ** 31 - 1)
    f = (10000.0 ** (-np.arange(rot // 2) * 2 / rot)).astype(np.float32)
    fd = torch.from_numpy(f).cuda()
    before = host(x).reshape(rows, H, D)
    fn = kda.rotary_bwd if back else kda.rotary_fwd
    args = (x, ints(pos).view(lead), fd)
    y = fn(*args, interleaved, offset, scale, **({"grad_x" if back else "y": x} if in_place else {}))
    want = ref.rotate(before, pos, f.astype(np.float64), interleaved, offset, scale, -1 if back else 1)
    bound = ref.rotate_bound(before, rot // 2, interleaved, offset, scale, dtype)
    part = np.zeros_like(want, bool)
    part[..., offset:offset + rot] = True
    bound += np.where(part, ref.U[dtype] * np.abs(want), 0.0)
    ref.check("y", host(y).reshape(want.shape), want, bound, bound)
    assert (y.data_ptr() == x.data_ptr()) == in_place


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("lead,H,D,rot,offset", [
    ((1,), 1, 2, 2, 0), ((3,), 2, 64, 64, 0), ((2, 5), 3, 192, 64, 128), ((1, 301), 4, 128, 32, 40), ((7,), 5, 37, 10, 3),
    ((513,), 1, 256, 128, 0), ((2,), 130, 96, 48, 16), ((2, 3, 4), 2, 80, 80, 0), ((3,), 1, 5000, 4096, 8), ((1,), 40, 1200, 16, 1184), ((2,), 2, 32767, 64, 903)])
def test_rotary(kda, dtype, interleaved, lead, H, D, rot, offset):
    check_rotary(kda, 1, lead, H, D, rot, offset, interleaved, dtype)
    check_rotary(kda, 2, lead, H, D, rot, offset, interleaved, dtype, scale=1.25, in_place=True)
    check_rotary(kda, 3, lead, H, D, rot, offset, interleaved, dtype, back=True)


@pytest.mark.parametrize("start", [10 ** 6, 2 ** 31 - 5000, -2 ** 31, -77])
def test_rotary_far_positions(kda, start):
    for interleaved in (True, False):
        check_rotary(kda, 4, (40,), 2, 128, 128, 0, interleaved, "fp32", start=start)


@pytest.mark.parametrize("layout,pad", [("sliced", 8), ("sliced", 3), ("heads", 0)])
def test_rotary_strides(kda, layout, pad):
    for dtype in ("bf16", "fp32"):
        for in_place in (False, True):
            check_rotary(kda, 5, (2, 9) if layout == "sliced" else (9,), 3, 192, 64, 128, True, dtype, layout=layout, pad=pad, in_place=in_place)
            check_rotary(kda, 6, (2, 9) if layout == "sliced" else (9,), 3, 64, 64, 0, False, dtype, layout=layout, pad=pad, in_place=in_place)


def test_rotary_leaves_what_lies_between(kda):
    """In place on a slice: the other columns of the buffer keep their bits."""
    import torch
    wide = torch.arange(2 * 3 * 32, device="cuda", dtype=torch.float32).view(2, 3, 32)
    kept = wide.clone()
    f, _ = kda.rotary_frequencies(8)
    kda.rotary_fwd(wide[..., 8:24], ints([5, 6]), f, offset=4, y=wide[..., 8:24])
    keep = torch.ones(32, dtype=torch.bool, device="cuda")
    keep[12:20] = False
    assert torch.equal(wide[..., keep], kept[..., keep]) and not torch.equal(wide, kept)


def test_rotary_frequencies(kda):
    f, scale = kda.rotary_frequencies(64, 10000.0, device="cpu")
    assert scale == 1.0 and np.allclose(f.numpy(), 10000.0 ** (-np.arange(0, 64, 2) / 64), rtol=1e-7)
    f2, _ = kda.rotary_frequencies(64, factor=4.0, device="cpu")
    assert np.allclose(f2.numpy(), f.numpy() / 4, rtol=1e-7)
    f3, scale = kda.rotary_frequencies(64, factor=4.0, original_length=4096, device="cpu")
    turns = 4096 * f.double().numpy() / (2 * np.pi)
    assert np.allclose(f3.numpy()[turns > 32], f.numpy()[turns > 32], rtol=1e-7) and np.isclose(scale, 1 + 0.1 * np.log(4))
    assert np.allclose(f3.numpy()[turns < 1], f.numpy()[turns < 1] / 4, rtol=1e-7)
    assert ((f3 <= f * (1 + 1e-6)) & (f3 >= f / 4 * (1 - 1e-6))).all()
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, factor=0.5), dict(rot=8, base=-1.0)):
        with pytest.raises(ValueError):
            kda.rotary_frequencies(**bad)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,dl,dr,page,blocks,pad", [(1, 512, 64, 64, 2, 8), (70, 512, 64, 16, 9, 8), (33, 40, 8, 7, 6, 3), (5, 13, 6, 1, 9, 0),
                                                    (3, 5, 130, 2, 3, 1)])
@pytest.mark.parametrize("turned", ["interleaved", "halves", "no"])
def test_append(kda, dtype, T, dl, dr, page, blocks, pad, turned):
    import torch
    wide = make(7, (T, dl + dr + pad), dtype)
    latent, rope = wide[:, :dl], wide[:, dl + pad:]
    cache = make(8, (blocks, page, dl + dr), dtype)
    kept = cache.clone()
    r = np.random.default_rng(9)
    slots = r.permutation(blocks * page)[:T]
    slots[::4] = [-1, blocks * page, -2 ** 31, 2 ** 31 - 1][T % 4]  # of every four one goes nowhere
    if T == 1:
        slots[0] = blocks * page - 1
    pos, f = r.integers(0, 10 ** 6, T), (10000.0 ** (-np.arange(dr // 2) * 2 / dr)).astype(np.float32)
    more = () if turned == "no" else (ints(pos), torch.from_numpy(f).cuda(), turned == "interleaved", 1.5)
    assert kda.latent_cache_append(latent, rope, cache, ints(slots), *more) is cache
    flat, old = host(cache).reshape(-1, dl + dr), host(kept).reshape(-1, dl + dr)
    rr = host(rope)[:, None]
    turned_rows = rr if turned == "no" else ref.rotate(rr, pos, f.astype(np.float64), turned == "interleaved", 0, 1.5)
    bound = 0 * rr if turned == "no" else ref.rotate_bound(rr, dr // 2, turned == "interleaved", 0, 1.5, dtype) + ref.U[dtype] * np.abs(turned_rows)
    hit = {}
    for i, s in enumerate(slots):
        if 0 <= s < blocks * page:
            hit[int(s)] = i
    for s in range(blocks * page):
        if s not in hit:
            assert (flat[s] == old[s]).all(), s
        else:
            i = hit[s]
            assert (flat[s, :dl] == host(latent)[i]).all()
            assert (np.abs(flat[s, dl:] - turned_rows[i, 0]) <= bound[i, 0]).all(), s


# ---- attention over prompts --------------------------------------------------------------------------------

FIXED = [(1, 1, 1), (2, 5, 5), (1, 64, 64), (1, 129, 200), (2, 70, 33), (1, 33, 257), (1, 1, 300), (3, 131, 131), (1, 300, 1), (1, 40, 0)]
PACKED = [([1], [1]), ([5, 0, 3, 129, 1], [5, 4, 0, 200, 1]), ([70, 128, 0, 1, 257], [33, 128, 0, 64, 257]), ([0, 0, 2], [3, 0, 2]),
          ([64] * 5, [64] * 5)]
DIMS = [(128, 64, 128), (64, 32, 64), (72, 24, 104), (8, 8, 8), (128, 8, 16), (16, 64, 128)]


def prompts(seed, case, H, dims, dtype, layout="dense", extra=0):
    """(device tensors, numpy views with one row axis, offsets, keywords); extra: rows behind the last sequence, NaN."""
    dn, dr, dv = dims
    if isinstance(case, tuple) and isinstance(case[0], int):
        B, Tq, Tk = case
        off_q, off_k, kw = [b * Tq for b in range(B + 1)], [b * Tk for b in range(B + 1)], {}
    else:
        B, (nq, nk) = 1, case
        off_q, off_k = np.concatenate([[0], np.cumsum(nq)]).tolist(), np.concatenate([[0], np.cumsum(nk)]).tolist()
        Tq, Tk, kw = off_q[-1] + extra, off_k[-1] + extra, dict(cu_seqlens_q=ints(off_q), cu_seqlens_k=ints(off_k))
    heads = layout if B == 1 or layout != "heads" else "dense"
    t = dict(q=make(seed, (B, Tq, H, dn + dr), dtype, 1.5, heads), kr=make(seed + 1, (B, Tk, dr), dtype, 1.5, "sliced" if layout == "sliced" else "dense"))
    if layout == "sliced":  # one projection's output
        wide = make(seed + 2, (B, Tk, H, dn + dv), dtype)
        t["k"], t["v"] = wide[..., :dn], wide[..., dn:]
    else:
        t["k"], t["v"] = make(seed + 2, (B, Tk, H, dn), dtype, 1.0, heads), make(seed + 3, (B, Tk, H, dv), dtype, 1.0, heads)
    if extra:
        t["q"][:, off_q[-1]:] = float("nan")
        for n in ("k", "v", "kr"):
            t[n][:, off_k[-1]:] = float("nan")
    flat = {n: host(a).reshape(-1, *a.shape[2:]) for n, a in t.items()}
    return t, flat, off_q, off_k, kw


def check_fwd(kda, seed, case, H, dims, dtype, causal, layout="dense", out=None, extra=0, scale=0.11):
    import torch
    t, x, off_q, off_k, kw = prompts(seed, case, H, dims, dtype, layout, extra)
    B, Tq = t["q"].shape[:2]
    o = torch.full((B, Tq, H, dims[2]), 7.0, dtype=tdtype(out or dtype), device="cuda")
    lse = torch.full((B, Tq, H), 7.0, device="cuda")
    got = kda.latent_attention_fwd(t["q"], t["k"], t["kr"], t["v"], scale, causal, o=o, lse=lse, **kw)
    assert got[0] is o and got[1] is lse
    rows = off_q[-1]
    want = ref.attend(*(x[n] for n in ("q", "k", "kr", "v")), off_q, off_k, scale, causal, dtype, out or dtype)
    o2, l2 = host(o).reshape(-1, H, dims[2]), host(lse).reshape(-1, H)
    ref.check("o", o2[:rows], want["o"][:rows], want["eo"][:rows], want["no"][:rows])
    ref.check("lse", l2[:rows], want["lse"][:rows], want["el"][:rows], want["el"][:rows])
    assert (o2[rows:] == 7).all() and (l2[rows:] == 7).all()
    return t, x, off_q, off_k, kw, o, lse


def check_bwd(kda, seed, case, H, dims, dtype, causal, layout="dense", grad=None, extra=0, scale=0.11):
    import torch
    t, x, off_q, off_k, kw, o, lse = check_fwd(kda, seed, case, H, dims, dtype, causal, layout, extra=extra, scale=scale)
    dn, dr, dv = dims
    go = make(seed + 9, tuple(o.shape), dtype, layout="sliced" if layout == "sliced" else "dense")
    grad = grad or dtype
    new = lambda *s: torch.full(s, 7.0, dtype=tdtype(grad), device="cuda")  # noqa: E731
    B, Tq, Tk = t["q"].shape[0], t["q"].shape[1], t["k"].shape[1]
    wide = new(B, Tk, H, dn + dv)  # dk and dv as parts of one projection's gradient
    out = dict(dq=new(B, Tq, H, dn + dr), dk=wide[..., :dn], dv=wide[..., dn:], dk_rope=new(B, Tk, dr))
    got = kda.latent_attention_bwd(t["q"], t["k"], t["kr"], t["v"], o, lse, go, scale, causal, grad_dtype=tdtype(grad), out=out, **kw)
    flat = lambda a: host(a).reshape(-1, *a.shape[2:])  # noqa: E731
    want = ref.attend_grads(*(x[n] for n in ("q", "k", "kr", "v")), flat(o), flat(lse), flat(go), off_q, off_k, scale, causal, dtype, grad)
    for n in ("dq", "dk", "dk_rope", "dv"):
        rows = (off_q if n == "dq" else off_k)[-1]
        a = flat(got[n])
        ref.check(n, a[:rows], *(b[:rows] for b in want[n]))
        assert (a[rows:] == 7).all(), n


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", FIXED + PACKED, ids=str)
def test_attention_and_gradients_over_lengths(kda, dtype, causal, case):
    check_bwd(kda, 10, case, 2, (128, 64, 128), dtype, causal)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("H", [1, 3, 8])
def test_attention_and_gradients_over_head_sizes(kda, dtype, dims, H):
    check_bwd(kda, 20, (2, 67, 90), H, dims, dtype, True)
    check_bwd(kda, 30, ([40, 0, 1, 131], [40, 7, 3, 140]), H, dims, dtype, True, layout="sliced")


@pytest.mark.parametrize("layout", ["sliced", "heads"])
def test_attention_layouts_and_types(kda, layout):
    check_bwd(kda, 40, (1, 100, 150), 4, (128, 64, 128), "bf16", True, layout, grad="fp32")
    check_bwd(kda, 41, (1, 100, 150), 4, (128, 64, 128), "fp32", True, layout, grad="bf16")
    check_fwd(kda, 42, (1, 100, 150), 4, (64, 32, 64), "bf16", False, layout, out="fp32")
    check_fwd(kda, 43, (1, 100, 150), 4, (64, 32, 64), "fp32", True, layout, out="bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_behind_the_last_sequence(kda, dtype):
    """NaN there enters nothing, and outputs keep what they hold there."""
    check_bwd(kda, 50, ([30, 101], [40, 90]), 2, (128, 64, 128), dtype, True, extra=13)
    check_bwd(kda, 51, ([30, 101], [40, 90]), 2, (64, 32, 64), dtype, False, extra=70)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_large_scores(kda, dtype):
    """Rows whose maximum moves by hundreds from tile to tile: weights far below and above the first ones."""
    import torch
    t, x, off_q, off_k, kw = prompts(60, (1, 70, 400), 2, (128, 64, 128), dtype)
    ramp = torch.linspace(-3, 3, 400, device="cuda")[torch.randperm(400, generator=torch.Generator().manual_seed(0)).cuda()]
    t["q"][..., 0], t["k"][..., 0] = 16.0, (ramp[:, None] * 16).to(t["k"].dtype)
    x = {n: host(a).reshape(-1, *a.shape[2:]) for n, a in t.items()}
    o, lse = kda.latent_attention_fwd(t["q"], t["k"], t["kr"], t["v"], 1.0, True)
    want = ref.attend(*(x[n] for n in ("q", "k", "kr", "v")), off_q, off_k, 1.0, True, dtype, dtype)
    ref.check("o", host(o)[0], want["o"], want["eo"], want["no"])
    ref.check("lse", host(lse)[0], want["lse"], want["el"], want["el"])


def test_infinite_values_stay_in_their_rows(kda):
    """A query of infinities gives NaN in its own row alone; NaN and infinite keys behind a query's last tile do not reach
    it."""
    import torch
    t, _, _, _, _ = prompts(61, (1, 130, 130), 2, (128, 64, 128), "bf16")
    clean = kda.latent_attention_fwd(t["q"], t["k"], t["kr"], t["v"])
    t["q"][0, 5, 1] = float("inf")
    o, lse = kda.latent_attention_fwd(t["q"], t["k"], t["kr"], t["v"])
    assert torch.isnan(o[0, 5, 1]).all()
    keep = torch.ones(130, 2, dtype=torch.bool, device="cuda")
    keep[5, 1] = False
    assert torch.equal(o[0][keep], clean[0][0][keep]) and torch.equal(lse[0][keep], clean[1][0][keep])


# ---- single tokens over the cache --------------------------------------------------------------------------

def check_step(kda, seed, lengths, H, dl, dr, page, dtype, out=None, layout="dense", table_edit=None, std=1.0, scale=0.05, spare=2, wider=0):
    import torch
    N = len(lengths)
    r = np.random.default_rng(seed)
    pages = [-(-max(0, n) // page) for n in lengths]
    width = max(max(pages), 1)
    blocks = sum(pages) + spare
    cache = make(seed, (blocks, page, dl + dr), dtype, std)
    order, table, at = r.permutation(blocks), np.full((N, width), -7), 0
    used = np.zeros((blocks, page), bool)
    for n, p in enumerate(pages):
        table[n, :p] = order[at:at + p]
        at += p
        for pos in range(max(0, lengths[n])):
            used[table[n, pos // page], pos % page] = True
    cache[torch.from_numpy(~used).cuda()] = float("nan")  # never written
    if table_edit:
        table_edit(table)
    dev = ints(np.concatenate([table, np.full((N, wider), -9)], 1))[:, :width]
    ql, qr = make(seed + 1, (N, H, dl), dtype, layout=layout), make(seed + 2, (N, H, dr), dtype, layout=layout)
    o, lse = kda.latent_attention_step(ql, qr, cache, dev, ints(lengths), scale, out_dtype=tdtype(out or dtype))
    want = ref.step(host(ql), host(qr), host(cache), table, lengths, scale, dtype, out or dtype)
    ref.check("o", host(o), want["o"], want["eo"], want["no"])
    ref.check("lse", host(lse), want["lse"], want["el"], want["el"])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lengths,page", [([1], 1), ([0], 16), ([0, 1, 15, 16, 17, 31, 32, 33], 16), ([64, 65, 200, 0, 129], 64), ([100, 3, 77], 7),
                                          ([500], 3), ([2100], 64), ([40] * 40, 16)])
def test_step_over_lengths(kda, dtype, lengths, page):
    check_step(kda, 70, lengths, 16, 512, 64, page, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H", [1, 5, 16, 17, 32, 33, 64, 65, 128])
def test_step_over_heads(kda, dtype, H):
    check_step(kda, 80, [130, 0, 61], H, 512, 64, 16, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dl,dr", [(512, 64), (256, 32), (128, 64), (200, 8), (8, 8), (136, 40), (504, 56)])
def test_step_over_sizes(kda, dtype, dl, dr):
    check_step(kda, 90, [300, 7, 64], 20, dl, dr, 16, dtype)
    check_step(kda, 91, [33, 150], 40, dl, dr, 5, dtype, layout="sliced", wider=3)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,longest,H,page", [(1100, 40, 4, 16), (1024, 130, 33, 5), (1500, 2100, 4, 64), (700, 70, 20, 16), (513, 2, 40, 1), (1023, 33, 17, 64)])
def test_step_of_many_sequences(kda, dtype, N, longest, H, page):
    """A workgroup per sequence, and runs of tiles that pass over several sequences, some without rows."""
    r = np.random.default_rng(N)
    lengths = r.integers(0, min(longest, 100) + 1, N) * (r.random(N) < 0.8)
    lengths[r.integers(N)] = longest
    lengths[-3:] = 0, 1, 0
    lengths[:2] = 0, -3
    check_step(kda, 96, [int(n) for n in lengths], H, 64, 16, page, dtype)


def test_step_of_the_most_sequences(kda):
    """65,535 sequences of 128 heads, of one row each or none: the row itself, and its scaled score (a sum of 16 products of
    bf16 in fp32, off by at most 20 half steps of their absolute sum)."""
    import torch
    N, H, dl, dr = 65535, 128, 8, 8
    ql, qr, cache = make(97, (N, H, dl), "bf16"), make(98, (N, H, dr), "bf16"), make(99, (N, 1, dl + dr), "bf16")
    table = torch.randperm(N, device="cuda", dtype=torch.int32)[:, None]
    lengths = torch.ones(N, device="cuda", dtype=torch.int32)
    lengths[::7] = 0
    o, lse = kda.latent_attention_step(ql, qr, cache, table, lengths, 0.25)
    rows = cache[table[:, 0].long(), 0]
    some = lengths > 0
    assert torch.equal(o[some], rows[some][:, None, :dl].expand(-1, H, -1)) and (o[~some] == 0).all() and (lse[~some] == -float("inf")).all()
    products = torch.cat([ql, qr], -1)[some].double() * rows[some].double()[:, None]
    bound = 0.25 * 20 * 2.0 ** -24 * products.abs().sum(-1) + 4 * 2.0 ** -24
    assert ((lse[some].double() - 0.25 * products.sum(-1)).abs() <= bound).all()


def test_step_layouts_types_and_large_scores(kda):
    check_step(kda, 92, [100, 40], 16, 512, 64, 16, "bf16", out="fp32", layout="heads")
    check_step(kda, 93, [100, 40], 16, 512, 64, 16, "fp32", out="bf16", layout="heads")
    check_step(kda, 94, [700, 90], 16, 512, 64, 16, "bf16", std=4.0, scale=0.5)
    check_step(kda, 95, [700, 90], 16, 512, 64, 16, "fp32", std=4.0, scale=0.5)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_step_on_bad_pages(kda, dtype):
    """Blocks that do not exist hold no rows, also a whole sequence of them; lengths beyond the table end with it."""
    def edit(table):
        table[0, 1], table[0, 3], table[1, :] = -1, 10 ** 6, 2 ** 31 - 1
    check_step(kda, 96, [90, 40, 33], 16, 512, 64, 16, dtype, table_edit=edit)
    check_step(kda, 97, [160, 160 + 16], 4, 128, 32, 16, dtype)
    import torch
    cache, table = make(1, (10, 16, 576), dtype), ints(np.arange(10).reshape(1, 10))
    ql, qr = make(2, (1, 16, 512), dtype), make(3, (1, 16, 64), dtype)
    a = [kda.latent_attention_step(ql, qr, cache, table, ints([n]), 0.05) for n in (160, 161, 2 ** 31 - 1)]
    assert all(torch.equal(a[0][0], b[0]) and torch.equal(a[0][1], b[1]) for b in a[1:])
    o, lse = kda.latent_attention_step(ql, qr, cache, table, ints([-3]), 0.05)
    assert (o == 0).all() and (lse == -float("inf")).all()
    o, lse = kda.latent_attention_step(ql, qr, cache[:0], table, ints([5]), 0.05)
    assert (o == 0).all() and (lse == -float("inf")).all()


# ---- offsets past 32 bits ----------------------------------------------------------------------------------

def test_step_in_a_cache_past_four_gigabytes(kda):
    import torch
    page, W, blocks = 64, 576, 70000
    cache = torch.empty(blocks, page, W, dtype=torch.bfloat16, device="cuda")  # 5.2 GB
    pages = [0, blocks - 1, blocks // 2, blocks - 2]
    part = make(5, (4, page, W), "bf16")
    cache[pages] = part
    ql, qr = make(6, (1, 16, 512), "bf16"), make(7, (1, 16, 64), "bf16")
    got = kda.latent_attention_step(ql, qr, cache, ints([pages]), ints([250]), 0.05)
    same = kda.latent_attention_step(ql, qr, part, ints([[0, 1, 2, 3]]), ints([250]), 0.05)
    assert torch.equal(got[0], same[0]) and torch.equal(got[1], same[1])
    latent, rope = make(8, (2, 512), "bf16"), make(9, (2, 64), "bf16")
    last = blocks * page - 1
    kda.latent_cache_append(latent, rope, cache, ints([last, 70]))
    assert torch.equal(cache[-1, -1], torch.cat([latent[0], rope[0]])) and torch.equal(cache[1, 6], torch.cat([latent[1], rope[1]]))
    assert torch.equal(cache[pages[1], :-1], part[1, :-1])


def test_attention_with_rows_past_32_bits(kda):
    """Rows 2^22 - 8 elements apart: the last ones of every tensor lie more than 2^32 bytes on."""
    import torch
    T, H, far = 700, 2, (1 << 22) - 8
    buf = torch.empty(T * far, dtype=torch.bfloat16, device="cuda")
    place = lambda at, w: torch.as_strided(buf, (1, T, H, w), (T * far, far, w, 1), at)  # noqa: E731
    views = dict(q=place(0, 192), k=place(1000, 128), v=place(2000, 128), go=place(3000, 128), o=place(4000, 128), dq=place(5000, 192),
                 dk=place(6000, 128), dv=place(7000, 128))
    kr, dkr = torch.as_strided(buf, (1, T, 64), (T * far, far, 1), 8000), torch.as_strided(buf, (1, T, 64), (T * far, far, 1), 9000)
    dense = {n: make(i, tuple(views[n].shape), "bf16") for i, n in enumerate(("q", "k", "v", "go"))}
    r = make(9, (1, T, 64), "bf16")
    for n, a in dense.items():
        views[n].copy_(a)
    kr.copy_(r)
    o, lse = kda.latent_attention_fwd(dense["q"], dense["k"], r, dense["v"])
    o2, lse2 = kda.latent_attention_fwd(views["q"], views["k"], kr, views["v"], o=views["o"])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    bf = torch.bfloat16
    g = kda.latent_attention_bwd(dense["q"], dense["k"], r, dense["v"], o, lse, dense["go"], grad_dtype=bf)
    g2 = kda.latent_attention_bwd(views["q"], views["k"], kr, views["v"], o2, lse2, views["go"], grad_dtype=bf,
                                  out=dict(dq=views["dq"], dk=views["dk"], dv=views["dv"], dk_rope=dkr))
    for n in g:
        assert torch.equal(g[n], g2[n]), n
    x = torch.as_strided(buf, (T, H, 192), (far, 192, 1), 10000)
    x.copy_(dense["q"][0])
    f, _ = kda.rotary_frequencies(64)
    pos = ints(np.arange(T))
    want = kda.rotary_fwd(dense["q"][0], pos, f, True, 128)
    assert torch.equal(kda.rotary_fwd(x, pos, f, True, 128, y=x), want)


# ---- calls ---------------------------------------------------------------------------------------------------

def everything(kda, t):
    """One call of every entry point on the tensors of `run_inputs`."""
    import torch
    f, _ = t["freq"]
    out = [kda.rotary_fwd(t["q"], t["pos"], f, True, 128), kda.rotary_bwd(t["q"], t["pos"], f, False, 0)]
    cache = torch.empty_like(t["cache"])
    cache.copy_(t["cache"])
    out.append(kda.latent_cache_append(t["latent"], t["rope"], cache, t["slots"], t["pos"][0], f, True))
    out += kda.latent_attention_step(t["ql"], t["qr"], cache, t["table"], t["lengths"], 0.05)
    o, lse = kda.latent_attention_fwd(t["q"], t["k"], t["kr"], t["v"], cu_seqlens_q=t["cu"], cu_seqlens_k=t["cu"])
    out += [o, lse]
    out += kda.latent_attention_bwd(t["q"], t["k"], t["kr"], t["v"], o, lse, t["go"], cu_seqlens_q=t["cu"], cu_seqlens_k=t["cu"]).values()
    return out


def run_inputs(kda, dtype="bf16"):
    T, H = 300, 2
    t = dict(q=make(1, (1, T, H, 192), dtype), k=make(2, (1, T, H, 128), dtype), v=make(3, (1, T, H, 128), dtype), kr=make(4, (1, T, 64), dtype),
             go=make(5, (1, T, H, 128), dtype), cu=ints([0, 100, 100, 271]), pos=ints(np.arange(T)[None]), freq=kda.rotary_frequencies(64),
             cache=make(6, (30, 16, 576), dtype), latent=make(7, (T, 512), dtype), rope=make(8, (T, 64), dtype), slots=ints(np.arange(T) + 50),
             ql=make(9, (3, 16, 512), dtype), qr=make(10, (3, 16, 64), dtype), table=ints(np.arange(30).reshape(3, 10)), lengths=ints([160, 0, 99]))
    for n in ("q", "k", "v", "kr", "go"):
        t[n][:, 271:] = 0
    return t


def covered(outs):
    """The outputs without the rows behind the last sequence, which a call leaves as they were."""
    return [a[:, :271] if a.dim() >= 3 and a.shape[1] == 300 else a for a in outs]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_streams_graphs_and_repeats(kda, dtype):
    """Every entry point on a side stream, captured once and replayed with other inputs in between, against eager calls
    on the default stream: the same bits each time."""
    import torch
    t = run_inputs(kda, dtype)
    eager = covered(everything(kda, t))
    assert all(torch.equal(a, b) for a, b in zip(eager, covered(everything(kda, t))))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = covered(everything(kda, t))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kept = covered(everything(kda, t))
    for rep in range(4):
        t["q"].mul_(0.75)
        t["latent"].mul_(1.25)
        t["lengths"].copy_(ints([[100, 3, 160], [0, 0, 0], [1, 160, 16], [160, 160, 160]][rep]))
        eager = covered(everything(kda, t))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, kept)), rep


def test_two_graphs_share_a_workspace(kda):
    """The caller's workspace serves calls one after the other, in two graphs as well."""
    import torch
    t = run_inputs(kda)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    q2 = t["ql"] * 2

    def one(ql):
        return kda.latent_attention_step(ql, t["qr"], t["cache"], t["table"], t["lengths"], 0.05, workspace=ws)
    want = [one(t["ql"]), one(q2)]
    graphs, kept = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g, ql in zip(graphs, (t["ql"], q2)):
        with torch.cuda.graph(g):
            kept.append(one(ql))
    for rep in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, kept):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refusals(kda):
    import torch
    from gated_delta_rule_52_amd._lib import KdaError
    t = run_inputs(kda)
    f, _ = t["freq"]
    args = (t["q"], t["k"], t["kr"], t["v"])
    bad = [
        lambda: kda.rotary_fwd(t["q"].cpu(), t["pos"], f),
        lambda: kda.rotary_fwd(t["q"], t["pos"].long(), f),
        lambda: kda.rotary_fwd(t["q"], t["pos"][:, 1:], f),
        lambda: kda.rotary_fwd(t["q"], t["pos"], f.double()),
        lambda: kda.rotary_fwd(t["q"].half(), t["pos"], f),
        lambda: kda.rotary_fwd(t["q"], t["pos"], f, offset=129),
        lambda: kda.rotary_fwd(t["q"], t["pos"], f, y=t["q"][:, :, :, 1:]),
        lambda: kda.rotary_fwd(t["q"][0, 0], t["pos"], f),
        lambda: kda.latent_cache_append(t["latent"], t["rope"].float(), t["cache"], t["slots"]),
        lambda: kda.latent_cache_append(t["latent"], t["rope"], t["cache"], t["slots"], t["pos"][0]),
        lambda: kda.latent_cache_append(t["latent"], t["rope"], t["cache"][:, ::2], t["slots"]),
        lambda: kda.latent_cache_append(t["latent"], t["rope"][:, :62], t["cache"], t["slots"]),
        lambda: kda.latent_attention_step(t["ql"], t["qr"], t["cache"], t["table"].long(), t["lengths"], 0.1),
        lambda: kda.latent_attention_step(t["ql"], t["qr"], t["cache"], t["table"], t["lengths"][:2], 0.1),
        lambda: kda.latent_attention_step(t["ql"], t["qr"][:, :8], t["cache"], t["table"], t["lengths"], 0.1),
        lambda: kda.latent_attention_step(t["ql"], t["qr"], t["cache"], t["table"], t["lengths"], -0.1),
        lambda: kda.latent_attention_step(t["ql"][..., 1:], t["qr"], t["cache"][..., 1:], t["table"], t["lengths"], 0.1),
        lambda: kda.latent_attention_step(t["ql"], t["qr"], t["cache"], t["table"], t["lengths"], 0.1, o=t["ql"]),
        lambda: kda.latent_attention_fwd(*args[:3], t["v"].float()),
        lambda: kda.latent_attention_fwd(*args[:2], t["kr"][:, 1:], t["v"]),
        lambda: kda.latent_attention_fwd(*args, cu_seqlens_q=t["cu"]),
        lambda: kda.latent_attention_fwd(*args, cu_seqlens_q=t["cu"], cu_seqlens_k=t["cu"][1:]),
        lambda: kda.latent_attention_fwd(*args, scale=0.0),
        lambda: kda.latent_attention_fwd(t["q"][..., 4:], t["k"][..., 4:], t["kr"], t["v"]),
        lambda: kda.latent_attention_fwd(t["q"].expand(2, -1, -1, -1), *(a.expand(2, *a.shape[1:]) for a in args[1:])),
        lambda: kda.latent_attention_bwd(*args, t["go"], t["q"][..., 0], t["go"]),
        lambda: kda.latent_attention_bwd(*args, t["go"], torch.zeros(1, 300, 2, device="cuda"), t["go"], grad_dtype=torch.float16),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, KdaError)):
            call()
            print("accepted", i)


def test_layer_run(kda):
    """A latent attention layer as it is used.  A prompt: projections, rotary positions on queries and the shared key, the cache, attention over
    expanded keys and values, and the gradients through all of it against the same layer in 64 bits by autograd on the
    CPU.  Then single tokens from the cache in the absorbed form, each equal to the longer prompt's last row."""
    import torch
    B, T, more, dim, H, dn, dr, dv, dl, page = 2, 45, 4, 48, 4, 32, 16, 24, 64, 8
    g = torch.Generator().manual_seed(0)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g) * std  # noqa: E731
    P = dict(wq=n(dim, H * (dn + dr), std=dim ** -.5), wc=n(dim, dl + dr, std=dim ** -.5), wkv=n(dl, H * (dn + dv), std=dl ** -.5),
             wo=n(H * dv, dim, std=(H * dv) ** -.5))
    x, gy = n(B, T + more, dim), n(B, T, dim)
    f, fscale = kda.rotary_frequencies(dr, factor=8.0, original_length=64)
    fc = f.double().cpu()

    def turn(a, pos):
        ang = pos.double()[:, None] * fc
        ang = ang if a.dim() == 3 else ang[:, None]
        p, q = a[..., 0::2], a[..., 1::2]
        c, s = torch.cos(ang) * fscale, torch.sin(ang) * fscale
        return torch.stack([p * c - q * s, q * c + p * s], -1).flatten(-2)

    def plain(R, x):
        L = x.shape[1]
        pos = torch.arange(L)
        q = (x @ R["wq"]).view(B, L, H, dn + dr)
        q = torch.cat([q[..., :dn], turn(q[..., dn:], pos)], -1)
        c = x @ R["wc"]
        kr = turn(c[..., dl:], pos)
        kv = (c[..., :dl] @ R["wkv"]).view(B, L, H, dn + dv)
        k = torch.cat([kv[..., :dn], kr[:, :, None].expand(-1, -1, H, -1)], -1)
        s = torch.einsum("bihd,bjhd->bhij", q, k) * (dn + dr) ** -.5
        s = s.masked_fill(torch.ones(L, L, dtype=torch.bool).triu(1), -float("inf"))
        return torch.einsum("bhij,bjhd->bihd", torch.softmax(s, -1), kv[..., dn:]).reshape(B, L, H * dv) @ R["wo"]

    R = {k: v.double().requires_grad_() for k, v in P.items()}
    xd = x[:, :T].double().requires_grad_()
    want = plain(R, xd)
    (want * gy).sum().backward()

    Q = {k: v.cuda() for k, v in P.items()}
    xs, go = x.cuda(), gy.cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda").expand(B, T).contiguous()
    blocks = -(-(T + more) // page)
    cache = torch.full((B * blocks, page, dl + dr), float("nan"), device="cuda")
    table = ints(np.random.default_rng(0).permutation(B * blocks).reshape(B, blocks))
    slots = lambda b, t: table[b, t // page] * page + t % page  # noqa: E731
    q0 = (xs[:, :T] @ Q["wq"]).view(B, T, H, dn + dr)
    q = kda.rotary_fwd(q0, pos, f, True, dn, fscale)
    c = xs[:, :T] @ Q["wc"]
    bi, ti = torch.arange(B, device="cuda").repeat_interleave(T), torch.arange(T, device="cuda").repeat(B)
    flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
    kda.latent_cache_append(flat(c)[:, :dl], flat(c)[:, dl:], cache, slots(bi, ti).to(torch.int32), pos.view(-1), f, True, fscale)
    kr = kda.rotary_fwd(c[:, :, None, dl:], pos, f, True, 0, fscale)[:, :, 0]
    kv = (c[..., :dl] @ Q["wkv"]).view(B, T, H, dn + dv)
    o, lse = kda.latent_attention_fwd(q, kv[..., :dn], kr, kv[..., dn:])
    out = o.reshape(B, T, H * dv) @ Q["wo"]

    grads = dict(wo=flat(o.reshape(B, T, H * dv)).t() @ flat(go))
    dkv = torch.empty_like(kv)
    ga = kda.latent_attention_bwd(q, kv[..., :dn], kr, kv[..., dn:], o, lse, (go @ Q["wo"].t()).view(B, T, H, dv),
                                  out=dict(dq=torch.empty_like(q), dk=dkv[..., :dn], dv=dkv[..., dn:], dk_rope=torch.empty_like(kr)))
    dq = kda.rotary_bwd(ga["dq"], pos, f, True, dn, fscale, grad_x=ga["dq"])
    dc = torch.empty_like(c)
    dc[..., :dl] = dkv.view(B, T, -1) @ Q["wkv"].t()
    dc[..., dl:] = kda.rotary_bwd(ga["dk_rope"][:, :, None], pos, f, True, 0, fscale)[:, :, 0]
    grads.update(wq=flat(xs[:, :T]).t() @ flat(dq.reshape(B, T, -1)), wc=flat(xs[:, :T]).t() @ flat(dc),
                 wkv=flat(c[..., :dl]).t() @ flat(dkv.view(B, T, -1)))
    dx = dq.reshape(B, T, -1) @ Q["wq"].t() + dc @ Q["wc"].t()
    # fp32 through a chain of about 6 operators of about 100 roundings each in the norm
    near = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    assert near(out, want.detach()) < 600 * 2 ** -24
    assert near(dx, xd.grad) < 2400 * 2 ** -24
    for k, v in grads.items():
        assert near(v, R[k].grad) < 2400 * 2 ** -24, (k, near(v, R[k].grad))

    # decoding from the cache; the key's and the value's projections go to the queries and the outputs
    wk, wv = (w.permute(1, 0, 2).contiguous() for w in Q["wkv"].view(dl, H, dn + dv).split([dn, dv], -1))  # [H, dl, .]
    full = plain({k: v.detach() for k, v in R.items()}, x.double())
    for t in range(T, T + more):
        p = torch.full((B,), t, dtype=torch.int32, device="cuda")
        qt = (xs[:, t] @ Q["wq"]).view(B, H, dn + dr)
        kda.rotary_fwd(qt, p, f, True, dn, fscale, y=qt)
        c = xs[:, t] @ Q["wc"]
        kda.latent_cache_append(c[:, :dl], c[:, dl:], cache, slots(torch.arange(B, device="cuda"), p.long()).to(torch.int32), p, f, True, fscale)
        ql = torch.matmul(qt[..., :dn].transpose(0, 1), wk.transpose(1, 2).contiguous()).transpose(0, 1)  # heads in front of rows in memory
        ol, _ = kda.latent_attention_step(ql, qt[..., dn:], cache, table, p + 1, (dn + dr) ** -.5)
        out = torch.matmul(ol.transpose(0, 1), wv).transpose(0, 1).reshape(B, H * dv) @ Q["wo"]
        assert near(out, full[:, t]) < 600 * 2 ** -24, t
