"""Layer operators at the largest sizes that one launch takes."""
import pytest

from test_gpu_layer import kda  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def test_norm_of_many_head_rows(kda):
    """More than 2^26 rows of a head's 128 outputs: the same bits as row ranges of it by themselves."""
    import torch
    rows, dim = 2 ** 26 + 7, 128
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.empty(rows, dim, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = 1 + 0.1 * torch.randn(dim, generator=g, device="cuda")
    y = torch.full_like(x, float("nan"))
    kda.layer_norm_fwd(x, w, y=y)
    for a, b in ((0, 1000), (2 ** 25 - 5, 2 ** 25 + 1000), (rows - 1003, rows)):
        assert torch.equal(y[a:b], kda.layer_norm_fwd(x[a:b].clone(), w)), a
    assert not any(bool(part.isnan().any()) for part in y.split(1 << 22))


def test_conv_of_many_rows(kda):
    """2^27 rows and more of few channels: the same bits as two calls, the second from the state that the first leaves."""
    import torch
    T, dim, cut = 2 ** 27 + 1003, 12, 2 ** 26 + 13
    g = torch.Generator("cuda").manual_seed(2)
    x, gy = (torch.empty(1, T, dim, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    w, b = torch.randn(dim, 4, generator=g, device="cuda"), torch.randn(dim, generator=g, device="cuda")
    y, final = kda.short_conv_fwd(x, w, b, silu=True)
    y0, state = kda.short_conv_fwd(x[:, :cut], w, b, silu=True)
    y1, state = kda.short_conv_fwd(x[:, cut:], w, b, initial_state=state, silu=True)
    assert torch.equal(y[:, :cut], y0) and torch.equal(y[:, cut:], y1) and torch.equal(final, state)
    del y, y0, y1
    # rows far from the cut get their gradient from rows near them alone
    got = kda.short_conv_bwd(x, w, gy, b, silu=True, grad_dtype=torch.bfloat16)["dx"]
    for a, e in ((0, 5000), (cut - 2500, cut + 2500), (T - 5000, T)):
        part = kda.short_conv_bwd(x[:, a:e], w, gy[:, a:e], b, silu=True, initial_state=x[:, a - 3:a].clone() if a else None,
                                  grad_dtype=torch.bfloat16)["dx"]
        keep = part.shape[1] if e == T else part.shape[1] - 3  # the last three also reach rows behind
        assert torch.equal(got[:, a:a + keep], part[:, :keep]), a
