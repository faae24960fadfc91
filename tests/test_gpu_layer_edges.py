"""The operators around the scan at the edges of what they accept: broadcast
rows, non-finite values beside a sequence's end, very long sequences."""
import pytest
import torch

import state_space_model_fwd_gb300 as ssd
from tests import layer_reference as ref

pytestmark = pytest.mark.gpu


# ---- block norm over broadcast rows ----------------------------------------
def norm_calls(t):
    """Forward and gradient over the operands in t, [b, L, dim] each."""
    fwd = ssd.ssd_block_norm_fwd(t["x"], t["weight"], z=t["z"], residual=t["residual"], scale=t["scale"])
    bwd = ssd.ssd_block_norm_bwd(t["dout"], t["x"], t["weight"], z=t["z"], scale=t["scale"], residual_out=t["residual"],
                                 dresidual_out=t["dresidual"])
    return fwd + bwd


@pytest.mark.parametrize("name", ["x", "z", "residual", "dout", "dresidual"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim", [64, 1001])
def test_broadcast_rows_of_the_norm(name, dtype, dim):
    b, L = 4, 8
    g = torch.Generator(device="cuda").manual_seed(dim)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)
    t = {k: rnd(b, L, dim).to(dtype) for k in ("x", "z", "residual", "dout", "dresidual")}
    t["weight"], t["scale"] = rnd(dim), rnd(dim)
    # a row a sequence, a row a token: two strides
    for wide in (rnd(b, 1, dim).to(dtype).expand(b, L, dim), rnd(1, L, dim).to(dtype).expand(b, L, dim)):
        assert 0 in wide.stride()
        with pytest.raises(ValueError, match="one stride"):
            norm_calls(dict(t, **{name: wide}))
        norm_calls(dict(t, **{name: wide.contiguous()}))
    # one row for all: read in place
    wide = rnd(dim).to(dtype).expand(b, L, dim)
    for u, v in zip(norm_calls(dict(t, **{name: wide})), norm_calls(dict(t, **{name: wide.contiguous()}))):
        assert torch.equal(u, v)


# ---- non-finite values at the end of a sequence ----------------------------
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("C", [24, 21])
@pytest.mark.parametrize("cu", [None, [0, 5, 6, 50, 50, 83]], ids=["equal", "packed"])
def test_conv_gradient_where_the_last_token_is_not_finite(value, dtype, C, cu):
    """Without SiLU dp is dy: a value in a sequence's last row reaches dweight's
    last tap alone, and one in its last but one row the last two."""
    b, L, W = (2, 83, 4) if cu is None else (1, 83, 4)
    g = torch.Generator().manual_seed(C)
    n = lambda *s: torch.randn(*s, generator=g)
    x, dy = n(b, L, C), n(b, L, C)
    x[0, 82, 3] = value
    x[0, 81, 5] = value
    if cu:
        x[0, 5, 7], x[0, 49, 9] = value, value
    x, dy = x.to(dtype).cuda(), dy.to(dtype).cuda()
    weight = n(C, W).cuda()
    got = ssd.ssd_conv_bwd(dy, x, weight, silu=False, cu_seqlens=cu)
    leaves = [ref.d(x).requires_grad_(True), ref.d(weight).requires_grad_(True)]
    want = ref.gradients(ref.conv(*leaves, None, None, cu, False), [ref.d(dy), None], leaves)
    assert not bool(torch.isfinite(want[1]).all()) and bool(torch.isfinite(want[1][[3, 5], :2]).all())
    ref.check(got[0], want[0], "dx", rel=1e-5)
    ref.check(got[1], want[1], "dweight", rel=1e-5, scale=float(b * L) ** 0.5 * 3)


SCAN = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "init")


@pytest.mark.parametrize("name", ["x", "B"])
@pytest.mark.parametrize("N", [8, 16, 32])
@pytest.mark.parametrize("cu", [None, [0, 30, 31, 31, 61]], ids=["equal", "packed"])
def test_scan_gradient_where_the_last_token_is_not_finite(name, N, cu):
    """The last token's x or B reaches the last state, and no earlier one: dA,
    which takes the state before each token, stays finite."""
    b, L, ch = (2, 61, 40) if cu is None else (1, 61, 40)
    g = torch.Generator().manual_seed(N)
    n = lambda *s: torch.randn(*s, generator=g)
    nst = b if cu is None else len(cu) - 1
    t = dict(x=n(b, L, ch), dt=0.5 * n(b, L, ch), A=-torch.arange(1, N + 1.0) * torch.exp(0.2 * n(ch, N)), B=n(b, L, 1, N),
             C=n(b, L, 1, N), D=n(ch), z=n(b, L, ch), dt_bias=n(ch) - 3, init=n(nst, ch, N))
    dy, dfin = n(b, L, ch), n(nst, ch, N)
    bad = float("nan") if name == "x" else float("inf")
    for k in [L - 1] if cu is None else [29, L - 1]:
        t[name][0, k].view(-1)[3] = bad
    leaves = [t[k].double().requires_grad_(True) for k in SCAN]
    want = ref.gradients(ref.scan(*leaves, cu), [dy.double(), dfin.double()], leaves)
    assert bool(torch.isfinite(want[2]).all())
    got = ssd.ssd_channel_scan_bwd(dy.cuda(), *[t[k].cuda() for k in SCAN], cu_seqlens=cu, dfinal_state=dfin.cuda())
    for k, a, w in zip(SCAN, got, want):
        ref.check(a, w, "d" + k, rel=3e-5)


# ---- the longest sequence --------------------------------------------------
def test_channel_scan_over_the_longest_sequence():
    """2^31 - 4096 tokens of one channel: the last of 1216 chunks ends less than
    a chunk before 2^31.  One token repeated by stride 0, so the state tends to
    h = delta x B / (1 - exp(delta A)) and stays there."""
    L, N = (1 << 31) - 4096, 8
    x, dt = torch.full((1, 1, 1), 0.75, device="cuda").bfloat16(), torch.zeros(1, 1, 1, device="cuda").bfloat16()
    B, C = (torch.randn(1, 1, 1, N, device="cuda").bfloat16() for _ in range(2))
    A, D = -torch.arange(1.0, N + 1, device="cuda")[None], torch.ones(1, device="cuda")
    y = torch.full((1, L, 1), float("nan"), device="cuda", dtype=torch.bfloat16)
    wide = lambda t: t.expand(1, L, *t.shape[2:])
    _, fin = ssd.ssd_channel_scan_fwd(wide(x), wide(dt), A, wide(B), wide(C), D, y=y)
    delta = torch.log(torch.tensor(2.0, dtype=torch.float64))
    h = delta * 0.75 * B.double().cpu().flatten() / (1 - torch.exp(delta * A.double().cpu().flatten()))
    # relative to h, with 1 / (1 - exp(delta A)) <= 2: the exponential 2.4e-7 and its argument 1e-7, delta 4e-7 through both
    # its uses 7e-7, the roundings of a step 2.4e-7; together 1.3e-6.  256 tokens leave 2^-256 of the start.
    assert float((fin.double().cpu().flatten() - h).abs().max()) <= 2e-6 * float(h.abs().max())
    want = float((h * C.double().cpu().flatten()).sum() + 0.75)
    size = float((h * C.double().cpu().flatten()).abs().sum() + 0.75)
    tail = y[0, 256:, 0]
    lo, hi = float(tail.min()), float(tail.max())  # (a token that was not written is NaN, and so are these)
    bound = 2.0 ** -8 * abs(want) + 4e-6 * size
    assert abs(lo - want) <= bound and abs(hi - want) <= bound, (lo, hi, want)
