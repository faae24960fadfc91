"""Strided operands of the operators around the scan: views into wider, longer
NaN-filled arrays give bit for bit what contiguous tensors give (nothing
outside a view is read), whatever the alignment; and the ``stream`` argument."""
import pytest
import torch

import state_space_model_fwd_gb300 as ssd

pytestmark = pytest.mark.gpu


def view(t, pad, at, longer=0):
    """The same values in a view whose rows lie among NaNs."""
    if t is None:
        return None
    b, L = t.shape[:2]
    n = t[0, 0].numel()
    w = torch.full((b, L + longer, n + pad), float("nan"), device="cuda", dtype=t.dtype)
    v = w[:, :L, at:at + n]
    v.copy_(t.reshape(b, L, n))
    return v.unflatten(-1, t.shape[2:]) if t.dim() == 4 else v


def same(a, b):
    for x, y in zip(a, b):
        if x is None:
            assert y is None
        else:
            assert torch.equal(x, y) and bool(torch.isfinite(x).all())


VIEWS = [(1, 1, 0), (3, 0, 2), (8, 8, 0), (16, 8, 5), (41, 13, 1)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,at,longer", VIEWS)
def test_channel_scan(dtype, pad, at, longer):
    g = torch.Generator(device="cuda").manual_seed(pad)
    rnd = lambda *s, ty=dtype: torch.randn(*s, device="cuda", generator=g).to(ty)
    b, L, G, N, ch = 3, 61, 2, 16, 80
    f32 = torch.float32
    x, z, dy = (rnd(b, L, ch) for _ in range(3))
    dt = (0.5 * rnd(b, L, ch)).to(dtype)
    A, B, C = -8 * torch.rand(ch, N, device="cuda", generator=g), rnd(b, L, G, N), rnd(b, L, G, N)
    D, bias, init = rnd(ch, ty=f32), rnd(ch, ty=f32) - 3, rnd(b, ch, N, ty=f32)
    w = lambda t: view(t, pad, at, longer)
    plain, strided = (x, dt, A, B, C, D, z, bias, init), (w(x), w(dt), A, w(B), w(C), D, w(z), bias, init)
    same(ssd.ssd_channel_scan_fwd(*plain), ssd.ssd_channel_scan_fwd(*strided))
    same(ssd.ssd_channel_scan_bwd(dy, *plain), ssd.ssd_channel_scan_bwd(w(dy), *strided))
    out = torch.full((b, L + longer, ch + pad), 9.0, device="cuda", dtype=dtype)
    y, _ = ssd.ssd_channel_scan_fwd(*strided, y=out[:, :L, at:at + ch])
    assert torch.equal(y, ssd.ssd_channel_scan_fwd(*plain)[0])
    assert bool((out[:, :, :at] == 9).all()) and bool((out[:, :, at + ch:] == 9).all()) and bool((out[:, L:] == 9).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,at,longer", VIEWS)
def test_convolution(dtype, pad, at, longer):
    g = torch.Generator(device="cuda").manual_seed(pad)
    rnd = lambda *s, ty=dtype: torch.randn(*s, device="cuda", generator=g).to(ty)
    x, dy, init = rnd(2, 45, 72), rnd(2, 45, 72), rnd(2, 3, 72)
    weight, bias = rnd(72, 4, ty=torch.float32), rnd(72, ty=torch.float32)
    w = lambda t: view(t, pad, at, longer)
    same(ssd.ssd_conv_fwd(x, weight, bias, init), ssd.ssd_conv_fwd(w(x), weight, bias, init))
    a, b = (ssd.ssd_conv_bwd(*gx, weight, bias, init) for gx in ((dy, x), (w(dy), w(x))))
    same((a[0], a[3]), (b[0], b[3]))
    for u, v in zip(a[1:3], b[1:3]):  # other tiles, other partial sums: 90 terms of size 1
        assert float((u - v).abs().max()) <= 1e-4


def test_broadcast_rows_are_read_in_place():
    """B and C shared by the batch as stride-0 views."""
    x, dt = torch.randn(4, 30, 32, device="cuda"), torch.randn(4, 30, 32, device="cuda") - 2
    B, C = torch.randn(1, 30, 1, 16, device="cuda"), torch.randn(1, 30, 1, 16, device="cuda")
    A = -torch.rand(32, 16, device="cuda")
    wide = [t.expand(4, 30, 1, 16) for t in (B, C)]
    same(ssd.ssd_channel_scan_fwd(x, dt, A, *wide), ssd.ssd_channel_scan_fwd(x, dt, A, *[t.contiguous() for t in wide]))


def test_stream_argument():
    s = torch.cuda.Stream()
    x, weight = torch.randn(2, 64, 96, device="cuda"), torch.randn(96, 4, device="cuda")
    norm = torch.ones(96, device="cuda")
    want = ssd.ssd_conv_fwd(x, weight)[0]
    want2 = ssd.ssd_block_norm_fwd(want, norm)[0]
    torch.cuda.synchronize()
    y, _ = ssd.ssd_conv_fwd(x, weight, stream=s)
    out, _ = ssd.ssd_block_norm_fwd(y, norm, stream=s)
    s.synchronize()
    assert torch.equal(y, want) and torch.equal(out, want2)


def test_captured_in_a_graph():
    """One token's calls replayed: the states move on with every replay."""
    b, ch = 2, 64
    x, dt = torch.randn(b, ch, device="cuda"), torch.randn(b, ch, device="cuda") - 2
    A, B, C = -torch.rand(ch, 16, device="cuda"), torch.randn(b, 1, 16, device="cuda"), torch.randn(b, 1, 16, device="cuda")
    weight = torch.randn(ch, 4, device="cuda")
    conv, state = torch.zeros(b, 3, ch, device="cuda"), torch.zeros(b, ch, 16, device="cuda")

    def step():
        return ssd.ssd_channel_scan_step(ssd.ssd_conv_step(x, weight, state=conv), dt, A, B, C, state=state)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    conv.zero_(), state.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    conv.zero_(), state.zero_()
    got = []
    for _ in range(4):
        graph.replay()
        got.append(y.clone())
    after = state.clone()
    conv.zero_(), state.zero_()
    for k in range(4):
        assert torch.equal(step(), got[k])
    assert torch.equal(state, after)
