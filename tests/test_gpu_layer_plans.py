"""The operators around the scan at sizes whose plans small cases do not reach:
rows run whole beside rows cut into chunks, blocks that walk several chunks,
tiles or rows, the pass over chunks by single warps, long tiles.  Expected
values are the float64 definitions, or small calls bit for bit."""
import ctypes

import pytest
import torch

import state_space_model_fwd_gb300 as ssd
from state_space_model_fwd_gb300 import _layer
from tests import layer_reference as ref
from tests import test_gpu_block_norm as norm_tests
from tests import test_gpu_channel_scan as scan_tests

pytestmark = pytest.mark.gpu
SMS = 152


# ---- channel scan, forward -------------------------------------------------
def scan_workspace(t):
    b, L, ch = t["x"].shape
    shape = _layer._channel_shape_t(b, L, ch, t["B"].shape[3], t["B"].shape[2], 1 if t["x"].dtype == torch.bfloat16 else 0, 1)
    lib = ssd.load_library()
    return lib.ssd_channel_scan_workspace_size(ctypes.byref(shape), None, 0)


# A block row is 32 channels of a batch row; two for each of the 608 schedulers run whole.
@pytest.mark.parametrize("dtype,b,L,ch,N,gate,cut", [
    ("f32", 40, 70, 1024, 16, True, 64),     # 1280: 1216 whole, 64 cut into two chunks
    ("bf16", 40, 70, 1024, 8, False, 64),
    ("f32", 77, 67, 520, 32, True, 93),      # 17 block rows of 32 or 8 channels each: 1309
    ("f32", 44, 9, 1280, 8, True, 0),        # 1760: what is left over would fill 7/8 of the schedulers
    ("bf16", 152, 5, 1024, 8, True, 0),      # 4864: eight for every scheduler
])
def test_scan_rows_whole_and_cut(dtype, b, L, ch, N, gate, cut):
    t = scan_tests.make(dtype, b, L, ch, N, gate=gate, seed=21)
    chunk = -(-(-(-L // 2)) // 8) * 8
    states = cut * -(-L // chunk) * 32 * 4
    assert scan_workspace(t) == (-(-states * N // 256) + -(-states // 256)) * 256
    y, fin = ssd.ssd_channel_scan_fwd(*scan_tests.args_of(t))
    # up to 64 tokens of few block rows are one pass each (held to the definition elsewhere): the same arithmetic in the
    # same order, so the same bits; a row in two chunks starts the second from the first one's state itself
    for r in range(0, b, 30):
        state = t["init"][r:r + 30]
        for k in range(0, L, 64):
            part = dict(t, init=state.contiguous())
            for name in ("x", "dt", "B", "C", "z"):
                part[name] = None if t[name] is None else t[name][r:r + 30, k:k + 64]
            assert scan_workspace(part) == 0
            yk, state = ssd.ssd_channel_scan_fwd(*scan_tests.args_of(part))
            assert torch.equal(y[r:r + 30, k:k + 64], yk)
        assert torch.equal(fin[r:r + 30], state)


# ---- channel scan, gradient ------------------------------------------------
# Blocks of 128 channels, two an SM in all, share a group's chunks of 32 (8 states), 28 (16) or 16 tokens (32 states);
# single warps pass over the chunks where 304 of them have work.
@pytest.mark.parametrize("dtype,b,L,ch,N,cu", [
    ("f32", 3, 400, 1024, 16, None),                              # 45 chunks on 38 blocks a quad, 384 warps in the pass
    ("bf16", 1, 500, 2464, 16, [0, 3, 3, 150, 151, 500]),         # 18 on 15, 308 warps, packed
    ("f32", 2, 330, 640, 32, None),                               # 42 on 60: one each, 320 warps
    ("f32", 1, 4900, 100, 32, [0, 1, 17, 2000, 2000, 4900]),      # 307 on 304, eight warps a pass over 307 chunks
])
def test_scan_gradient_walks_several_chunks(dtype, b, L, ch, N, cu):
    t = scan_tests.make(dtype, b, L, ch, N, cu=cu, seed=22)
    nst = b if cu is None else len(cu) - 1
    g = torch.Generator().manual_seed(23)
    dy = torch.randn(b, L, ch, generator=g).to(t["x"].dtype)
    dfin = 0.3 * torch.randn(nst, ch, N, generator=g)
    got = ssd.ssd_channel_scan_bwd(dy.cuda(), *scan_tests.args_of(t), cu_seqlens=cu, dfinal_state=dfin.cuda())
    leaves = [ref.d(t[k]).requires_grad_(True) for k in scan_tests.NAMES]
    want = ref.gradients(ref.scan(*leaves, cu), [dy.double(), dfin.double()], leaves)
    for name, a, w in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dinit"), got, want):
        # (the small cases' bound: the sums over tokens are of at most 60 terms, then of at most 304 partial sums, whose
        # roundings of 2^-24 of a partial sum stay below 3e-5 of the result's size even if all have one sign)
        ref.check(a, w, name, rel=3e-5)


# ---- block norm, gradient --------------------------------------------------
# A team walks the rows of its columns: 12 warps an SM up to 512 columns, else blocks of 512 columns a warp, 15 warps an SM.
@pytest.mark.parametrize("case", [
    (dtype, rows, dim, group, gate, residual, True, pad)
    for dtype in ("f32", "bf16") for gate in ("none", "before", "after")
    for rows, dim, group, residual, pad in [
        (2500, 256, 128, "f32", 0),      # 912 warp teams: two or three rows each
        (2500, 1024, 1024, None, 0),     # 1064 blocks
        (2200, 1001, 1001, "f32", 0),    # odd columns, one value at a time
        (400, 10240, 10240, None, 0),    # 152 blocks of the widest kind
        (331, 5120, 5120, "f32", 8),     # 152 blocks: two rows each, one block in nine three
    ]], ids=lambda c: "-".join(str(v) for v in c))
def test_norm_gradient_walks_several_rows(case):
    dtype, rows, dim, group = case[:4]
    warps = -(-group // 512)
    assert rows > SMS * (12 if warps == 1 else max(15 // warps, 1)) // (dim // group)
    norm_tests.test_gradient(case)


# ---- convolution -----------------------------------------------------------
def conv_reference(x, weight, bias, init, cu):
    """One product over windows for every sequence, on the GPU."""
    ys, finals = [], []
    W = weight.shape[1]
    for s, r, lo, hi in ref.spans(x.shape[0], x.shape[1], cu):
        line = torch.cat([init[s], x[r, lo:hi]])
        if hi > lo:
            ys.append(ref.silu(sum(line[k:k + hi - lo] * weight[:, k] for k in range(W)) + bias))
        finals.append(line[hi - lo:])
    return torch.cat(ys).reshape(x.shape), torch.stack(finals)


def conv_case(dtype, b, L, C, W, cu):
    g = torch.Generator(device="cuda").manual_seed(L)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)
    nst = b if cu is None else len(cu) - 1
    return n(b, L, C).to(dtype), n(C, W) / W ** 0.5, 0.1 * n(C), n(nst, W - 1, C).to(dtype)


# The longest tile of 8 to 128 tokens that leaves 16 warps an SM, of 128 channels each (32 where rows are not aligned).
@pytest.mark.parametrize("tile,dtype,b,L,C,W,cu", [
    (16, torch.bfloat16, 1, 2500, 2048, 4, None),
    (32, torch.float32, 2, 2499, 2048, 3, None),
    (64, torch.bfloat16, 1, 9733, 2048, 4, [0, 1, 65, 65, 4000, 4003, 9733]),
    (128, torch.bfloat16, 3, 6501, 2048, 2, None),
    (128, torch.float32, 1, 4900, 2047, 4, [0, 129, 2000, 2002, 4899, 4900]),
])
def test_conv_tiles(tile, dtype, b, L, C, W, cu):
    blocks = -(-(C // 4 if C % 8 == 0 else C) // 32)
    assert blocks * (b * L // tile) >= SMS * 16 and (tile == 128 or blocks * (b * L // (2 * tile)) < SMS * 16)
    t = conv_case(dtype, b, L, C, W, cu)
    y, fin = ssd.ssd_conv_fwd(*t, cu_seqlens=cu)
    want, wfin = conv_reference(*[v.double() for v in t], cu)
    ref.check(y, want.cpu(), "y", rel=4e-6)  # (as in the tests of the small cases)
    assert torch.equal(fin.double(), wfin)


# Two blocks an SM in all, of eight warps, walk tiles of 32 to 256 tokens.
@pytest.mark.parametrize("dtype,b,L,C,W,cu", [
    (torch.bfloat16, 100, 33, 2048, 4, None),                               # 200 tiles on 152 warps a channel block
    (torch.float32, 1, 8500, 2047, 4, [0, 1, 300, 300, 302, 8000, 8500]),   # 64 tiles of 133 on 32 warps
    (torch.float32, 2, 4300, 2047, 3, None),
])
def test_conv_gradient_walks_several_tiles(dtype, b, L, C, W, cu):
    t = conv_case(dtype, b, L, C, W, cu)
    g = torch.Generator(device="cuda").manual_seed(31)
    dy = torch.randn(b, L, C, device="cuda", generator=g).to(dtype)
    dfin = torch.randn(t[3].shape, device="cuda", generator=g).to(dtype)
    got = ssd.ssd_conv_bwd(dy, *t, cu_seqlens=cu, dfinal_state=dfin)
    leaves = [v.double().requires_grad_(True) for v in t]
    want = torch.autograd.grad(conv_reference(*leaves, cu), leaves, [dy.double(), dfin.double()])
    for name, a, w in zip(("dx", "dweight", "dbias", "dinit"), got, want):
        # (as in the tests of the small cases: sums over the tokens of terms of size 1)
        ref.check(a, w.cpu(), name, rel=1e-5, scale=3 * (b * L) ** 0.5 if name in ("dweight", "dbias") else None)


# ---- softplus --------------------------------------------------------------
def test_softplus_by_itself():
    """One token from a zero state with x = B = 1: the state is delta."""
    v = torch.cat([torch.linspace(-80, 30, 4001), torch.linspace(-1, 1, 999)]).cuda()
    ch = v.numel()
    one, A = torch.ones(1, 1, ch, device="cuda"), -torch.ones(ch, 8, device="cuda")
    B = torch.ones(1, 1, 1, 8, device="cuda")
    _, fin = ssd.ssd_channel_scan_fwd(one, v.view(1, 1, ch), A, B, B)
    d, exact = fin[0, :, 0].double(), torch.nn.functional.softplus(v.double(), threshold=1e3)
    assert torch.equal(fin[0], fin[0, :, :1].expand(ch, 8))
    # exp(-|v|): the product with log2(e) is rounded, 2^-24 + 1.3e-8 (the constant) of |v|; the exponential 2.4e-7; the
    # reciprocal, the polynomial and the last roundings 4e-7
    off = ((d - exact).abs() / exact).cpu()
    bound = 8e-7 + 8e-8 * v.double().abs().cpu()
    assert bool((off <= bound).all()), (v.cpu()[off > bound][:5], off[off > bound][:5])
    # the plain composition in fp32, where it is accurate
    plain = torch.log1p(torch.exp(v[v < 10])).double()
    assert bool(((d[v < 10] - plain).abs() <= (bound.cuda()[v < 10] + 4e-7 + 1.2e-7 * v[v < 10].abs()) * plain).all())
