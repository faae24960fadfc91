"""The short causal convolution on the GPU against its definition in float64:
prompts (equal lengths and packed), gradients, one token at a time."""
import ctypes

import pytest
import torch

import state_space_model_fwd_gb300 as ssd
from tests import layer_reference as ref

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(dtype, b, L, C, W, cu=None, bias=True, init=False, row=0, at=0, seed=0, dev="cuda"):
    g = torch.Generator().manual_seed(seed * 131 + C + L)
    n = lambda *s: torch.randn(*s, generator=g)
    nst = b if cu is None else len(cu) - 1
    row = row or C
    x = n(b, L, row).to(DT[dtype]).to(dev)[:, :, at:at + C]
    return dict(x=x, weight=(n(C, W) / W ** 0.5).to(dev), bias=(0.1 * n(C)).to(dev) if bias else None,
                init=n(nst, W - 1, C).to(DT[dtype]).to(dev) if init else None)


# (dtype, b, L, C, W, offsets, bias, init, row width, first column)
CASES = [
    ("bf16", 2, 37, 64, 4, None, True, True, 0, 0),
    ("bf16", 1, 1, 8, 4, None, True, False, 0, 0),              # one token, shorter than the window
    ("bf16", 3, 2, 16, 4, None, False, True, 0, 0),             # two tokens: the final state keeps an initial row
    ("f32", 2, 70, 36, 3, None, True, True, 0, 0),
    ("f32", 1, 129, 257, 2, None, True, False, 0, 0),           # odd channels: one element a lane
    ("bf16", 1, 300, 1792, 4, None, True, False, 3352, 1536),   # a slice of a wider projection
    ("bf16", 1, 65, 48, 3, None, True, True, 65, 1),            # unaligned slice
    ("bf16", 1, 100, 64, 4, [0, 0, 1, 3, 3, 40, 97, 100, 100], True, True, 0, 0),
    ("f32", 1, 33, 20, 4, [0, 33], False, False, 0, 0),
    ("bf16", 1, 515, 40, 4, [0] + list(range(3, 516, 2)) + [515], True, True, 0, 0),
    ("f32", 1, 0, 8, 4, [0, 0, 0], True, True, 0, 0),           # nothing but empty sequences
    ("f32", 2, 0, 8, 3, None, True, True, 0, 0),
]
IDS = [f"{c[0]}-b{c[1]}-L{c[2]}-C{c[3]}-W{c[4]}{'-packed' if c[5] else ''}" for c in CASES]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("act", [True, False])
def test_forward(case, act):
    dtype, b, L, C, W, cu, bias, init, row, at = case
    t = make(dtype, b, L, C, W, cu, bias, init, row, at)
    y, fin = ssd.ssd_conv_fwd(t["x"], t["weight"], t["bias"], t["init"], silu=act, cu_seqlens=cu)
    want, wfin = ref.conv(*[ref.d(t[k]) for k in ("x", "weight", "bias", "init")], cu, act)
    # W + 1 roundings of sums of W terms of size 1, and the exponential's 2^-21
    ref.check(y, want, "y", rel=4e-6)
    assert torch.equal(fin.double().cpu(), wfin), "the final state is a copy"


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_gradient(case):
    dtype, b, L, C, W, cu, bias, init, row, at = case
    t = make(dtype, b, L, C, W, cu, bias, init, row, at, seed=1)
    g = torch.Generator().manual_seed(5)
    dy = torch.randn(b, L, C, generator=g).to(DT[dtype]).cuda()
    nst = b if cu is None else len(cu) - 1
    dfin = torch.randn(nst, W - 1, C, generator=g).to(DT[dtype]).cuda() if init else None
    got = ssd.ssd_conv_bwd(dy, t["x"], t["weight"], t["bias"], t["init"], cu_seqlens=cu, dfinal_state=dfin)
    leaves = [ref.d(t[k]) for k in ("x", "weight", "bias", "init")]
    for v in leaves:
        if v is not None:
            v.requires_grad_(True)
    out = ref.conv(*leaves, cu)
    want = ref.gradients(out, [ref.d(dy), ref.d(dfin)], leaves)
    for name, a, w in zip(("dx", "dweight", "dbias", "dinit"), got, want):
        # sums over the tokens: up to a few hundred additions one after another, of terms of size 1
        s = None if not name.startswith("dw") and name != "dbias" else float(max(b * L, 1)) ** 0.5 * 3
        ref.check(a, w, name, rel=1e-5, scale=s)


@pytest.mark.gpu
def test_parts_are_the_columns_of_one_output():
    t = make("bf16", 2, 77, 128, 4, seed=2, row=200, at=40)
    y, fin = ssd.ssd_conv_fwd(t["x"], t["weight"], t["bias"])
    ys, fin2 = ssd.ssd_conv_fwd(t["x"], t["weight"], t["bias"], split=[64, 32, 32])
    assert torch.equal(torch.cat(ys, -1), y) and torch.equal(fin, fin2)
    assert all(v.is_contiguous() for v in ys)
    odd, _ = ssd.ssd_conv_fwd(t["x"], t["weight"], t["bias"], split=[61, 1, 63, 3])
    assert torch.equal(torch.cat(odd, -1), y)
    dy = torch.randn(2, 77, 128, device="cuda").bfloat16()
    one = ssd.ssd_conv_bwd(dy, t["x"], t["weight"], t["bias"])
    parts = ssd.ssd_conv_bwd(list(dy.split([64, 32, 32], -1)), t["x"], t["weight"], t["bias"])
    for a, b in zip(one, parts):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.gpu
def test_gradient_goes_into_a_slice():
    t = make("bf16", 2, 50, 64, 4, seed=3)
    dy = torch.randn(2, 50, 64, device="cuda").bfloat16()
    wide = torch.full((2, 50, 96), 7.0, device="cuda", dtype=torch.bfloat16)
    dx, *_ = ssd.ssd_conv_bwd(dy, t["x"], t["weight"], t["bias"], dx=wide[:, :, 16:80])
    plain, *_ = ssd.ssd_conv_bwd(dy, t["x"], t["weight"], t["bias"])
    assert torch.equal(dx, plain)
    assert bool((wide[:, :, :16] == 7).all()) and bool((wide[:, :, 80:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,C,W", [("bf16", 64, 4), ("f32", 37, 3), ("bf16", 1792, 2)])
def test_tokens_one_by_one_are_the_prompt(dtype, C, W):
    t = make(dtype, 3, 9, C, W, init=True, seed=4)
    y, fin = ssd.ssd_conv_fwd(t["x"], t["weight"], t["bias"], t["init"])
    state = t["init"].clone()
    for k in range(9):
        yk = ssd.ssd_conv_step(t["x"][:, k], t["weight"], t["bias"], state=state)
        ref.check(yk, ref.d(y[:, k]), f"token {k}", rel=2e-6 if dtype == "f32" else 2.0 ** -8)
    assert torch.equal(state, fin)


@pytest.mark.gpu
def test_gradient_agrees_with_differences():
    t = make("f32", 1, 41, 24, 4, [0, 7, 30, 41], True, True, seed=6)
    cu = [0, 7, 30, 41]
    g = torch.Generator(device="cuda").manual_seed(9)
    dy = torch.randn(1, 41, 24, device="cuda", generator=g)
    grads = ssd.ssd_conv_bwd(dy, t["x"], t["weight"], t["bias"], t["init"], cu_seqlens=cu)
    for i, k in enumerate(("x", "weight", "bias", "init")):
        v = torch.randn(t[k].shape, device="cuda", generator=g)
        vals = []
        for e in (1e-2, -1e-2):
            u = dict(t, **{k: (t[k] + e * v).contiguous()})
            y, _ = ssd.ssd_conv_fwd(u["x"], u["weight"], u["bias"], u["init"], cu_seqlens=cu)
            vals.append((y.double() * dy.double()).sum())
        slope = float(vals[0] - vals[1]) / 2e-2
        # truncation 1e-4 f''' and fp32 rounding of y over the step, both below 1e-3 of |v| |grad|
        size = float((grads[i].double().norm() * v.double().norm()))
        assert abs(slope - float((grads[i].double() * v.double()).sum())) <= 1e-3 * size, k


@pytest.mark.gpu
def test_nothing_crosses_a_boundary():
    """A non-finite row stays within its sequence, forward and backward."""
    t = make("f32", 1, 60, 32, 4, seed=7)
    cu = [0, 20, 21, 60]
    x = t["x"].clone()
    x[0, 20] = float("nan")
    x[0, 19, 3] = float("inf")
    y, _ = ssd.ssd_conv_fwd(x, t["weight"], t["bias"], cu_seqlens=cu)
    clean, _ = ssd.ssd_conv_fwd(t["x"], t["weight"], t["bias"], cu_seqlens=cu)
    assert torch.equal(y[0, :19], clean[0, :19]) and torch.equal(y[0, 21:], clean[0, 21:])
    dy = torch.randn_like(x)
    dx, *_ = ssd.ssd_conv_bwd(dy, x, t["weight"], t["bias"], cu_seqlens=cu)
    dclean, *_ = ssd.ssd_conv_bwd(dy, t["x"], t["weight"], t["bias"], cu_seqlens=cu)
    assert torch.equal(dx[0, :16], dclean[0, :16]) and torch.equal(dx[0, 21:], dclean[0, 21:])


@pytest.mark.gpu
def test_more_sequences_than_one_launch_holds():
    lens = torch.randint(0, 4, (2500,), generator=torch.Generator().manual_seed(3)).tolist()
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    t = make("f32", 1, cu[-1], 8, 3, cu, True, True, seed=8)
    y, fin = ssd.ssd_conv_fwd(t["x"], t["weight"], t["bias"], t["init"], cu_seqlens=cu)
    leaves = [ref.d(t[k]).requires_grad_(True) for k in ("x", "weight", "bias", "init")]
    out = ref.conv(*leaves, cu)
    ref.check(y, out[0], "y", rel=4e-6)
    assert torch.equal(fin.double().cpu(), out[1])
    dy, dfin = torch.randn_like(t["x"]), torch.randn_like(fin)
    got = ssd.ssd_conv_bwd(dy, t["x"], t["weight"], t["bias"], t["init"], cu_seqlens=cu, dfinal_state=dfin)
    want = ref.gradients(out, [ref.d(dy), ref.d(dfin)], leaves)
    for name, a, w in zip(("dx", "dweight", "dbias", "dinit"), got, want):
        ref.check(a, w, name, rel=1e-5, scale=200.0 if name in ("dweight", "dbias") else None)


@pytest.mark.gpu
def test_runs_on_the_given_stream_and_repeats_bitwise():
    t = make("bf16", 4, 333, 256, 4, seed=9)
    dy = torch.randn(4, 333, 256, device="cuda").bfloat16()
    first = ssd.ssd_conv_bwd(dy, t["x"], t["weight"], t["bias"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = ssd.ssd_conv_bwd(dy, t["x"], t["weight"], t["bias"])
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(first, again):
        assert (a is None and b is None) or torch.equal(a, b)


# ---- refusals (host only) --------------------------------------------------
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from state_space_model_fwd_gb300 import _build
    _build.build()
    return ssd.load_library()


def c_shape(**kw):
    from state_space_model_fwd_gb300 import _layer
    v = dict(batch=1, seqlen=64, channels=64, width=4, parts=[64], dtype=1, silu=1)
    v.update(kw)
    parts = v.pop("parts")
    return _layer._conv_shape_t(v["batch"], v["seqlen"], v["channels"], v["width"], len(parts),
                                (ctypes.c_int64 * 4)(*parts[:4]), v["dtype"], v["silu"])


def c_rows(ptr=FAKE, bs=64 * 64, rs=64):
    from state_space_model_fwd_gb300 import _layer
    return _layer._rows_t(ptr, bs, rs)


def c_fwd(lib, shape, cu=None, x=None, y=None, w=FAKE):
    x, y = x or c_rows(), y or c_rows()
    arr = (ctypes.c_int64 * len(cu))(*cu) if cu else None
    return lib.ssd_conv_fwd(ctypes.byref(shape), arr, len(cu) - 1 if cu else 0, ctypes.byref(x), w, None, None,
                            ctypes.byref(y), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(width=5), UNSUPPORTED), (dict(width=1), UNSUPPORTED), (dict(width=0), INVALID), (dict(channels=0), INVALID),
    (dict(batch=-1), INVALID), (dict(dtype=7), INVALID), (dict(parts=[32, 31]), INVALID), (dict(parts=[64, 0]), INVALID),
    (dict(parts=[]), INVALID), (dict(seqlen=1 << 31), UNSUPPORTED),
])
def test_shapes_are_checked(lib, kw, code):
    assert c_fwd(lib, c_shape(**kw)) == code
    assert lib.ssd_conv_bwd_workspace_size(ctypes.byref(c_shape(**kw)), None, 0) == 0


def test_pointers_strides_and_offsets_are_checked(lib):
    s = c_shape()
    assert c_fwd(lib, s, w=None) == INVALID
    assert c_fwd(lib, s, x=c_rows(ptr=None)) == INVALID
    assert c_fwd(lib, s, x=c_rows(ptr=FAKE + 1)) == INVALID          # not aligned to its element
    assert c_fwd(lib, s, y=c_rows(rs=63)) == INVALID                 # rows that overlap
    assert c_fwd(lib, c_shape(batch=2), y=c_rows(bs=100)) == INVALID
    for cu in ([0, 10, 5, 64], [1, 64], [0, 63]):
        assert c_fwd(lib, s, cu=cu) == INVALID
    assert c_fwd(lib, c_shape(batch=2), cu=[0, 64]) == INVALID
    assert c_fwd(lib, c_shape(batch=0)) == OK
    r = c_rows()
    need = lib.ssd_conv_bwd_workspace_size(ctypes.byref(s), None, 0)
    assert need > 0
    args = [ctypes.byref(r), ctypes.byref(r), FAKE, None, None, None, ctypes.byref(r), FAKE, None, None]
    assert lib.ssd_conv_bwd(ctypes.byref(s), None, 0, *args, FAKE, need - 1, None) == WORKSPACE
    assert lib.ssd_conv_bwd(ctypes.byref(s), None, 0, *args, None, 0, None) == WORKSPACE
    assert lib.ssd_conv_step(ctypes.byref(c_shape(parts=[32, 32])), ctypes.byref(r), FAKE, None, FAKE, ctypes.byref(r),
                             None) == INVALID


def test_binding_refuses(lib):
    x = torch.zeros(1, 8, 16)
    with pytest.raises(TypeError):
        ssd.ssd_conv_fwd(x, torch.zeros(16, 4))
    with pytest.raises(TypeError):
        ssd.ssd_conv_step(x[:, 0], torch.zeros(16, 4), state=torch.zeros(1, 3, 16))


@pytest.mark.gpu
def test_binding_refuses_on_the_gpu():
    t = make("f32", 2, 8, 16, 4, init=True)
    with pytest.raises(ValueError):
        ssd.ssd_conv_fwd(t["x"], t["weight"][:8].contiguous(), t["bias"])
    with pytest.raises(ValueError):
        ssd.ssd_conv_fwd(t["x"].transpose(1, 2), t["weight"][:8].contiguous())
    with pytest.raises(TypeError):
        ssd.ssd_conv_fwd(t["x"].half(), t["weight"])
    with pytest.raises(ValueError):
        ssd.ssd_conv_fwd(t["x"], t["weight"], t["bias"], t["init"], final_state=t["init"])
    with pytest.raises(ssd.SSDError):
        ssd.ssd_conv_fwd(t["x"], t["weight"], split=[8, 9])
    with pytest.raises(ssd.SSDError):
        ssd.ssd_conv_fwd(t["x"][:1], t["weight"], cu_seqlens=[0, 9])
