"""The channel scan on the GPU against its definition in float64: prompts
(equal lengths and packed), gradients, one token at a time."""
import ctypes

import pytest
import torch

import state_space_model_fwd_gb300 as ssd
from tests import layer_reference as ref

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NAMES = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "init")


def make(dtype, b, L, ch, N, G=1, cu=None, gate=True, init=True, skip=True, bias=True, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed * 1009 + ch * 7 + L)
    n = lambda *s: torch.randn(*s, generator=g)
    ty = DT[dtype]
    nst = b if cu is None else len(cu) - 1
    rows = lambda w: n(b, L, w + pad).to(ty).cuda()[:, :, pad:]
    u = torch.exp(torch.rand(ch, generator=g) * 4.6 - 6.9)
    t = dict(x=rows(ch), dt=(0.5 * rows(ch).float()).to(ty), A=-torch.arange(1, N + 1.0) * torch.exp(0.2 * n(ch, N)),
             B=rows(G * N).unflatten(-1, (G, N)), C=rows(G * N).unflatten(-1, (G, N)),
             D=1 + 0.1 * n(ch) if skip else None, z=rows(ch) if gate else None,
             dt_bias=u + torch.log(-torch.expm1(-u)) if bias else None,
             init=0.3 * n(nst, ch, N) if init else None)
    if not bias:
        t["dt"] = t["dt"] - 3
    return {k: None if v is None else v.cuda() for k, v in t.items()}


# (dtype, b, L, channels, N, G, offsets, gate, init, skip, bias, columns before)
CASES = [
    ("f32", 1, 1, 32, 16, 1, None, True, True, True, True, 0),
    ("f32", 2, 37, 40, 16, 1, None, True, True, True, True, 0),        # a block with 8 channels
    ("bf16", 2, 75, 64, 16, 2, None, True, False, True, True, 0),      # two groups
    ("bf16", 1, 333, 33, 16, 1, None, False, True, True, True, 3),     # several chunks, odd columns, no gate
    ("f32", 1, 200, 96, 8, 3, None, True, True, False, False, 0),
    ("f32", 1, 150, 64, 32, 1, None, True, True, True, True, 0),
    ("bf16", 1, 90, 48, 32, 2, None, False, False, True, True, 0),
    ("f32", 1, 300, 64, 16, 1, [0, 0, 1, 2, 70, 128, 128, 192, 300, 300], True, True, True, True, 0),
    ("bf16", 1, 257, 160, 16, 1, [0, 31, 32, 33, 256, 257], True, True, True, True, 5),
    ("f32", 1, 130, 32, 8, 1, [0, 129, 130], True, False, True, True, 0),
    ("f32", 1, 70, 32, 32, 1, [0, 16, 20, 70], True, True, True, True, 0),
    ("f32", 1, 0, 32, 16, 1, [0, 0, 0], True, True, True, True, 0),
    ("f32", 2, 0, 32, 16, 1, None, True, True, True, True, 0),
]
IDS = [f"{c[0]}-b{c[1]}-L{c[2]}-ch{c[3]}-N{c[4]}-G{c[5]}{'-packed' if c[6] else ''}" for c in CASES]


def args_of(t):
    return [t[k] for k in NAMES]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    dtype, b, L, ch, N, G, cu, gate, init, skip, bias, pad = case
    t = make(dtype, b, L, ch, N, G, cu, gate, init, skip, bias, pad=pad)
    y, fin = ssd.ssd_channel_scan_fwd(*args_of(t), cu_seqlens=cu)
    want, wfin = ref.scan(*[ref.d(t[k]) for k in NAMES], cu)
    # a state is a sum of terms decayed by products of exponentials, each
    # good to a few 2^-22; y sums 16 to 32 of them
    ref.check(y, want, "y", rel=1e-5)
    ref.check(fin, wfin, "final_state", rel=1e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_gradient(case):
    dtype, b, L, ch, N, G, cu, gate, init, skip, bias, pad = case
    t = make(dtype, b, L, ch, N, G, cu, gate, init, skip, bias, pad=pad, seed=1)
    g = torch.Generator().manual_seed(11)
    nst = b if cu is None else len(cu) - 1
    dy = torch.randn(b, L, ch, generator=g).to(DT[dtype]).cuda()
    dfin = 0.3 * torch.randn(nst, ch, N, generator=g).cuda() if init else None
    got = ssd.ssd_channel_scan_bwd(dy, *args_of(t), cu_seqlens=cu, dfinal_state=dfin)
    leaves = [ref.d(t[k]) for k in NAMES]
    for v in leaves:
        if v is not None:
            v.requires_grad_(True)
    out = ref.scan(*leaves, cu)
    want = ref.gradients(out, [ref.d(dy), ref.d(dfin)], leaves)
    for name, a, w in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dinit"), got, want):
        # sums over tokens and channels whose terms may be several times the result's size
        ref.check(a, w, name, rel=3e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("soft", [True, False])
def test_plain_delta(soft):
    t = make("f32", 1, 60, 32, 16, bias=soft, seed=2)
    t["dt"] = t["dt"].abs() * 0.1 if not soft else t["dt"] * 30  # large arguments of the softplus too
    y, fin = ssd.ssd_channel_scan_fwd(*args_of(t), dt_softplus=soft)
    leaves = [ref.d(t[k]) for k in NAMES]
    for v in leaves:
        if v is not None:
            v.requires_grad_(True)
    out = ref.scan(*leaves, None, soft)
    ref.check(y, out[0], "y", rel=2e-5)
    ref.check(fin, out[1], "final_state", rel=2e-5)
    dy = torch.randn_like(t["x"])
    got = ssd.ssd_channel_scan_bwd(dy, *args_of(t), dt_softplus=soft)
    want = ref.gradients(out, [ref.d(dy), None], leaves)
    for name, a, w in zip(NAMES, got, want):
        ref.check(a, w, "d" + name, rel=5e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,ch,N,G", [("f32", 40, 16, 1), ("bf16", 64, 8, 2), ("bf16", 1001, 16, 1), ("f32", 48, 32, 3)])
def test_tokens_one_by_one(dtype, ch, N, G):
    t = make(dtype, 3, 6, ch, N, G, seed=3)
    state = t["init"].clone()
    rows = []
    for k in range(6):
        rows.append(ssd.ssd_channel_scan_step(t["x"][:, k], t["dt"][:, k], t["A"], t["B"][:, k], t["C"][:, k], t["D"],
                                              t["z"][:, k], t["dt_bias"], state=state))
    want, wfin = ref.scan(*[ref.d(t[k]) for k in NAMES])
    ref.check(torch.stack(rows, 1), want, "y", rel=1e-5)
    ref.check(state, wfin, "state", rel=1e-5)


@pytest.mark.gpu
def test_prompt_then_tokens_is_one_sequence():
    t = make("f32", 2, 120, 64, 16, seed=4)
    cut = {k: (v[:, :100] if k in ("x", "dt", "z", "B", "C") else v) for k, v in t.items()}  # strided views
    y0, state = ssd.ssd_channel_scan_fwd(*args_of(cut))
    for k in range(100, 120):
        ssd.ssd_channel_scan_step(t["x"][:, k], t["dt"][:, k], t["A"], t["B"][:, k], t["C"][:, k], t["D"], t["z"][:, k],
                                  t["dt_bias"], state=state)
    y, fin = ssd.ssd_channel_scan_fwd(*args_of(t))
    ref.check(y0, ref.d(y[:, :100]), "y", rel=1e-5)
    ref.check(state, ref.d(fin), "state", rel=1e-5)


@pytest.mark.gpu
def test_gradient_agrees_with_differences():
    cu = [0, 5, 60, 100]
    t = make("f32", 1, 100, 32, 16, cu=cu, seed=5)
    g = torch.Generator(device="cuda").manual_seed(3)
    dy = torch.randn(1, 100, 32, device="cuda", generator=g)
    dfin = torch.randn(3, 32, 16, device="cuda", generator=g)
    grads = ssd.ssd_channel_scan_bwd(dy, *args_of(t), cu_seqlens=cu, dfinal_state=dfin)
    for i, k in enumerate(NAMES):
        v = torch.randn(t[k].shape, device="cuda", generator=g)
        vals = []
        for e in (3e-3, -3e-3):
            u = dict(t, **{k: t[k] + e * v})
            y, fin = ssd.ssd_channel_scan_fwd(*args_of(u), cu_seqlens=cu)
            vals.append((y.double() * dy.double()).sum() + (fin.double() * dfin.double()).sum())
        slope = float(vals[0] - vals[1]) / 6e-3
        size = float(grads[i].double().norm() * v.double().norm())
        # truncation 1e-5 of the third derivative, fp32 rounding over the step: below 2e-3 of |grad| |v|
        assert abs(slope - float((grads[i].double() * v.double()).sum())) <= 2e-3 * size, k


@pytest.mark.gpu
def test_nothing_crosses_a_boundary():
    cu = [0, 40, 41, 100]
    t = make("f32", 1, 100, 32, 16, cu=cu, init=False, seed=6)
    bad = dict(t, x=t["x"].clone(), B=t["B"].clone())
    bad["x"][0, 40] = float("nan")
    bad["B"][0, 40] = float("inf")
    y, fin = ssd.ssd_channel_scan_fwd(*args_of(bad), cu_seqlens=cu)
    y0, fin0 = ssd.ssd_channel_scan_fwd(*args_of(t), cu_seqlens=cu)
    for s in (slice(0, 40), slice(41, 100)):
        assert torch.equal(y[0, s], y0[0, s])
    assert torch.equal(fin[0], fin0[0]) and torch.equal(fin[2], fin0[2])
    dy = torch.randn_like(t["x"])
    got = ssd.ssd_channel_scan_bwd(dy, *args_of(bad), cu_seqlens=cu)
    clean = ssd.ssd_channel_scan_bwd(dy, *args_of(t), cu_seqlens=cu)
    for i in (0, 1, 3, 4, 6):
        for s in (slice(0, 40), slice(41, 100)):
            assert torch.equal(got[i][0, s], clean[i][0, s]), i


@pytest.mark.gpu
def test_many_sequences_and_repeats_bitwise_on_another_stream():
    lens = torch.randint(0, 5, (1500,), generator=torch.Generator().manual_seed(8)).tolist()
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    t = make("f32", 1, cu[-1], 32, 8, cu=cu, seed=7)
    first = ssd.ssd_channel_scan_fwd(*args_of(t), cu_seqlens=cu)
    want = ref.scan(*[ref.d(t[k]) for k in NAMES], cu)
    ref.check(first[0], want[0], "y", rel=1e-5)
    ref.check(first[1], want[1], "final_state", rel=1e-5)
    dy = torch.randn_like(t["x"])
    grads = ssd.ssd_channel_scan_bwd(dy, *args_of(t), cu_seqlens=cu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = ssd.ssd_channel_scan_fwd(*args_of(t), cu_seqlens=cu)
        grads2 = ssd.ssd_channel_scan_bwd(dy, *args_of(t), cu_seqlens=cu)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(first + grads, again + grads2):
        assert (a is None and b is None) or torch.equal(a, b)


# ---- refusals (host only) --------------------------------------------------
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from state_space_model_fwd_gb300 import _build
    _build.build()
    return ssd.load_library()


def c_call(lib, cu=None, ws=(None, 0), rows=None, A=FAKE, y=None, **kw):
    from state_space_model_fwd_gb300 import _layer
    v = dict(batch=1, seqlen=640, channels=64, dstate=16, ngroups=1, dtype=1, soft=1)
    v.update(kw)
    shape = _layer._channel_shape_t(v["batch"], v["seqlen"], v["channels"], v["dstate"], v["ngroups"], v["dtype"], v["soft"])
    r = rows or _layer._rows_t(FAKE, 640 * 64, 64)
    ins = _layer._channel_inputs_t(r, r, _layer._rows_t(None, 0, 0), r, r, A, None, None, None)
    yr = y or _layer._rows_t(FAKE, 640 * 64, 64)
    arr = (ctypes.c_int64 * len(cu))(*cu) if cu else None
    n = len(cu) - 1 if cu else 0
    size = lib.ssd_channel_scan_workspace_size(ctypes.byref(shape), arr, n)
    return lib.ssd_channel_scan_fwd(ctypes.byref(shape), arr, n, ctypes.byref(ins), ctypes.byref(yr), None, ws[0], ws[1],
                                    None), size


@pytest.mark.parametrize("kw,code", [
    (dict(dstate=12), UNSUPPORTED), (dict(dstate=64), UNSUPPORTED), (dict(dstate=0), INVALID), (dict(channels=0), INVALID),
    (dict(ngroups=3), INVALID), (dict(dtype=5), INVALID), (dict(batch=-1), INVALID), (dict(seqlen=1 << 31), UNSUPPORTED),
    (dict(cu=[0, 5, 4, 640]), INVALID), (dict(cu=[0, 639]), INVALID), (dict(batch=2, cu=[0, 640]), INVALID),
])
def test_shapes_and_offsets_are_checked(lib, kw, code):
    st, size = c_call(lib, **kw)
    assert st == code and size == 0


def test_pointers_and_workspace_are_checked(lib):
    from state_space_model_fwd_gb300 import _layer
    assert c_call(lib, A=None)[0] == INVALID
    assert c_call(lib, A=FAKE + 4)[0] == INVALID
    assert c_call(lib, rows=_layer._rows_t(None, 0, 64))[0] == INVALID
    assert c_call(lib, y=_layer._rows_t(FAKE, 640 * 64, 60))[0] == INVALID
    st, size = c_call(lib)                    # few warps: chunks, whose states need the workspace
    assert st == WORKSPACE and size > 0
    assert c_call(lib, ws=(FAKE, size - 1))[0] == WORKSPACE
    assert c_call(lib, batch=0)[0] == OK


@pytest.mark.gpu
def test_binding_refuses_on_the_gpu():
    t = make("f32", 1, 8, 32, 16)
    with pytest.raises(TypeError):
        ssd.ssd_channel_scan_fwd(*[v if k != "z" else v.bfloat16() for k, v in t.items()])
    with pytest.raises(ValueError):
        ssd.ssd_channel_scan_fwd(*args_of(dict(t, A=t["A"][:, :8].contiguous())))
    with pytest.raises(ValueError):
        ssd.ssd_channel_scan_fwd(*args_of(t), final_state=t["init"])
    with pytest.raises(ssd.SSDError):
        ssd.ssd_channel_scan_fwd(*args_of(t), cu_seqlens=[0, 9])
    with pytest.raises(TypeError):
        ssd.ssd_channel_scan_step(t["x"][:, 0].cpu(), t["dt"][:, 0], t["A"], t["B"][:, 0], t["C"][:, 0], state=t["init"])
