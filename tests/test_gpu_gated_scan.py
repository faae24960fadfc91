"""The gated scan on the GPU against its definition in float64: prompts (equal
lengths and packed), gradients, one token at a time."""
import ctypes

import pytest
import torch

import state_space_model_fwd_gb300 as ssd
from tests import layer_reference as ref

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NAMES = ("x", "r", "decay", "i", "z", "init")


def definition(x, r, decay, i, z, init, cu=None, rate=8.0):
    """One sequence and one token after another, in float64."""
    b, L, ch = x.shape
    log_a = -rate * ref.softplus(decay) * torch.sigmoid(r)
    a = torch.exp(log_a)
    u = torch.sqrt(-torch.expm1(2 * log_a)) * x
    u = u if i is None else u * torch.sigmoid(i)
    rows, finals = {}, []
    for s, k, lo, hi in ref.spans(b, L, cu):
        h = x.new_zeros(ch) if init is None else init[s]
        for t in range(lo, hi):
            h = a[k, t] * h + u[k, t]
            rows[k, t] = h if z is None else h * ref.silu(z[k, t])
        finals.append(h)
    y = torch.stack([rows[k, t] for k in range(b) for t in range(L)]).reshape(b, L, ch) if b * L else x.clone()
    return y, (torch.stack(finals) if finals else x.new_zeros(0, ch))


def make(dtype, b, L, ch, cu=None, igate=True, gate=True, init=True, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed * 1009 + ch * 7 + L)
    n = lambda *s: torch.randn(*s, generator=g)
    rows = lambda: n(b, L, ch + pad).to(DT[dtype]).cuda()[:, :, pad:]
    sp = -torch.log(0.9 + 0.099 * torch.rand(ch, generator=g))
    t = dict(x=rows(), r=rows(), decay=sp + torch.log(-torch.expm1(-sp)), i=rows() if igate else None,
             z=rows() if gate else None, init=0.5 * n(b if cu is None else len(cu) - 1, ch) if init else None)
    return {k: None if v is None else v.cuda() for k, v in t.items()}


def args_of(t):
    return [t[k] for k in NAMES]


# (dtype, b, L, channels, offsets, input gate, gate, init, columns before)
CASES = [
    ("f32", 1, 1, 64, None, True, True, True, 0),
    ("bf16", 2, 15, 64, None, True, False, False, 0),            # one warp
    ("f32", 3, 57, 66, None, True, True, True, 0),               # two channels in the second block
    ("bf16", 2, 129, 130, None, False, True, True, 2),           # two tiles forward, no input gate
    ("f32", 1, 300, 33, None, True, True, False, 0),             # odd: one element at a time
    ("bf16", 1, 200, 70, None, True, True, True, 3),             # pairs across their boundary
    ("f32", 1, 1100, 64, None, True, False, True, 0),            # a second group of tiles in the gradient
    ("bf16", 2, 2200, 40, None, True, True, True, 0),            # and in the forward kernel
    ("f32", 1, 300, 64, [0, 0, 1, 2, 70, 128, 128, 192, 300, 300], True, True, True, 0),
    ("bf16", 1, 257, 160, [0, 31, 32, 33, 256, 257], True, True, True, 5),
    ("f32", 1, 130, 1, [0, 129, 130], True, False, False, 0),
    ("bf16", 1, 2500, 64, [0, 16, 17, 1040, 2111, 2112, 2500], False, True, True, 0),
    ("f32", 1, 0, 32, [0, 0, 0], True, True, True, 0),
    ("f32", 2, 0, 32, None, True, True, True, 0),
]
IDS = [f"{c[0]}-b{c[1]}-L{c[2]}-ch{c[3]}{'-packed' if c[4] else ''}" for c in CASES]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    dtype, b, L, ch, cu, igate, gate, init, pad = case
    t = make(dtype, b, L, ch, cu, igate, gate, init, pad=pad)
    y, fin = ssd.ssd_gated_scan_fwd(*args_of(t), cu_seqlens=cu)
    want, wfin = definition(*[ref.d(t[k]) for k in NAMES], cu)
    # beta and a are each good to a few 2^-22; a state with decay a sums up to 1 / (1 - a) <= 2000 terms whose errors in a,
    # 2^-24 each and independent, add up to sqrt(2000) 2^-24 = 3e-6 of it
    ref.check(y, want, "y", rel=1e-5)
    ref.check(fin, wfin, "final_state", rel=1e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("kept", [True, False], ids=["kept", "formed"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_gradient(case, kept):
    dtype, b, L, ch, cu, igate, gate, init, pad = case
    t = make(dtype, b, L, ch, cu, igate, gate, init, pad=pad, seed=1)
    g = torch.Generator().manual_seed(11)
    dy = torch.randn(b, L, ch, generator=g).to(DT[dtype]).cuda()
    dfin = torch.randn(b if cu is None else len(cu) - 1, ch, generator=g).cuda() if init else None
    states = ssd.ssd_gated_scan_fwd(*args_of(t), cu_seqlens=cu, return_chunk_states=True)[2] if kept else None
    got = ssd.ssd_gated_scan_bwd(dy, *args_of(t), cu_seqlens=cu, dfinal_state=dfin, chunk_states=states)
    leaves = [ref.d(t[k]) for k in NAMES]
    for v in leaves:
        if v is not None:
            v.requires_grad_(True)
    out = definition(*leaves, cu)
    want = ref.gradients(out, [ref.d(dy), ref.d(dfin)], leaves)
    # dr is a difference of two terms, a h and s(i) x a^2 / beta, of up to ten times its size
    for name, a, w in zip(("dx", "dr", "ddecay", "di", "dz", "dinit"), got, want):
        ref.check(a, w, name, rel=1e-4 if name in ("dr", "ddecay") else 2e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,b,L,ch,gate", [
    ("bf16", 1001, 5, 64, True), ("f32", 1001, 9, 64, False), ("bf16", 500, 17, 100, True), ("f32", 403, 20, 40, True),
    ("bf16", 2601, 3, 6, False), ("f32", 2601, 1, 5, True), ("bf16", 333, 33, 63, False), ("f32", 333, 26, 64, True),
])
def test_many_short_rows(dtype, b, L, ch, gate):
    """Several rows to a block, some blocks with fewer than others."""
    t = make(dtype, b, L, ch, gate=gate, seed=6)
    want, wfin = definition(*[ref.d(t[k]) for k in NAMES])
    y, fin, states = ssd.ssd_gated_scan_fwd(*args_of(t), return_chunk_states=True)
    ref.check(y, want, "y", rel=1e-5)  # as in test_forward, of fewer tokens
    ref.check(fin, wfin, "final_state", rel=1e-5)
    assert torch.equal(states[:, 0], t["init"])
    dy = torch.randn(b, L, ch, generator=torch.Generator().manual_seed(12)).to(DT[dtype]).cuda()
    got = ssd.ssd_gated_scan_bwd(dy, *args_of(t), chunk_states=states)
    leaves = [ref.d(t[k]) for k in NAMES]
    for v in leaves:
        if v is not None:
            v.requires_grad_(True)
    want = ref.gradients(definition(*leaves), [ref.d(dy), None], leaves)
    for name, a, w in zip(("dx", "dr", "ddecay", "di", "dz", "dinit"), got, want):
        ref.check(a, w, name, rel=1e-4 if name in ("dr", "ddecay") else 2e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_all_decays(dtype):
    """From states that are forgotten at once to ones that are kept for good, gates shut and open."""
    t = make(dtype, 1, 90, 64, seed=2)
    t["decay"] = torch.linspace(-30, 30, 64, device="cuda")
    t["r"] = (t["r"].float() * 20).to(DT[dtype])
    t["r"][:, 5], t["r"][:, 50], t["i"][:, 7], t["i"][:, 9] = 300.0, -300.0, 300.0, -300.0
    y, fin = ssd.ssd_gated_scan_fwd(*args_of(t))
    leaves = [ref.d(t[k]).requires_grad_(True) for k in NAMES]
    out = definition(*leaves)
    ref.check(y, out[0], "y", rel=1e-5)
    ref.check(fin, out[1], "final_state", rel=1e-5)
    dy = torch.randn_like(t["x"])
    got = ssd.ssd_gated_scan_bwd(dy, *args_of(t))
    # r = -300 leaves l = 0, where the definition's derivative of sqrt(1 - a^2) is infinite and autograd gives NaN for
    # infinity times zero: the limit is 0
    want = ref.gradients(out, [ref.d(dy), None], leaves)
    ref.check(got[0], want[0], "dx", rel=2e-5)
    dr = torch.where(ref.d(t["r"]) < -200, 0.0, want[1])
    assert torch.isfinite(dr).all() and torch.isfinite(got[2]).all()
    ref.check(got[1], dr, "dr", rel=1e-4)


@pytest.mark.gpu
@pytest.mark.parametrize("gates", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("dtype,L,cu", [("f32", 40, None), ("bf16", 150, None), ("f32", 150, [0, 1, 60, 64, 129, 150])])
def test_gradient_of_states_that_fade_within_a_token(dtype, L, cu, gates):
    """m = -log a from 1 to 16, signs chosen so that nothing cancels: every gradient is good relative to itself."""
    ch = 64
    g = torch.Generator().manual_seed(21)
    uni = lambda *s: 1 + torch.rand(*s, generator=g)
    n = 1 if cu is None else len(cu) - 1
    sign = 1 - 2.0 * (torch.arange(L) % 2)[:, None]  # x against the state that the tokens before it leave
    softplus = torch.linspace(1.3, 15, ch) / 4      # rate 8, s(r) around 1/2
    t = dict(x=uni(1, L, ch) * sign, r=0.2 * torch.randn(1, L, ch, generator=g), i=None, z=None,
             decay=softplus + torch.log(-torch.expm1(-softplus)), init=torch.empty(n, ch))
    starts = [0] if cu is None else cu[:-1]
    for s, at in enumerate(starts):
        t["init"][s] = -uni(ch) * sign[at]
    if gates:
        t["i"], t["z"] = torch.randn(1, L, ch, generator=g), uni(1, L, ch)
    t = {k: None if v is None else v.to(DT[dtype] if k in ("x", "r", "i", "z") else torch.float32).cuda() for k, v in t.items()}
    dy = uni(1, L, ch).to(DT[dtype]).cuda()
    dfin = uni(n, ch).cuda()
    m = 8 * ref.softplus(ref.d(t["decay"])) * torch.sigmoid(ref.d(t["r"]))
    assert m.min() > 0.8 and 12 < m.max() < 20
    leaves = [None if t[k] is None else ref.d(t[k]) for k in NAMES]
    leaves[2] = leaves[2].expand(L, ch).clone()      # a decay for every token: its gradient's terms
    for v in leaves:
        if v is not None:
            v.requires_grad_(True)
    want = ref.gradients(definition(*leaves, cu), [ref.d(dy), ref.d(dfin)], leaves)
    terms, want[2] = want[2], want[2].sum(0)
    got = ssd.ssd_gated_scan_bwd(dy, *args_of(t), cu_seqlens=cu, dfinal_state=dfin)
    # m is good to 2^-20.5 of itself (softplus and the sigmoid a few 2^-23 each), 1.2e-5 at 17, which is a's relative error; its
    # exponential adds 2^-20 for the rounded argument; dr and ddecay have m once more, and a state of the same kind beside it
    for name, a, w in zip(("dx", "dr", "ddecay", "di", "dz", "dinit"), got, want):
        ref.check(a, w, name, rel=4e-5, scale=None if w is None else terms.abs().sum(0) if name == "ddecay" else w.abs())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_all_decays_all_gradients(dtype):
    """As test_all_decays; every gradient, dr and ddecay against their own channel's size."""
    t = make(dtype, 1, 90, 64, seed=2)
    t["decay"] = torch.linspace(-30, 30, 64, device="cuda")
    t["r"] = (t["r"].float() * 20).to(DT[dtype])
    t["r"][:, 5], t["r"][:, 50], t["i"][:, 7], t["i"][:, 9] = 300.0, -300.0, 300.0, -300.0
    g = torch.Generator().manual_seed(22)
    dy = torch.randn(1, 90, 64, generator=g).to(DT[dtype]).cuda()
    dfin = torch.randn(1, 64, generator=g).cuda()
    got = ssd.ssd_gated_scan_bwd(dy, *args_of(t), dfinal_state=dfin)
    leaves = [ref.d(t[k]) for k in NAMES]
    leaves[2] = leaves[2].expand(90, 64).clone()
    for v in leaves:
        v.requires_grad_(True)
    want = ref.gradients(definition(*leaves), [ref.d(dy), ref.d(dfin)], leaves)
    shut = ref.d(t["r"]) < -200  # the limit, where autograd multiplies infinity and zero
    want[1] = torch.where(shut, 0.0, want[1])
    terms = torch.where(shut[0], 0.0, want[2])
    want[2] = terms.sum(0)
    channel = lambda w: torch.maximum(w.abs(), w.square().mean(-2, keepdim=True).sqrt())
    # as in test_gradient; a is good to 2^-20.5 m, 6e-5 where it leaves fp32's range
    ref.check(got[0], want[0], "dx", rel=2e-5)
    ref.check(got[1], want[1], "dr", rel=2e-4, scale=channel(want[1]))
    ref.check(got[2], want[2], "ddecay", rel=2e-4, scale=terms.abs().sum(0))
    ref.check(got[3], want[3], "di", rel=2e-5)
    ref.check(got[4], want[4], "dz", rel=2e-5)
    ref.check(got[5], want[5], "dinit", rel=1e-4, scale=want[5].abs())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,ch,igate,gate", [("f32", 40, True, True), ("bf16", 64, True, False), ("bf16", 1001, False, True)])
def test_tokens_one_by_one(dtype, ch, igate, gate):
    t = make(dtype, 3, 6, ch, igate=igate, gate=gate, seed=3)
    state = t["init"].clone()
    at = lambda v, k: None if v is None else v[:, k]
    rows = [ssd.ssd_gated_scan_step(t["x"][:, k], t["r"][:, k], t["decay"], at(t["i"], k), at(t["z"], k), state=state)
            for k in range(6)]
    want, wfin = definition(*[ref.d(t[k]) for k in NAMES])
    ref.check(torch.stack(rows, 1), want, "y", rel=1e-5)
    ref.check(state, wfin, "state", rel=1e-5)


@pytest.mark.gpu
def test_prompt_then_tokens_is_one_sequence():
    t = make("f32", 2, 220, 64, seed=4)
    cut = {k: (v[:, :200] if k in ("x", "r", "i", "z") else v) for k, v in t.items()}  # strided views
    y0, state = ssd.ssd_gated_scan_fwd(*args_of(cut))
    for k in range(200, 220):
        ssd.ssd_gated_scan_step(t["x"][:, k], t["r"][:, k], t["decay"], t["i"][:, k], t["z"][:, k], state=state)
    y, fin = ssd.ssd_gated_scan_fwd(*args_of(t))
    ref.check(y0, ref.d(y[:, :200]), "y", rel=1e-5)
    ref.check(state, ref.d(fin), "state", rel=1e-5)


@pytest.mark.gpu
def test_gradient_agrees_with_differences():
    cu = [0, 5, 60, 200]
    t = make("f32", 1, 200, 64, cu=cu, seed=5)
    g = torch.Generator(device="cuda").manual_seed(3)
    dy = torch.randn(1, 200, 64, generator=g, device="cuda")
    dfin = torch.randn(3, 64, generator=g, device="cuda")
    grads = dict(zip(("x", "r", "decay", "i", "z", "init"),
                     ssd.ssd_gated_scan_bwd(dy, *args_of(t), cu_seqlens=cu, dfinal_state=dfin)))
    for k in NAMES:
        v = torch.randn(t[k].shape, generator=g, device="cuda")
        vals = []
        for e in (3e-3, -3e-3):
            y, fin = ssd.ssd_gated_scan_fwd(*args_of(dict(t, **{k: t[k] + e * v})), cu_seqlens=cu)
            vals.append((y.double() * dy.double()).sum() + (fin.double() * dfin.double()).sum())
        slope = float(vals[0] - vals[1]) / 6e-3
        size = float(grads[k].double().norm() * v.double().norm())
        # truncation 1e-5 of the third derivative, fp32 rounding over the step: below 2e-3 of |grad| |v|
        assert abs(slope - float((grads[k].double() * v.double()).sum())) <= 2e-3 * size, k


@pytest.mark.gpu
def test_nothing_crosses_a_boundary():
    cu = [0, 40, 41, 64, 128, 700]
    t = make("f32", 1, 700, 64, cu=cu, init=False, seed=6)
    bad = dict(t, x=t["x"].clone(), r=t["r"].clone())
    bad["x"][0, 40] = float("nan")
    bad["x"][0, 100] = float("inf")
    bad["r"][0, 63] = float("nan")
    y, fin = ssd.ssd_gated_scan_fwd(*args_of(bad), cu_seqlens=cu)
    y0, fin0 = ssd.ssd_gated_scan_fwd(*args_of(t), cu_seqlens=cu)
    dy = torch.randn_like(t["x"])
    got = ssd.ssd_gated_scan_bwd(dy, *args_of(bad), cu_seqlens=cu)
    clean = ssd.ssd_gated_scan_bwd(dy, *args_of(t), cu_seqlens=cu)
    for s in (0, 4):
        span = slice(cu[s], cu[s + 1])
        assert torch.equal(y[0, span], y0[0, span]) and torch.equal(fin[s], fin0[s])
        for k in (0, 1, 3, 4):
            assert torch.equal(got[k][0, span], clean[k][0, span]), k
    # inside a sequence it goes on, towards later tokens in the state and towards earlier ones in the gradient
    assert torch.isnan(y[0, 40]).all() and torch.isnan(fin[2]).all() and not torch.isfinite(fin[3]).any()
    assert torch.isfinite(y[0, 41:63]).all() and torch.isnan(got[0][0, 41:64]).all()


@pytest.mark.gpu
def test_many_sequences_and_repeats_bitwise_on_another_stream():
    lens = torch.randint(0, 5, (1500,), generator=torch.Generator().manual_seed(8)).tolist()
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    t = make("f32", 1, cu[-1], 32, cu=cu, seed=7)
    first = ssd.ssd_gated_scan_fwd(*args_of(t), cu_seqlens=cu, return_chunk_states=True)
    want = definition(*[ref.d(t[k]) for k in NAMES], cu)
    ref.check(first[0], want[0], "y", rel=1e-5)
    ref.check(first[1], want[1], "final_state", rel=1e-5)
    dy = torch.randn_like(t["x"])
    grads = ssd.ssd_gated_scan_bwd(dy, *args_of(t), cu_seqlens=cu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = ssd.ssd_gated_scan_fwd(*args_of(t), cu_seqlens=cu, return_chunk_states=True, stream=s)
    grads2 = ssd.ssd_gated_scan_bwd(dy, *args_of(t), cu_seqlens=cu, chunk_states=again[2], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(first + grads, again + grads2):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.gpu
def test_captured_and_replayed():
    t = make("bf16", 2, 700, 128, seed=9)
    dy = torch.randn_like(t["x"])
    y = torch.empty_like(t["x"])
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")  # one workspace for both graphs
    graphs, outs = [], []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = ssd.ssd_gated_scan_fwd(*args_of(t), y=y, workspace=ws, return_chunk_states=True)
            outs.append(out + ssd.ssd_gated_scan_bwd(dy, *args_of(t), chunk_states=out[2], workspace=ws))
        graphs.append(g)
    for _ in range(2):
        t["x"].normal_()
        for g in graphs:
            g.replay()
        want = ssd.ssd_gated_scan_fwd(*args_of(t), return_chunk_states=True)
        want = want + ssd.ssd_gated_scan_bwd(dy, *args_of(t))
        for o in outs:
            for a, b in zip(o, want):
                assert torch.equal(a, b)


@pytest.mark.gpu
def test_reads_and_writes_among_nans():
    """Operands are slices of wider rows full of NaN; outputs keep what lies around them."""
    for pad, dtype in ((2, "bf16"), (3, "f32")):
        b, L, ch = 2, 150, 70
        t = make(dtype, b, L, ch, seed=12)
        wide = {}
        for k in ("x", "r", "i", "z"):
            w = torch.full((b, L + 2, ch + 2 * pad), float("nan"), dtype=DT[dtype], device="cuda")
            w[:, 1:-1, pad:-pad] = t[k]
            wide[k] = w[:, 1:-1, pad:-pad]
        out = torch.full((b, L + 2, ch + 2 * pad), 7.0, dtype=DT[dtype], device="cuda")
        y = out[:, 1:-1, pad:-pad]
        got = ssd.ssd_gated_scan_fwd(*args_of(dict(t, **wide)), y=y)
        want = ssd.ssd_gated_scan_fwd(*args_of(t))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        out[:, 1:-1, pad:-pad] = 7.0
        assert bool((out == 7.0).all())
        dy = torch.randn_like(t["x"])
        for a, w in zip(ssd.ssd_gated_scan_bwd(dy, *args_of(dict(t, **wide))), ssd.ssd_gated_scan_bwd(dy, *args_of(t))):
            assert torch.equal(a, w)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,L,ch,pads", [
    ("bf16", 70, 64, (1, 7, 8, 2, 3)), ("bf16", 33, 130, (5, 4, 0, 9, 1)), ("bf16", 20, 5, (3, 1, 6, 0, 2)), ("bf16", 300, 72, (8, 16, 0, 24, 8)),
    ("bf16", 41, 192, (2, 4, 6, 2, 10)), ("f32", 50, 64, (1, 3, 2, 4, 1)), ("f32", 21, 3, (1, 2, 3, 0, 1)), ("f32", 90, 100, (2, 4, 0, 6, 2)),
])
def test_every_alignment(dtype, L, ch, pads):
    """Each operand at its own distance from a 16-byte boundary, in rows at every one, among NaN."""
    t = make(dtype, 2, L, ch, seed=15)
    dy = torch.randn(2, L, ch, generator=torch.Generator().manual_seed(3)).to(DT[dtype]).cuda()
    far = {}
    for k, pad in zip(("x", "r", "i", "z", "dy"), pads):
        odd = pad % 2
        w = torch.full((2, L, ch + pad + odd), float("nan"), dtype=DT[dtype], device="cuda")
        far[k] = w[:, :, pad:pad + ch]
        far[k][:] = dy if k == "dy" else t[k]
    far_dy = far.pop("dy")
    got = ssd.ssd_gated_scan_fwd(*args_of(dict(t, **far)), return_chunk_states=True)
    want = ssd.ssd_gated_scan_fwd(*args_of(t), return_chunk_states=True)
    for a, w in zip(got, want):
        assert torch.equal(a, w)
    for a, w in zip(ssd.ssd_gated_scan_bwd(far_dy, *args_of(dict(t, **far))), ssd.ssd_gated_scan_bwd(dy, *args_of(t))):
        assert torch.equal(a, w)
    state, one = t["init"].clone(), t["init"].clone()
    token = lambda d: [d[k][:, 0] for k in ("x", "r")] + [t["decay"]] + [d[k][:, 0] for k in ("i", "z")]
    assert torch.equal(ssd.ssd_gated_scan_step(*token(far), state=state), ssd.ssd_gated_scan_step(*token(t), state=one))
    assert torch.equal(state, one)


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["x", "r", "i", "z", "dy", "y", "all"])
@pytest.mark.parametrize("dtype,b,ch,width,cu", [
    ("bf16", 1, 66, 67, None), ("f32", 1, 66, 69, None), ("bf16", 2, 1002, 1003, None), ("f32", 3, 130, 131, None),
    ("bf16", 1, 64, 67, None), ("f32", 1, 5, 7, None), ("bf16", 1, 66, 67, [0, 0, 1, 1]), ("f32", 1, 66, 69, [0, 0, 1, 1]),
    ("bf16", 1, 64, 67, [0, 0, 1, 1]), ("f32", 1, 5, 7, [0, 1]),
])
def test_one_token_out_of_odd_rows(dtype, b, ch, width, cu, which):
    """A prompt of one token has no next row: the stride to it means nothing."""
    t = make(dtype, b, 1, ch, cu=cu, seed=16)
    dy = torch.randn(b, 1, ch, generator=torch.Generator().manual_seed(4)).to(DT[dtype]).cuda()
    first = lambda: torch.full((b, 4, width), float("nan"), dtype=DT[dtype], device="cuda")[:, :1, :ch]

    def far(k, v):
        if which not in (k, "all"):
            return v
        w = first()
        w[:] = v
        assert w.stride()[1:] == (width, 1)
        return w
    odd = {k: far(k, v) if k in ("x", "r", "i", "z") else v for k, v in t.items()}
    y = first() if which in ("y", "all") else None
    got = ssd.ssd_gated_scan_fwd(*args_of(odd), cu_seqlens=cu, y=y, return_chunk_states=True)
    want = ssd.ssd_gated_scan_fwd(*args_of(t), cu_seqlens=cu, return_chunk_states=True)
    wy, wfin = definition(*[ref.d(t[k]) for k in NAMES], cu)
    ref.check(got[0], wy, "y", rel=1e-5)  # as in test_forward
    ref.check(got[1], wfin, "final_state", rel=1e-5)
    for a, w in zip(got, want):
        assert torch.equal(a, w)
    for states in (want[2], None):
        for a, w in zip(ssd.ssd_gated_scan_bwd(far("dy", dy), *args_of(odd), cu_seqlens=cu, chunk_states=states),
                        ssd.ssd_gated_scan_bwd(dy, *args_of(t), cu_seqlens=cu, chunk_states=states)):
            assert torch.equal(a, w)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,L,ch", [("bf16", 1, 66), ("f32", 1, 66), ("bf16", 40, 66), ("f32", 40, 66)])
def test_the_strides_of_an_absent_gate_mean_nothing(lib, dtype, L, ch):
    from state_space_model_fwd_gb300 import _layer
    t = make(dtype, 2, L, ch, igate=False, gate=False, seed=17)
    dy = torch.randn(2, L, ch, generator=torch.Generator().manual_seed(5)).to(DT[dtype]).cuda()
    want = ssd.ssd_gated_scan_fwd(*args_of(t))
    grads = ssd.ssd_gated_scan_bwd(dy, *args_of(t))
    rows = lambda v: _layer._rows_t(v.data_ptr(), L * ch, ch)
    absent = _layer._rows_t(None, 335, 67)
    shape = _layer._gated_shape_t(2, L, ch, 8.0, 1 if dtype == "bf16" else 0)
    ins = _layer._gated_inputs_t(rows(t["x"]), rows(t["r"]), absent, absent, t["decay"].data_ptr(), t["init"].data_ptr())
    y, fin = torch.empty_like(want[0]), torch.empty_like(want[1])
    dx, dr, ddecay, dinit = (torch.empty_like(grads[k]) for k in (0, 1, 2, 5))
    out = _layer._gated_grads_t(rows(dx), rows(dr), absent, absent, ddecay.data_ptr(), dinit.data_ptr())
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.ssd_gated_scan_bwd_workspace_size(ctypes.byref(shape), None, 0, 0) <= ws.numel()
    assert lib.ssd_gated_scan_fwd(ctypes.byref(shape), None, 0, ctypes.byref(ins), ctypes.byref(rows(y)), fin.data_ptr(), None,
                                  ws.data_ptr(), ws.numel(), stream) == OK
    assert lib.ssd_gated_scan_bwd(ctypes.byref(shape), None, 0, ctypes.byref(rows(dy)), ctypes.byref(ins), None, None,
                                  ctypes.byref(out), ws.data_ptr(), ws.numel(), stream) == OK
    for a, w in zip((y, fin, dx, dr, ddecay, dinit), (*want, *(grads[k] for k in (0, 1, 2, 5)))):
        assert torch.equal(a, w)


@pytest.mark.gpu
def test_more_than_2_31_elements():
    L, ch, cut = 262400, 8192, 260000
    x, r, i = (torch.empty(1, L, ch, device="cuda", dtype=torch.bfloat16).normal_() for _ in range(3))
    decay = torch.randn(ch, device="cuda") - 4
    y, fin, states = ssd.ssd_gated_scan_fwd(x, r, decay, i, return_chunk_states=True)
    mid = ssd.ssd_gated_scan_fwd(x[:, :cut], r[:, :cut], decay, i[:, :cut])[1]
    last = [v[:, cut:] for v in (x, r, i)]
    want = ssd.ssd_gated_scan_fwd(last[0], last[1], decay, last[2], init_state=mid)
    got = ssd.ssd_gated_scan_bwd(x, x, r, decay, i, chunk_states=states)
    grads = ssd.ssd_gated_scan_bwd(last[0], last[0], last[1], decay, last[2], init_state=mid)
    # the states differ by fp32 roundings (test_forward, test_gradient), which may take a bf16 result to the next value
    for a, w, rel in ((y, want[0], 1e-5), *((got[k], grads[k], 1e-4) for k in (0, 1, 3))):
        a, w = a[:, cut:].float(), w.float()
        assert bool(((a - w).abs() <= 2.0 ** -7 * w.abs() + rel * w.square().mean().sqrt()).all())
    assert bool(((fin - want[1]).abs() <= 1e-5 * want[1].square().mean().sqrt()).all())


@pytest.mark.gpu
def test_one_row_for_all():
    t = make("f32", 2, 100, 64, seed=13)
    one = t["r"][:, :1].expand(2, 100, 64)
    got = ssd.ssd_gated_scan_fwd(*args_of(dict(t, r=one)))
    want = ssd.ssd_gated_scan_fwd(*args_of(dict(t, r=one.contiguous())))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ---- refusals (host only) --------------------------------------------------
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from state_space_model_fwd_gb300 import _build
    _build.build()
    return ssd.load_library()


def c_call(lib, cu=None, ws=(None, 0), rows=None, decay=FAKE, y=None, init=None, fin=None, bwd=False, states=None, **kw):
    from state_space_model_fwd_gb300 import _layer
    v = dict(batch=1, seqlen=640, channels=64, rate=8.0, dtype=1)
    v.update(kw)
    shape = _layer._gated_shape_t(v["batch"], v["seqlen"], v["channels"], v["rate"], v["dtype"])
    r = rows or _layer._rows_t(FAKE, 640 * 64, 64)
    none = _layer._rows_t(None, 0, 0)
    ins = _layer._gated_inputs_t(r, r, none, none, decay, init)
    yr = y or _layer._rows_t(FAKE, 640 * 64, 64)
    arr = (ctypes.c_int64 * len(cu))(*cu) if cu else None
    n = len(cu) - 1 if cu else 0
    if bwd:
        size = lib.ssd_gated_scan_bwd_workspace_size(ctypes.byref(shape), arr, n, states is not None)
        grads = _layer._gated_grads_t(yr, yr, none, none, FAKE, None)
        return lib.ssd_gated_scan_bwd(ctypes.byref(shape), arr, n, ctypes.byref(r), ctypes.byref(ins), fin, states,
                                      ctypes.byref(grads), ws[0], ws[1], None), size
    size = lib.ssd_gated_scan_workspace_size(ctypes.byref(shape), arr, n)
    return lib.ssd_gated_scan_fwd(ctypes.byref(shape), arr, n, ctypes.byref(ins), ctypes.byref(yr), fin, states, ws[0], ws[1],
                                  None), size


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(channels=0), INVALID), (dict(dtype=5), INVALID), (dict(batch=-1), INVALID), (dict(rate=0.0), INVALID),
    (dict(rate=float("nan")), INVALID), (dict(rate=float("inf")), INVALID), (dict(seqlen=1 << 31), UNSUPPORTED),
    (dict(channels=1 << 25), UNSUPPORTED), (dict(cu=[0, 5, 4, 640]), INVALID), (dict(cu=[0, 639]), INVALID),
    (dict(batch=2, cu=[0, 640]), INVALID), (dict(seqlen=1 << 30, channels=1 << 20), UNSUPPORTED),
])
def test_shapes_and_offsets_are_checked(lib, bwd, kw, code):
    st, size = c_call(lib, bwd=bwd, **kw)
    assert st == code and size == 0


@pytest.mark.parametrize("bwd", [False, True])
def test_pointers_and_workspace_are_checked(lib, bwd):
    from state_space_model_fwd_gb300 import _layer
    assert c_call(lib, bwd=bwd, decay=None)[0] == INVALID
    assert c_call(lib, bwd=bwd, decay=FAKE + 2)[0] == INVALID
    assert c_call(lib, bwd=bwd, rows=_layer._rows_t(None, 0, 64))[0] == INVALID
    assert c_call(lib, bwd=bwd, rows=_layer._rows_t(FAKE + 1, 640 * 64, 64))[0] == INVALID
    assert c_call(lib, bwd=bwd, rows=_layer._rows_t(FAKE, 640 * 64, 1 << 31))[0] == INVALID
    assert c_call(lib, bwd=bwd, y=_layer._rows_t(FAKE, 640 * 64, 60))[0] == INVALID
    assert c_call(lib, bwd=bwd, fin=FAKE + 2)[0] == INVALID
    assert c_call(lib, bwd=bwd, states=FAKE + 2)[0] == INVALID
    if not bwd:
        assert c_call(lib, init=FAKE, fin=FAKE)[0] == INVALID
    st, size = c_call(lib, bwd=bwd)                    # several tiles: links in the workspace
    assert st == WORKSPACE and size > 0
    assert c_call(lib, bwd=bwd, ws=(FAKE, size - 1))[0] == WORKSPACE
    assert c_call(lib, bwd=bwd, ws=(FAKE + 8, size))[0] == WORKSPACE
    if not bwd:
        assert c_call(lib, batch=0)[0] == OK
        assert c_call(lib, seqlen=100)[1] == 0         # one tile


@pytest.mark.gpu
def test_binding_refuses_on_the_gpu():
    t = make("f32", 1, 8, 32)
    with pytest.raises(TypeError):
        ssd.ssd_gated_scan_fwd(*[v if k != "z" else v.bfloat16() for k, v in t.items()])
    with pytest.raises(ValueError):
        ssd.ssd_gated_scan_fwd(*args_of(dict(t, decay=t["decay"][:8].contiguous())))
    with pytest.raises(TypeError):
        ssd.ssd_gated_scan_fwd(*args_of(dict(t, decay=None)))
    with pytest.raises(ValueError):
        ssd.ssd_gated_scan_fwd(*args_of(t), final_state=t["init"])
    with pytest.raises(ssd.SSDError):
        ssd.ssd_gated_scan_fwd(*args_of(t), cu_seqlens=[0, 9])
    with pytest.raises(ssd.SSDError):
        ssd.ssd_gated_scan_fwd(*args_of(t), rate=-1.0)
    with pytest.raises(ValueError):
        ssd.ssd_gated_scan_bwd(t["x"], *args_of(t), chunk_states=torch.zeros(1, 2, 32, device="cuda"))
    with pytest.raises(TypeError):
        ssd.ssd_gated_scan_step(t["x"][:, 0].cpu(), t["r"][:, 0], t["decay"], state=t["init"])
    with pytest.raises(TypeError):
        ssd.ssd_gated_scan_step(t["x"][:, 0], t["r"][:, 0], t["decay"], state=None)
