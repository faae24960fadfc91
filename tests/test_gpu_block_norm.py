"""The block norm on the GPU against its definition in float64."""
import ctypes

import pytest
import torch

import state_space_model_fwd_gb300 as ssd
from tests import layer_reference as ref

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5

# (dtype, rows, dim, group, gate, residual, scale, columns before)
CASES = [
    ("f32", 1, 1, 1, "none", None, False, 0),
    ("f32", 3, 64, 64, "before", None, False, 0),
    ("bf16", 37, 768, 768, "before", "f32", True, 0),
    ("bf16", 5, 2560, 2560, "none", "bf16", True, 0),
    ("bf16", 129, 1536, 192, "after", None, False, 0),
    ("f32", 17, 1001, 1001, "after", "f32", True, 0),          # odd columns: one value at a time
    ("bf16", 9, 130, 65, "before", "bf16", False, 3),          # unaligned rows
    ("f32", 4, 5120, 5120, "none", None, True, 0),
    ("bf16", 3, 10240, 10240, "before", "f32", False, 8),
    ("bf16", 2, 20000, 20000, "none", None, False, 0),
    ("f32", 2, 9001, 9001, "after", None, True, 0),
    ("bf16", 700, 256, 128, "before", "f32", True, 0),
    ("bf16", 0, 64, 64, "none", None, False, 0),
]
IDS = [f"{c[0]}-{c[1]}x{c[2]}/{c[3]}-{c[4]}-{c[5]}" for c in CASES]


def make(dtype, rows, dim, group, gate, residual, scale, pad, seed=0):
    g = torch.Generator().manual_seed(seed * 31 + dim + rows)
    n = lambda ty, std=1.0: (std * torch.randn(rows, dim + pad, generator=g)).to(ty).cuda()[:, pad:]
    ty = DT[dtype]
    return dict(x=n(ty), weight=(1 + 0.1 * torch.randn(dim, generator=g)).cuda(), z=n(ty) if gate != "none" else None,
                residual=n(DT[residual], 2.0) if residual else None,
                scale=(0.5 + 0.1 * torch.randn(dim, generator=g)).cuda() if scale else None)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    dtype, rows, dim, group, gate, residual, scale, pad = case
    t = make(*case)
    out, res = ssd.ssd_block_norm_fwd(t["x"], t["weight"], z=t["z"], residual=t["residual"], scale=t["scale"], eps=EPS,
                                      group_size=group, gate_after=gate == "after")
    want, s = ref.norm(*[ref.d(t[k]) for k in ("x", "weight", "z", "residual", "scale")], group, gate == "after", EPS)
    # the mean sums up to 32 values a thread and 1024 threads in a tree; the exponential of the gate adds 2^-21
    ref.check(out, want, "out", rel=4e-6)
    ref.check(res, s if residual else None, "residual_out", rel=2e-6)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_gradient(case):
    dtype, rows, dim, group, gate, residual, scale, pad = case
    t = make(*case, seed=1)
    g = torch.Generator().manual_seed(7)
    dout = torch.randn(rows, dim, generator=g).to(DT[dtype]).cuda()
    leaves = [ref.d(t[k]) for k in ("x", "weight", "z", "scale")]
    kw = {}
    res = None
    if residual:
        _, s = ssd.ssd_block_norm_fwd(t["x"], t["weight"], z=t["z"], residual=t["residual"], scale=t["scale"], eps=EPS,
                                      group_size=group, gate_after=gate == "after")
        kw = dict(residual_out=s, dresidual_out=torch.randn(rows, dim, generator=g).to(s.dtype).cuda())
        v = leaves[0]
        if gate == "before":
            v = v * ref.silu(leaves[2])
        v = v if leaves[3] is None else v * leaves[3]
        res = ref.d(s) - v  # the sum as it was stored
    got = ssd.ssd_block_norm_bwd(dout, t["x"], t["weight"], z=t["z"], scale=t["scale"], eps=EPS, group_size=group,
                                 gate_after=gate == "after", **kw)
    x, weight, z, sc = leaves
    for v in leaves + [res]:
        if v is not None:
            v.requires_grad_(True)
    out, summed = ref.norm(x, weight, z, res, sc, group, gate == "after", EPS)
    want = ref.gradients([out, summed if residual else None], [ref.d(dout), ref.d(kw.get("dresidual_out"))],
                         [x, weight, z, res, sc])
    # ds = rstd (gw - hat mean(gw hat)): the two terms are rstd |gw| each and may cancel (entirely, in groups of one)
    q = summed.detach().reshape(rows, dim // group, group)
    rstd = (1 / torch.sqrt((q * q).mean(-1, keepdim=True) + EPS)).expand(q.shape).reshape(rows, dim)
    terms = rstd * (ref.d(dout) * weight.detach()).abs()
    for name, a, w in zip(("dx", "dweight", "dz", "dresidual", "dscale"), got, want):
        size = None
        if name in ("dweight", "dscale"):
            size = 2.0 * max(rows, 1) ** 0.5  # column sums: up to 700 terms of size 1 to 3, in several partial sums
        elif name in ("dx", "dresidual") and w is not None and w.numel():
            size = torch.maximum(torch.maximum(w.abs(), w.pow(2).mean().sqrt()), terms)
        ref.check(a, w, name, rel=1e-5, scale=size)


@pytest.mark.gpu
def test_gradient_agrees_with_differences():
    t = make("f32", 6, 48, 24, "before", "f32", True, 0, seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda s: torch.randn(s, device="cuda", generator=g)
    dout, dres = rnd((6, 48)), rnd((6, 48))
    f = lambda u: ssd.ssd_block_norm_fwd(u["x"], u["weight"], z=u["z"], residual=u["residual"], scale=u["scale"],
                                         group_size=24)
    _, s = f(t)
    got = ssd.ssd_block_norm_bwd(dout, t["x"], t["weight"], z=t["z"], scale=t["scale"], residual_out=s,
                                 dresidual_out=dres, group_size=24)
    for k, grad in zip(("x", "weight", "z", "residual", "scale"), got):
        v = rnd(t[k].shape)
        vals = []
        for e in (3e-3, -3e-3):
            out, so = f(dict(t, **{k: t[k] + e * v}))
            vals.append((out.double() * dout.double()).sum() + (so.double() * dres.double()).sum())
        slope = float(vals[0] - vals[1]) / 6e-3
        # truncation 1e-5 of the third derivative and fp32 rounding over the step
        assert abs(slope - float((grad.double() * v.double()).sum())) <= 2e-3 * float(grad.double().norm() * v.double().norm()), k


@pytest.mark.gpu
def test_rows_of_zeros_and_in_place_residual():
    x = torch.zeros(4, 96, device="cuda")
    out, _ = ssd.ssd_block_norm_fwd(x, torch.ones(96, device="cuda"))
    assert torch.equal(out, x)  # 0 / sqrt(eps)
    dx, dw, *_ = ssd.ssd_block_norm_bwd(torch.ones_like(x), x, torch.ones(96, device="cuda"))
    assert torch.isfinite(dx).all() and float(dw.abs().max()) == 0
    t = make("bf16", 33, 512, 512, "none", "f32", False, 0, seed=4)
    out, res = ssd.ssd_block_norm_fwd(t["x"], t["weight"], residual=t["residual"])
    stream_res = t["residual"].clone()
    out2, same = ssd.ssd_block_norm_fwd(t["x"], t["weight"], residual=stream_res, residual_out=stream_res)
    assert same is stream_res and torch.equal(out, out2) and torch.equal(res, stream_res)


@pytest.mark.gpu
def test_leading_dimensions_and_streams():
    t = make("bf16", 60, 256, 256, "before", None, False, 0, seed=5)
    x3, z3 = t["x"].view(3, 20, 256), t["z"].view(3, 20, 256)
    a, _ = ssd.ssd_block_norm_fwd(t["x"], t["weight"], z=t["z"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b, _ = ssd.ssd_block_norm_fwd(x3, t["weight"], z=z3)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, b.view(60, 256))
    with pytest.raises(ValueError):
        ssd.ssd_block_norm_fwd(x3[:, :7], t["weight"], z=z3[:, :7])  # rows at two strides
    with pytest.raises(ssd.SSDError):
        ssd.ssd_block_norm_fwd(t["x"], t["weight"], group_size=100)
    with pytest.raises(TypeError):
        ssd.ssd_block_norm_fwd(t["x"], t["weight"].bfloat16())


# ---- refusals (host only) --------------------------------------------------
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
FAKE = 1 << 20


def test_arguments_are_checked():
    from state_space_model_fwd_gb300 import _build, _layer
    _build.build()
    lib = ssd.load_library()

    def call(rows=4, dim=64, group=64, eps=1e-5, dtype=1, rdtype=1, x=FAKE, rs=64, out_rs=64, w=FAKE, res=None):
        shape = _layer._norm_shape_t(rows, dim, group, eps, dtype, rdtype, 0)
        xr, o = _layer._rows_t(x, 0, rs), _layer._rows_t(FAKE, 0, out_rs)
        return lib.ssd_block_norm_fwd(ctypes.byref(shape), ctypes.byref(xr), w, None, res and ctypes.byref(res), None,
                                      ctypes.byref(o), None, None)

    assert call(group=48) == INVALID and call(group=0) == INVALID and call(dim=0) == INVALID
    assert call(dtype=9) == INVALID and call(dtype=0, rdtype=1) == INVALID and call(eps=-1.0) == INVALID
    assert call(x=None) == INVALID and call(x=FAKE + 1) == INVALID and call(w=None) == INVALID
    assert call(out_rs=63) == INVALID
    assert call(res=_layer._rows_t(FAKE, 0, 64)) == INVALID          # no place for the sum
    assert call(dim=65536, group=65536, rs=65536, out_rs=65536) == UNSUPPORTED
    assert call(rows=0) == OK
    s = _layer._norm_shape_t(4, 64, 64, 1e-5, 1, 1, 0)
    r = _layer._rows_t(FAKE, 0, 64)
    need = lib.ssd_block_norm_bwd_workspace_size(ctypes.byref(s))
    assert need > 0
    args = [ctypes.byref(s), ctypes.byref(r), ctypes.byref(r), FAKE, None, None, None, None, ctypes.byref(r), FAKE, None,
            None, None]
    assert lib.ssd_block_norm_bwd(*args, FAKE, need - 1, None) == WORKSPACE
    with pytest.raises(TypeError):
        ssd.ssd_block_norm_fwd(torch.zeros(2, 8), torch.ones(8))
