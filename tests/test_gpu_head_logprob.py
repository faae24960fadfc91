"""Log-probabilities straight from hidden states and output weights, and their
gradients, against the definitions in float64."""
import ctypes
import math

import pytest
import torch

import state_space_model_fwd_gb300 as ssd
from tests import layer_reference as ref
from tests.test_gpu_token_logprob import definition, want_gradient


def make(rows, dim, vocab, seed=0, pad=0, std=2.0):
    g = torch.Generator().manual_seed(seed * 13 + rows + 3 * dim + 7 * vocab)
    n = lambda r: torch.randn(r, dim + pad, generator=g)
    h = n(rows).bfloat16().cuda()[:, :dim]
    w = (n(vocab) * std / math.sqrt(dim)).bfloat16().cuda()[:, :dim]
    return h, w, torch.randint(0, vocab, (rows,), generator=g).cuda()


def logits(h, w):
    return ref.d(h) @ ref.d(w).t()


def check_forward(got, z, targets, dim):
    logprob, lse, entropy = got
    wlp, wlse, went = definition(z, targets)
    # z: fp32 sums of dim exact products, 16 at a time, each addition off by up to 2^-23 of the sum so far, in shares of at
    # most 1280: 80 additions, half of the sum on average, 40 2^-23 = 5e-6 of z at most; then as from logits
    size = 1 + wlse.abs() + z.abs().amax(-1)
    ref.check(lse, wlse, "lse", rel=4e-6, scale=size)
    ref.check(entropy, went, "entropy", rel=1e-5, scale=size)
    if targets is None:
        assert logprob is None
    else:
        ref.check(logprob, wlp, "logprob", rel=6e-6, scale=size + wlp.abs())


# (rows, dim, vocabulary, columns behind): one tile, cut tiles, several along each side, more tiles than SMs
CASES = [
    (1, 64, 256, 0), (3, 8, 5, 0), (128, 64, 64, 0), (129, 72, 257, 0), (130, 200, 1003, 8), (16, 2560, 5000, 0),
    (1, 128, 60000, 0), (300, 320, 40001, 0), (1000, 64, 777, 0), (37, 1000, 30000, 24), (4200, 64, 1300, 0),
    (40, 64, 270000, 0), (270000, 8, 5, 0),  # sums so long that they are cut
]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,dim,vocab,pad", CASES)
def test_forward(rows, dim, vocab, pad):
    h, w, targets = make(rows, dim, vocab, pad=pad)
    if rows > 2:
        targets[rows // 2] = -100
    z = logits(h, w)
    check_forward(ssd.ssd_head_logprob_fwd(h, w, targets), z, targets, dim)
    check_forward(ssd.ssd_head_logprob_fwd(h, w), z, None, dim)


@pytest.mark.gpu
def test_more_than_2_31_logits():
    rows, dim, vocab, few = 43100, 64, 50277, 200
    h, w, targets = make(rows, dim, vocab, seed=4)
    glp, _, gent = upstream(rows)
    logprob, lse, entropy = ssd.ssd_head_logprob_fwd(h, w, targets)
    part = ssd.ssd_head_logprob_fwd(h[-few:], w, targets[-few:])
    for a, b in zip((logprob, lse, entropy), part):  # (other tiles: fp32 sums in another order)
        assert bool(((a[-few:] - b).abs() <= 2e-6 * (1 + b.abs())).all())
    dh, dw = ssd.ssd_head_logprob_bwd(h, w, targets, lse, entropy, dlogprob=glp, dentropy=gent)
    want, _ = ssd.ssd_head_logprob_bwd(h[-few:], w, targets[-few:], part[1], part[2], dlogprob=glp[-few:], dentropy=gent[-few:],
                                       need_dweight=False)
    # one step of bf16 of dz here and there, and one of the result
    d, rms = (dh[-few:].float() - want.float()).abs(), want.float().square().mean().sqrt()
    assert bool((d <= 2.0 ** -7 * want.float().abs() + 2.0 ** -7 * rms).all())
    assert torch.isfinite(dw).all()


@pytest.mark.gpu
def test_gradient_of_the_weights_beyond_2_31_logits():
    """Only the last rows have a gradient: what the weights get is what those rows alone give."""
    rows, dim, vocab, few = 43100, 64, 50277, 200
    assert (rows - few) * vocab > 1 << 31
    h, w, targets = make(rows, dim, vocab, seed=4)
    glp, _, gent = upstream(rows)
    glp[:-few], gent[:-few] = 0, 0
    _, lse, entropy = ssd.ssd_head_logprob_fwd(h, w, targets)
    dh, dw = ssd.ssd_head_logprob_bwd(h, w, targets, lse, entropy, dlogprob=glp, dentropy=gent)
    part = ssd.ssd_head_logprob_fwd(h[-few:], w, targets[-few:])
    want = ssd.ssd_head_logprob_bwd(h[-few:], w, targets[-few:], part[1], part[2], dlogprob=glp[-few:], dentropy=gent[-few:])
    assert bool((dh[:-few] == 0).all())
    # dz from an lse that is 2e-6 (1 + |lse|) apart: the next bf16 value here and there, one step (2^-7) of a term of the sum, of
    # which the largest, the given tokens', have none; and a step of the result
    for a, b in ((dh[-few:], want[0]), (dw, want[1])):
        a, b = a.float(), b.float()
        assert bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -7 * b.square().mean().sqrt()).all())


@pytest.mark.gpu
def test_many_rows_with_the_same_tokens():
    """So many that the chunks they are summed in are longer than a block, and there are hundreds of them."""
    rows, dim, vocab = 270000, 8, 40
    h, w, targets = make(rows, dim, vocab, seed=2)
    targets[:1000] = 7
    targets[100000:160000] = -1
    glp = upstream(rows)[0]
    _, lse, _ = ssd.ssd_head_logprob_fwd(h, w, targets)
    _, dw = ssd.ssd_head_logprob_bwd(h, w, targets, lse, dlogprob=glp, need_dhidden=False)
    z = logits(h, w)
    _, wlse, went = definition(z, targets)
    zero = torch.zeros(rows, dtype=torch.float64)
    d = want_gradient(z, targets.cpu(), wlse, went, ref.d(glp), zero, zero)
    # as in test_the_given_tokens_part_is_not_rounded; and the fp32 sums, two parts of 8438 additions of 16 rows, each cut off by
    # up to 2^-24 of the sum so far: 5e-4 of that, which stays within the result and 3 of the terms' root sum of squares
    p = torch.exp(z - wlse[:, None])
    err = d.abs() * 2.0 ** -8 + 2e-5 * p * ref.d(glp).abs()[:, None]
    has = targets.cpu() >= 0
    err[has, targets.cpu()[has]] = 2e-5 * ref.d(glp).abs()[has]
    x = d.t() @ ref.d(h)
    h2 = ref.d(h) ** 2
    scale = 5 / math.sqrt(3) * ((err.t() ** 2) @ h2).sqrt() + 5e-4 * (x.abs() + 3 * ((d.t() ** 2) @ h2).sqrt())
    ref.check(dw, x, "dweight", rel=1.0, scale=scale)
    assert torch.equal(ssd.ssd_head_logprob_bwd(h, w, targets, lse, dlogprob=glp, need_dhidden=False)[1], dw)


def upstream(rows, seed=3):
    g = torch.Generator().manual_seed(seed)
    return [(torch.rand(rows, generator=g) - 0.3).cuda() for _ in range(3)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,dim,vocab,pad", CASES)
@pytest.mark.parametrize("which", ["logprob", "all"])
def test_gradient(rows, dim, vocab, pad, which):
    h, w, targets = make(rows, dim, vocab, pad=pad, seed=1)
    targets[0] = -1 if rows > 1 else 0
    glp, glse, gent = upstream(rows)
    _, lse, entropy = ssd.ssd_head_logprob_fwd(h, w, targets)
    kw = dict(dlogprob=glp) if which == "logprob" else dict(dlogprob=glp, dlse=glse, dentropy=gent)
    dh, dw = ssd.ssd_head_logprob_bwd(h, w, targets, lse, entropy, **kw)
    z = logits(h, w)
    zero = torch.zeros(rows, dtype=torch.float64)
    _, wlse, went = definition(z, targets)
    a, b, c = (ref.d(glp), ref.d(glse), ref.d(gent)) if which == "all" else (ref.d(glp), zero, zero)
    d = want_gradient(z, targets.cpu(), wlse, went, a, b, c)
    # each dz is off by half a step of bf16, 2^-8 of it at most, and by 2e-5 of p (its exponent's error); a sum of n such
    # errors of random sign stays below 5 of their root sum of squares (the fp32 sums are 2^-22 of the terms')
    err = d.abs() * 2.0 ** -8 + 2e-5 * torch.exp(z - wlse[:, None]) * (a.abs() + b.abs() + 20 * c.abs())[:, None]
    for got, x, e2, name in ((dh, d @ ref.d(w), (err ** 2) @ (ref.d(w) ** 2), "dhidden"),
                             (dw, d.t() @ ref.d(h), (err.t() ** 2) @ (ref.d(h) ** 2), "dweight")):
        ref.check(got, x, name, rel=1.0, scale=5 / math.sqrt(3) * e2.sqrt() + 1e-30)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,dim,vocab,kinds", [(1, 64, 300, 1), (40, 72, 1000, 2), (1500, 64, 500, 1), (3000, 2056, 257, 3),
                                                  (255, 64, 300, 1), (257, 72, 300, 2), (5000, 8, 131, 131)])
def test_the_given_tokens_part_is_not_rounded(rows, dim, vocab, kinds):
    """Where the given token's element outweighs the others; few and many rows with the same one, some without."""
    h, w, _ = make(rows, dim, vocab, seed=9)
    g = torch.Generator().manual_seed(4)
    targets = torch.tensor([5, vocab - 1, 130, *range(6, 130), 0, 1, 2, 3, 4])[:kinds].cuda()[torch.randint(0, kinds, (rows,), generator=g).cuda()]
    if rows > 30:
        targets[::7] = -100
    glp = upstream(rows)[0]
    _, lse, _ = ssd.ssd_head_logprob_fwd(h, w, targets)
    dh, dw = ssd.ssd_head_logprob_bwd(h, w, targets, lse, dlogprob=glp)
    z = logits(h, w)
    zero = torch.zeros(rows, dtype=torch.float64)
    _, wlse, went = definition(z, targets)
    d = want_gradient(z, targets.cpu(), wlse, went, ref.d(glp), zero, zero)
    # as in test_gradient, but the given token's dz counts with its fp32 error only
    p = torch.exp(z - wlse[:, None])
    err = d.abs() * 2.0 ** -8 + 2e-5 * p * ref.d(glp).abs()[:, None]
    has = targets.cpu() >= 0
    err[has, targets.cpu()[has]] = 2e-5 * ref.d(glp).abs()[has]
    for got, x, e2, name in ((dh, d @ ref.d(w), (err ** 2) @ (ref.d(w) ** 2), "dhidden"),
                             (dw, d.t() @ ref.d(h), (err.t() ** 2) @ (ref.d(h) ** 2), "dweight")):
        ref.check(got, x, name, rel=1.0, scale=5 / math.sqrt(3) * e2.sqrt() + 1e-30)
    again = ssd.ssd_head_logprob_bwd(h, w, targets, lse, dlogprob=glp)
    assert torch.equal(again[0], dh) and torch.equal(again[1], dw)


def peaked(rows, dim, vocab, seed=0):
    """Rows whose given token is nearly certain: its logit 26 and more, 1 - p from 1e-2 to 1e-4 and less; the others around 15."""
    g = torch.Generator().manual_seed(seed + rows + dim)
    w = torch.randn(vocab, dim, generator=g) * 2 / math.sqrt(dim)
    w[:, 0] = 1
    targets = torch.randperm(vocab, generator=g)[:rows]
    h = w[targets] * torch.linspace(2.9, 4.0, rows)[:, None]
    h[:, 0] = 15
    return h.bfloat16().cuda(), w.bfloat16().cuda(), targets.cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,dim,vocab", [(40, 2560, 1000), (256, 2560, 1000), (300, 2560, 1003), (40, 40960, 500), (256, 16384, 600),
                                            (200, 640, 1000)])
@pytest.mark.parametrize("which", ["logprob", "all"])
def test_gradient_of_rows_that_are_nearly_certain(rows, dim, vocab, which):
    h, w, targets = peaked(rows, dim, vocab)
    glp, glse, gent = upstream(rows)
    z = logits(h, w)
    at, wlse, went = definition(z, targets)
    rest = -torch.expm1(at)  # 1 - p
    assert rest.min() < 5e-4 and rest.max() < 0.2 and z.max() < 40
    _, lse, entropy = ssd.ssd_head_logprob_fwd(h, w, targets)
    kw = dict(dlogprob=glp) if which == "logprob" else dict(dlogprob=glp, dlse=1e-4 * glse, dentropy=1e-4 * gent)
    dh, dw = ssd.ssd_head_logprob_bwd(h, w, targets, lse, entropy, **kw)
    zero = torch.zeros(rows, dtype=torch.float64)
    a, b, c = (ref.d(glp), ref.d(1e-4 * glse), ref.d(1e-4 * gent)) if which == "all" else (ref.d(glp), zero, zero)
    d = want_gradient(z, targets.cpu(), wlse, went, a, b, c)
    # The given token's dz: 1 - p is exp of a difference of logits, which are fp32 sums in shares of at most 1280 (80 additions,
    # each off by up to 2^-23 of a sum up to 35, 3e-4; both sides alike), so 1e-3 of it; and lse's rounding, half a step, with its
    # logarithm's, 3e-7.  What else is given to the row: 1e-4 of p, good to 2e-5 of that.  The others as in
    # test_gradient.
    size = a.abs() + b.abs() + 40 * c.abs()
    err = d.abs() * 2.0 ** -8 + 1e-3 * torch.exp(z - wlse[:, None]) * size[:, None]
    k = torch.arange(rows)
    err[k, targets.cpu()] = a.abs() * (1e-3 * rest + 2.0 ** -24 * wlse + 3e-7) + 2e-5 * (b.abs() + 40 * c.abs())
    for got, x, e2, name in ((dh, d @ ref.d(w), (err ** 2) @ (ref.d(w) ** 2), "dhidden"),
                             (dw, d.t() @ ref.d(h), (err.t() ** 2) @ (ref.d(h) ** 2), "dweight")):
        ref.check(got, x, name, rel=1.0, scale=5 / math.sqrt(3) * e2.sqrt() + 1e-30)


@pytest.mark.gpu
def test_gradient_agrees_with_differences():
    h, w, targets = make(96, 128, 900, seed=4)
    glp, glse, gent = upstream(96)
    _, lse, entropy = ssd.ssd_head_logprob_fwd(h, w, targets)
    dh, dw = ssd.ssd_head_logprob_bwd(h, w, targets, lse, entropy, dlogprob=glp, dlse=glse, dentropy=gent)
    g = torch.Generator(device="cuda").manual_seed(2)
    for i, grad in enumerate((dh, dw)):
        v = torch.randn(grad.shape, generator=g, device="cuda")
        vals, moved = [], []
        for e in (0.03, -0.03):
            at = [h, w]
            at[i] = (at[i].float() + e * v * (1.0 if i == 0 else 0.1)).bfloat16()
            lp, ls, en = ssd.ssd_head_logprob_fwd(*at, targets)
            vals.append((lp.double() * glp + ls.double() * glse + en.double() * gent).sum())
            moved.append(at[i].double())
        step = moved[0] - moved[1]  # what rounding the operands to bf16 left of the step
        slope, along = float(vals[0] - vals[1]), float((grad.double() * step).sum())
        # truncation of third order at steps of 0.03, bf16 gradients: a few per cent of |grad| |step| at random directions
        assert abs(slope - along) <= 5e-3 * float(grad.double().norm() * step.norm()), i


@pytest.mark.gpu
def test_agrees_with_stored_logits():
    """The same numbers as from logits in memory, where those are exact in bf16."""
    g = torch.Generator().manual_seed(5)
    h = torch.zeros(200, 64)
    h[torch.arange(200), torch.randint(0, 64, (200,), generator=g)] = 1.0  # picks a column of the weights
    w = torch.randn(3001, 64, generator=g).bfloat16()
    h, w = h.bfloat16().cuda(), w.cuda()
    targets = torch.randint(0, 3001, (200,), generator=g).cuda()
    z = (h.float() @ w.float().t()).bfloat16()
    a = ssd.ssd_head_logprob_fwd(h, w, targets)
    b = ssd.ssd_token_logprob_fwd(z, targets)
    for x, y in zip(a, b):
        ref.check(x, ref.d(y), "", rel=3e-6, scale=20.0)  # two orders of the sums


@pytest.mark.gpu
def test_targets_and_infinities():
    h, w, targets = make(130, 64, 500, seed=6)
    targets[0], targets[1], targets[2] = 500, 1 << 40, -(1 << 40)
    logprob, lse, entropy = ssd.ssd_head_logprob_fwd(h, w, targets)
    assert torch.isnan(logprob[:2]).all() and logprob[2] == 0 and torch.isfinite(logprob[3:]).all() and torch.isfinite(lse).all()
    h[5, 3] = math.nan
    h[129, 0] = math.inf
    logprob, lse, entropy = ssd.ssd_head_logprob_fwd(h, w, targets)
    assert torch.isnan(lse[5]) and torch.isnan(entropy[5]) and not torch.isfinite(lse[129])
    keep = torch.ones(130, dtype=torch.bool)
    keep[[0, 1, 5, 129]] = False
    assert torch.isfinite(lse[keep]).all() and torch.isfinite(logprob[keep]).all()


@pytest.mark.gpu
def test_strides_leading_dimensions_and_what_is_wanted():
    h, w, targets = make(24, 96, 700, seed=7)
    glp = upstream(24)[0]
    first = ssd.ssd_head_logprob_fwd(h, w, targets)
    grads = ssd.ssd_head_logprob_bwd(h, w, targets, first[1], dlogprob=glp)
    wide_h = torch.full((24, 160), math.nan, dtype=torch.bfloat16, device="cuda")
    wide_w = torch.full((700, 160), math.nan, dtype=torch.bfloat16, device="cuda")
    wide_h[:, 8:104], wide_w[:, 32:128] = h, w
    hs, ws = wide_h[:, 8:104], wide_w[:, 32:128]
    for x, y in zip(first, ssd.ssd_head_logprob_fwd(hs, ws, targets)):
        assert torch.equal(x, y)
    for x, y in zip(grads, ssd.ssd_head_logprob_bwd(hs, ws, targets, first[1], dlogprob=glp)):
        assert torch.equal(x, y)
    for x, y in zip(first, ssd.ssd_head_logprob_fwd(h.view(4, 6, 96), w, targets.view(4, 6))):
        assert torch.equal(x, y.reshape(x.shape)) and y.shape == (4, 6)
    a, b = ssd.ssd_head_logprob_bwd(h.view(4, 6, 96), w, targets.view(4, 6), first[1].view(4, 6), dlogprob=glp.view(4, 6),
                                    need_dweight=False)
    assert b is None and torch.equal(a.reshape(24, 96), grads[0])
    a, b = ssd.ssd_head_logprob_bwd(h, w, targets, first[1], dlogprob=glp, need_dhidden=False)
    assert a is None and torch.equal(b, grads[1])
    logprob, lse, entropy = ssd.ssd_head_logprob_fwd(h, w, return_entropy=False)
    assert logprob is None and entropy is None and torch.equal(lse, first[1])


@pytest.mark.gpu
def test_captured_on_a_stream_and_bitwise():
    h, w, targets = make(300, 320, 9001, seed=8)
    glp, glse, gent = upstream(300)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kw = dict(dlogprob=glp, dlse=glse, dentropy=gent)
    first = ssd.ssd_head_logprob_fwd(h, w, targets, stream=s)
    first += ssd.ssd_head_logprob_bwd(h, w, targets, first[1], first[2], **kw, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")  # one workspace for all of it
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ssd.ssd_head_logprob_fwd(h, w, targets, workspace=ws)
        out += ssd.ssd_head_logprob_bwd(h, w, targets, out[1], out[2], **kw, workspace=ws)
    ws.fill_(255)  # NaN everywhere: nothing is read that was not written
    graph.replay()
    for a, b in zip(first, out):
        assert torch.equal(a, b)
    h.normal_()
    graph.replay()
    again = ssd.ssd_head_logprob_fwd(h, w, targets)
    again += ssd.ssd_head_logprob_bwd(h, w, targets, again[1], again[2], **kw)
    for a, b in zip(out, again):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_no_rows():
    w = torch.randn(100, 64, device="cuda").bfloat16()
    h = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(0, dtype=torch.int64, device="cuda")
    logprob, lse, entropy = ssd.ssd_head_logprob_fwd(h, w, t)
    assert logprob.shape == lse.shape == (0,)
    dh, dw = ssd.ssd_head_logprob_bwd(h, w, t, lse, dlogprob=lse)
    assert dh.shape == (0, 64) and bool((dw == 0).all())


# ---- refusals (host only) --------------------------------------------------
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from state_space_model_fwd_gb300 import _build
    _build.build()
    return ssd.load_library()


def c_call(lib, bwd=False, hidden=(FAKE, 0, 64), weight=(FAKE, 0, 64), dh=(FAKE, 0, 64), dw=(FAKE, 0, 64), targets=FAKE,
           logprob=FAKE, lse=FAKE, entropy=FAKE, glp=FAKE, gent=None, ws=(None, 0), **kw):
    from state_space_model_fwd_gb300 import _layer, _logprob
    v = dict(rows=4, vocab=1000, dim=64, dtype=1)
    v.update(kw)
    shape = _logprob._head_shape_t(v["rows"], v["vocab"], v["dim"], v["dtype"])
    r = lambda t: ctypes.byref(_layer._rows_t(*t))
    if bwd:
        return lib.ssd_head_logprob_bwd(ctypes.byref(shape), r(hidden), r(weight), targets, lse, entropy, glp, None, gent, r(dh),
                                        r(dw), ws[0], ws[1], None), lib.ssd_head_logprob_bwd_workspace_size(ctypes.byref(shape))
    return lib.ssd_head_logprob_fwd(ctypes.byref(shape), r(hidden), r(weight), targets, logprob, lse, entropy, ws[0], ws[1],
                                    None), lib.ssd_head_logprob_workspace_size(ctypes.byref(shape))


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(vocab=0), INVALID), (dict(rows=-1), INVALID), (dict(dim=0), INVALID), (dict(dtype=7), INVALID),
    (dict(dtype=0), UNSUPPORTED), (dict(dim=60), UNSUPPORTED), (dict(vocab=(1 << 22) + 1), UNSUPPORTED),
    (dict(rows=(1 << 22) + 1), UNSUPPORTED), (dict(rows=1 << 22, vocab=1 << 22), UNSUPPORTED),
])
def test_shapes_are_checked(lib, bwd, kw, code):
    st, size = c_call(lib, bwd, **kw)
    assert st == code and size == 0


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw", [
    dict(hidden=(None, 0, 64)), dict(hidden=(FAKE + 8, 0, 64)), dict(hidden=(FAKE, 0, 68)), dict(hidden=(FAKE, 0, 0)),
    dict(weight=(FAKE, 0, 56)), dict(weight=(FAKE + 2, 0, 64)), dict(targets=FAKE + 4), dict(lse=FAKE + 1), dict(targets=None),
])
def test_operands_are_checked(lib, bwd, kw):
    assert c_call(lib, bwd, **kw)[0] == INVALID


@pytest.mark.parametrize("kw", [dict(lse=None), dict(entropy=None, gent=FAKE), dict(dh=(FAKE, 0, 60)), dict(dw=(FAKE + 8, 0, 64)),
                                dict(dw=(FAKE, 0, 0))])
def test_operands_of_the_gradient_are_checked(lib, kw):
    assert c_call(lib, True, **kw)[0] == INVALID


@pytest.mark.parametrize("bwd", [False, True])
def test_workspace_is_checked(lib, bwd):
    st, size = c_call(lib, bwd)
    assert st == WORKSPACE and size > 0
    assert c_call(lib, bwd, ws=(FAKE, size - 1))[0] == WORKSPACE
    assert c_call(lib, bwd, ws=(FAKE + 8, size))[0] == WORKSPACE


@pytest.mark.gpu
def test_binding_refuses_on_the_gpu():
    h, w, targets = make(4, 64, 100)
    lse = torch.zeros(4, device="cuda")
    with pytest.raises(ssd.SSDError):
        ssd.ssd_head_logprob_fwd(h.float(), w.float(), targets)
    with pytest.raises(TypeError):
        ssd.ssd_head_logprob_fwd(h, w.float(), targets)
    with pytest.raises(ValueError):
        ssd.ssd_head_logprob_fwd(h, w[:, :56].contiguous(), targets)
    with pytest.raises(ssd.SSDError):
        ssd.ssd_head_logprob_fwd(h[:, :60].contiguous(), w[:, :60].contiguous(), targets)
    with pytest.raises(ssd.SSDError):  # rows off their 16-byte boundary
        ssd.ssd_head_logprob_fwd(torch.zeros(4, 68, dtype=torch.bfloat16, device="cuda")[:, :64], w, targets)
    with pytest.raises(ValueError):
        ssd.ssd_head_logprob_bwd(h, w, None, lse, dlogprob=lse)
    with pytest.raises(ValueError):
        ssd.ssd_head_logprob_bwd(h, w, targets, lse, dentropy=lse)
