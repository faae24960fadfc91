"""Log-probabilities, entropies and top alternatives on the GPU against their
definitions in float64, and the gradient."""
import ctypes
import math

import pytest
import torch

import state_space_model_fwd_gb300 as ssd
from tests import layer_reference as ref

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def definition(z, targets):
    """(logprob, lse, entropy) of float64 rows."""
    lse = torch.logsumexp(z, -1)
    none = lse == -math.inf
    lp = torch.where(none[:, None], -math.inf, z - torch.where(none, 0.0, lse)[:, None])
    entropy = torch.special.entr(torch.exp(lp)).sum(-1)
    logprob = None
    if targets is not None:
        t = targets.cpu()
        logprob = torch.where(t < 0, 0.0, lp.gather(1, t.clamp(min=0)[:, None])[:, 0])
    return logprob, lse, entropy


def top_of(z, k):
    """Indices of the k largest, equal ones by index, NaN first."""
    return torch.sort(z, dim=-1, descending=True, stable=True)[1][:, :k]


def make(dtype, rows, vocab, std=3.0, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed * 101 + rows * 7 + vocab)
    z = (std * torch.randn(rows, vocab + pad, generator=g)).to(DT[dtype]).cuda()[:, pad:]
    return z, torch.randint(0, vocab, (rows,), generator=g).cuda()


def check_rows(got, z, targets, top):
    """z: float64 on the CPU"""
    logprob, lse, entropy, value, index = got
    wlp, wlse, went = definition(z, targets)
    # lse = m + log(sum): the sum is good to a few 2^-22 (exponential, rounded argument, additions), the last addition rounds;
    # the entropy is a difference of the log and a mean of z - m, up to log(vocab) + spread each
    size = 1 + wlse.abs().nan_to_num(0, 0, 0)
    ref.check(lse, wlse, "lse", rel=2e-6, scale=size)
    ref.check(entropy, went, "entropy", rel=3e-6, scale=size + 12)
    if targets is None:
        assert logprob is None
    else:
        ref.check(logprob, wlp, "logprob", rel=2e-6, scale=size + wlp.abs().nan_to_num(0, 0, 0))
    if not top:
        assert value is None and index is None
        return
    want = top_of(z, top)
    assert index.dtype == torch.int64 and torch.equal(index.cpu(), want)
    wv = z.gather(1, want)
    wv = torch.where(wlse[:, None] == -math.inf, wv, wv - torch.where(wlse == -math.inf, 0.0, wlse)[:, None])
    wv = torch.where(wv < -torch.finfo(torch.float32).max, -math.inf, wv)  # (the lowest value less the highest: past fp32's range)
    ref.check(value, wv, "top", rel=2e-6, scale=(size[:, None] + wv.abs()).nan_to_num(1, 1, 1))


# rows, vocabularies of one part and of several, odd ones, alternatives from none to the most, columns before
CASES = [
    ("f32", 1, 1, 1, 0), ("bf16", 3, 7, 7, 0), ("bf16", 5, 8, 3, 0), ("f32", 4, 1000, 0, 0), ("bf16", 300, 1003, 5, 1),
    ("bf16", 2, 4097, 64, 3), ("f32", 2, 8192, 8, 1), ("bf16", 4, 50280, 8, 0), ("bf16", 1, 131071, 64, 5), ("f32", 3, 65537, 20, 0),
    ("bf16", 200, 16385, 1, 0), ("f32", 400, 9000, 64, 2), ("bf16", 33, 32768, 64, 8),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,rows,vocab,top,pad", CASES)
def test_forward(dtype, rows, vocab, top, pad):
    z, targets = make(dtype, rows, vocab, pad=pad)
    targets[rows // 2] = -100 if rows > 2 else targets[0]
    check_rows(ssd.ssd_token_logprob_fwd(z, targets, top=top), ref.d(z), targets, top)
    check_rows(ssd.ssd_token_logprob_fwd(z, top=top), ref.d(z), None, top)


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [40, 5000, 40000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_rows(dtype, vocab):
    """Half the tokens masked; one token left; none left; finite masks of the type's lowest value."""
    z, targets = make(dtype, 6, vocab, seed=1)
    g = torch.Generator().manual_seed(5)
    z[torch.rand(6, vocab, generator=g).cuda() < 0.5] = -math.inf
    z[1] = -math.inf
    z[1, vocab - 3] = 2.5
    z[2] = -math.inf
    z[3] = torch.finfo(DT[dtype]).min
    z[4] = torch.finfo(DT[dtype]).min
    z[4, 11] = torch.finfo(DT[dtype]).max
    top = min(vocab, 64)
    targets[1] = vocab - 3
    targets[4] = 11
    check_rows(ssd.ssd_token_logprob_fwd(z, targets, top=top), ref.d(z), targets, top)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 700])
@pytest.mark.parametrize("what", ["equal", "two values", "rising", "falling", "few threads", "zeros", "nan"])
def test_alternatives_in_any_order(what, rows):
    """Ties, and orders that put the largest values into few threads' hands."""
    vocab = 50003
    i = torch.arange(vocab, dtype=torch.float32)
    if what == "equal":
        z = torch.full((vocab,), 1.5)
    elif what == "two values":
        z = (i % 1000 == 7).float()
    elif what == "rising":
        z = i * 1e-3
    elif what == "falling":
        z = -i * 1e-3
    elif what == "few threads":  # the same places of every 4096 columns, then of every 2048
        z = torch.where((i % 4096 < 128) | (i % 2048 < 64), 5 + i * 1e-5, -i * 1e-6)
    elif what == "zeros":
        z = torch.where(i % 2 == 0, torch.tensor(-0.0), torch.tensor(0.0))
    else:
        z = torch.sin(i)
        z[[3, 40000, 17]] = math.nan
    z = z.expand(rows, vocab).contiguous().cuda()
    got = ssd.ssd_token_logprob_fwd(z, top=64)
    want = top_of(ref.d(z[:1]), 64)
    assert torch.equal(got[4].cpu(), want.expand(rows, 64))
    if what != "nan":
        check_rows(ssd.ssd_token_logprob_fwd(z[:1], top=64), ref.d(z[:1]), None, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 700])
@pytest.mark.parametrize("what", ["all nan", "mostly nan", "nan first", "equal", "two values", "rising", "falling", "few threads"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_alternatives_of_either_type_in_any_order(dtype, what, rows):
    """More equal ones than there is room for, NaN among them, the first token's included."""
    vocab = 50003
    i = torch.arange(vocab, dtype=torch.float32)
    if what == "all nan":
        z = torch.full((vocab,), math.nan)
    elif what == "mostly nan":
        z = torch.where(i % 9 == 4, torch.sin(i), torch.tensor(math.nan))
    elif what == "nan first":
        z = torch.where(i < 30, torch.tensor(math.nan), torch.sin(i))
    elif what == "equal":
        z = torch.full((vocab,), 1.5)
    elif what == "two values":
        z = (i % 1000 == 7).float()
    elif what == "rising":
        z = i * 1e-3
    elif what == "falling":
        z = -i * 1e-3
    else:
        z = torch.where((i % 4096 < 128) | (i % 2048 < 64), 5 + i * 1e-5, -i * 1e-6)
    z = z.to(DT[dtype]).expand(rows, vocab).contiguous().cuda()
    for top in (1, 5, 64):
        got = ssd.ssd_token_logprob_fwd(z, top=top)
        assert torch.equal(got[4].cpu(), top_of(ref.d(z[:1]), top).expand(rows, top)), top


@pytest.mark.gpu
def test_infinity_and_nan():
    z, targets = make("f32", 3, 9000, seed=2)
    z[0, 77] = math.inf
    z[1, 8999] = math.nan
    targets[0] = 5
    logprob, lse, entropy, _, _ = ssd.ssd_token_logprob_fwd(z, targets)
    assert lse[0] == math.inf and logprob[0] == -math.inf and torch.isnan(entropy[0])
    assert torch.isnan(lse[1]) and torch.isnan(logprob[1]) and torch.isnan(entropy[1])
    assert torch.isfinite(lse[2]) and torch.isfinite(entropy[2])
    targets[2] = 9000
    logprob, lse, entropy, _, _ = ssd.ssd_token_logprob_fwd(z, targets)
    assert torch.isnan(logprob[2]) and torch.isfinite(lse[2])


def grads(rows, seed=3):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(rows, generator=g).cuda() for _ in range(3)]


def want_gradient(z, targets, lse, entropy, glp, glse, gent):
    """The formula, with the chain rule's three parts apart."""
    lp = z - lse[:, None]
    p = torch.exp(lp)
    hit = torch.zeros_like(z)
    has = targets >= 0
    hit[has, targets[has]] = 1.0
    d = torch.where(has, glp, 0.0)[:, None] * (hit - p) + glse[:, None] * p
    return d - gent[:, None] * torch.where(p > 0, p * (lp + entropy[:, None]), 0.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,rows,vocab,pad", [
    ("f32", 1, 1, 0), ("bf16", 3, 7, 0), ("bf16", 5, 8, 1), ("f32", 4, 1001, 0), ("bf16", 40, 8193, 0), ("bf16", 3, 20000, 3),
    ("f32", 7, 4096, 2)])
@pytest.mark.parametrize("which", ["logprob", "all"])
def test_gradient(dtype, rows, vocab, pad, which):
    z, targets = make(dtype, rows, vocab, pad=pad, seed=4)
    targets[0] = -1
    glp, glse, gent = grads(rows)
    _, lse, entropy, _, _ = ssd.ssd_token_logprob_fwd(z, targets)
    kw = dict(dlogprob=glp) if which == "logprob" else dict(dlogprob=glp, dlse=glse, dentropy=gent)
    got = ssd.ssd_token_logprob_bwd(z, targets, lse, entropy, **kw)
    zd = ref.d(z)
    zero = torch.zeros(rows, dtype=torch.float64)
    _, wlse, went = definition(zd, targets)
    a, b, c = (ref.d(glp), ref.d(glse), ref.d(gent)) if which == "all" else (ref.d(glp), zero, zero)
    want = want_gradient(zd, targets.cpu(), wlse, went, a, b, c)
    # p is good to 2^-22 plus the rounding of lse and z - lse (2e-6 at 30) and is multiplied by up to |log p| + entropy
    size = (a.abs() + b.abs() + c.abs() * 40)[:, None] * torch.exp(zd - wlse[:, None]) + 1e-30
    hit = torch.zeros_like(zd)
    hit[targets.cpu() >= 0, targets.cpu()[targets.cpu() >= 0]] = 1.0
    ref.check(got, want, "dlogits", rel=5e-6, scale=size + hit * a.abs()[:, None])


@pytest.mark.gpu
def test_gradient_agrees_with_differences():
    z, targets = make("f32", 5, 300, std=2.0, seed=6)
    glp, glse, gent = grads(5)
    g = torch.Generator(device="cuda").manual_seed(1)
    v = torch.randn(5, 300, generator=g, device="cuda")
    _, lse, entropy, _, _ = ssd.ssd_token_logprob_fwd(z, targets)
    d = ssd.ssd_token_logprob_bwd(z, targets, lse, entropy, dlogprob=glp, dlse=glse, dentropy=gent)
    vals = []
    for e in (1e-2, -1e-2):
        lp, ls, en, _, _ = ssd.ssd_token_logprob_fwd(z + e * v, targets)
        vals.append((lp.double() * glp + ls.double() * glse + en.double() * gent).sum())
    slope = float(vals[0] - vals[1]) / 2e-2
    # truncation 1e-4 / 6 of the third derivative, fp32 rounding 1e-6 over the step
    assert abs(slope - float((d.double() * v).sum())) <= 2e-3 * float(d.double().norm() * v.double().norm())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_of_masked_rows(dtype):
    z, targets = make(dtype, 4, 5000, seed=7)
    z[:, ::3] = -math.inf
    z[2] = -math.inf
    targets[0], targets[1] = 0, 1     # a masked token given, and one that is not
    glp, glse, gent = grads(4)
    logprob, lse, entropy, _, _ = ssd.ssd_token_logprob_fwd(z, targets)
    assert logprob[0] == -math.inf and torch.isfinite(logprob[1])
    d = ssd.ssd_token_logprob_bwd(z, targets, lse, entropy, dlogprob=glp, dlse=glse, dentropy=gent)
    assert torch.isfinite(d).all() and bool((d[2] == 0).all())
    assert bool((d[1, ::3] == 0).all()) and d[0, 0] == glp[0].to(d.dtype) and bool((d[0, 3::3] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,vocab", [("bf16", 1003), ("f32", 4096), ("bf16", 20000)])
def test_in_place_strided_and_leading_dimensions(dtype, vocab):
    z, targets = make(dtype, 12, vocab, seed=8)
    glp, _, gent = grads(12)
    got = ssd.ssd_token_logprob_fwd(z, targets, top=4)
    shaped = ssd.ssd_token_logprob_fwd(z.view(3, 4, vocab), targets.view(3, 4), top=4)
    for a, b in zip(got, shaped):
        assert torch.equal(a, b.reshape(a.shape))
    _, lse, entropy, _, _ = got
    want = ssd.ssd_token_logprob_bwd(z, targets, lse, entropy, dlogprob=glp, dentropy=gent)
    # among NaN, at another alignment, into a slice whose surroundings stay
    for off in (0, 1, 8):
        wide = torch.full((12, vocab + 16), float("nan"), dtype=DT[dtype], device="cuda")
        wide[:, off:off + vocab] = z
        out = torch.full((12, vocab + 16), 7.0, dtype=DT[dtype], device="cuda")
        again = ssd.ssd_token_logprob_fwd(wide[:, off:off + vocab], targets, top=4)
        assert torch.equal(again[4], got[4]) and torch.isfinite(again[1]).all()
        d = ssd.ssd_token_logprob_bwd(wide[:, off:off + vocab], targets, lse, entropy, dlogprob=glp, dentropy=gent,
                                      dlogits=out[:, 3:3 + vocab])
        assert torch.equal(d, want)
        d[:] = 7.0
        assert bool((out == 7.0).all())
    copy = z.clone()
    assert torch.equal(ssd.ssd_token_logprob_bwd(copy, targets, lse, entropy, dlogprob=glp, dentropy=gent, dlogits=copy), want)
    assert copy.data_ptr() and torch.equal(copy, want)


@pytest.mark.gpu
def test_rows_far_apart():
    """The last rows of long prompts' logits: more than 2^31 elements from one to the next."""
    far = (1 << 31) + 8
    rows = torch.empty(far + 1000, dtype=torch.bfloat16, device="cuda").as_strided((2, 1000), (far, 1))
    rows[:] = make("bf16", 2, 1000, seed=11)[0]
    targets = torch.tensor([3, 999], device="cuda")
    got = ssd.ssd_token_logprob_fwd(rows, targets, top=3)
    for a, b in zip(got, ssd.ssd_token_logprob_fwd(rows.contiguous(), targets, top=3)):
        assert torch.equal(a, b)
    want = ssd.ssd_token_logprob_bwd(rows.contiguous(), targets, got[1], dlogprob=got[1])
    assert torch.equal(ssd.ssd_token_logprob_bwd(rows, targets, got[1], dlogprob=got[1], dlogits=rows), want)
    one = rows[:1].as_strided((1, 1000), (1 << 39, 1))  # (a single row's stride means nothing)
    assert torch.equal(ssd.ssd_token_logprob_fwd(one)[1], ssd.ssd_token_logprob_fwd(want[:1] * 0 + one)[1])


@pytest.mark.gpu
def test_more_than_2_31_elements():
    rows, vocab, few = 43000, 50277, 100
    z = torch.empty(rows, vocab, dtype=torch.bfloat16, device="cuda").normal_()
    targets = torch.randint(0, vocab, (rows,), device="cuda")
    glp = torch.randn(rows, device="cuda")
    got = ssd.ssd_token_logprob_fwd(z, targets, top=3)
    part = ssd.ssd_token_logprob_fwd(z[-few:], targets[-few:], top=3)
    # Of few rows each is shared by two blocks, of many it is not: the same positive terms in another order.  A thread adds up
    # to 200 of them, each addition off by 2^-24 of the sum so far, so the sums of two calls differ by 2 * 200 * 2^-24 = 2.4e-5
    # at most, lse and log-probabilities by as much, the entropy by (1 + 2 moment / sum) times that, below 17 times.
    for a, b, size in zip(got, part, (1, 1, 17, 1)):
        assert bool(((a[-few:] - b).abs() <= 2.5e-5 * size).all())
    assert torch.equal(got[4][-few:], part[4])
    want = ssd.ssd_token_logprob_bwd(z[-few:], targets[-few:], got[1][-few:].contiguous(), dlogprob=glp[-few:])
    assert torch.equal(ssd.ssd_token_logprob_bwd(z, targets, got[1], dlogprob=glp, dlogits=z)[-few:], want)


@pytest.mark.gpu
def test_captured_on_a_stream_and_bitwise():
    z, targets = make("bf16", 3, 50280, seed=9)
    glp = grads(3)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    first = ssd.ssd_token_logprob_fwd(z, targets, top=10, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = ssd.ssd_token_logprob_fwd(z, targets, top=10)
        d = ssd.ssd_token_logprob_bwd(z, targets, out[1], dlogprob=glp)
    g.replay()
    for a, b in zip(first, out):
        assert torch.equal(a, b)
    assert torch.equal(d, ssd.ssd_token_logprob_bwd(z, targets, first[1], dlogprob=glp))
    z.normal_()
    g.replay()
    for a, b in zip(out, ssd.ssd_token_logprob_fwd(z, targets, top=10)):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_no_rows():
    z = torch.zeros(0, 100, device="cuda")
    got = ssd.ssd_token_logprob_fwd(z, torch.zeros(0, dtype=torch.int64, device="cuda"), top=3)
    assert got[0].shape == (0,) and got[4].shape == (0, 3)
    assert ssd.ssd_token_logprob_bwd(z, None, got[1]).shape == (0, 100)


# ---- refusals (host only) --------------------------------------------------
OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from state_space_model_fwd_gb300 import _build
    _build.build()
    return ssd.load_library()


def c_call(lib, bwd=False, logits=(FAKE, 0, 1000), out=(FAKE, 0, 1000), targets=FAKE, logprob=FAKE, lse=FAKE, entropy=FAKE,
           value=FAKE, index=FAKE, glp=FAKE, gent=None, **kw):
    from state_space_model_fwd_gb300 import _layer, _logprob
    v = dict(rows=4, vocab=1000, top=0, dtype=1)
    v.update(kw)
    shape = _logprob._logprob_shape_t(v["rows"], v["vocab"], v["top"], v["dtype"])
    zr = _layer._rows_t(*logits)
    if bwd:
        return lib.ssd_token_logprob_bwd(ctypes.byref(shape), ctypes.byref(zr), targets, lse, entropy, glp, None, gent,
                                         ctypes.byref(_layer._rows_t(*out)), None)
    return lib.ssd_token_logprob_fwd(ctypes.byref(shape), ctypes.byref(zr), targets, logprob, lse, entropy, value, index, None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(vocab=0), INVALID), (dict(rows=-1), INVALID), (dict(dtype=3), INVALID), (dict(top=-1), INVALID),
    (dict(vocab=10, top=11), INVALID), (dict(top=65), UNSUPPORTED), (dict(vocab=(1 << 30) + 1), UNSUPPORTED),
    (dict(rows=(1 << 28) + 1), UNSUPPORTED), (dict(logits=(None, 0, 1000)), INVALID), (dict(logits=(FAKE + 1, 0, 1000)), INVALID),
    (dict(logits=(FAKE, 0, -1)), INVALID), (dict(logits=(FAKE, 0, 1 << 40)), INVALID), (dict(targets=FAKE + 4), INVALID),
    (dict(targets=None), INVALID), (dict(lse=FAKE + 2), INVALID), (dict(rows=0), OK),
])
def test_arguments_are_checked(lib, bwd, kw, code):
    assert c_call(lib, bwd, **kw) == code


@pytest.mark.parametrize("bwd,kw", [
    (False, dict(top=3, value=None)), (False, dict(top=3, index=None)), (False, dict(top=3, index=FAKE + 4)),
    (True, dict(lse=None)), (True, dict(out=(FAKE, 0, 999))), (True, dict(out=(None, 0, 1000))), (True, dict(entropy=None, gent=FAKE)),
])
def test_operands_that_have_to_be_there(lib, bwd, kw):
    assert c_call(lib, bwd, **kw) == INVALID


@pytest.mark.gpu
def test_binding_refuses_on_the_gpu():
    z, targets = make("f32", 4, 100)
    lse = torch.zeros(4, device="cuda")
    with pytest.raises(TypeError):
        ssd.ssd_token_logprob_fwd(z.half(), targets)
    with pytest.raises(TypeError):
        ssd.ssd_token_logprob_fwd(z, targets.int())
    with pytest.raises(ValueError):
        ssd.ssd_token_logprob_fwd(z, targets[:3])
    with pytest.raises(ValueError):
        ssd.ssd_token_logprob_fwd(z.t(), targets)
    with pytest.raises(ssd.SSDError):
        ssd.ssd_token_logprob_fwd(z, targets, top=65)
    with pytest.raises(ssd.SSDError):
        ssd.ssd_token_logprob_fwd(z, targets, top=101)
    for top in (-1, 1 << 50):
        with pytest.raises(ssd.SSDError):
            ssd.ssd_token_logprob_fwd(z, targets, top=top)
    with pytest.raises(TypeError):
        ssd.ssd_token_logprob_bwd(z, targets, None)
    with pytest.raises(ValueError):
        ssd.ssd_token_logprob_bwd(z, None, lse, dlogprob=lse)
    with pytest.raises(ValueError):
        ssd.ssd_token_logprob_bwd(z, targets, lse, dentropy=lse)
    with pytest.raises(ValueError):
        ssd.ssd_token_logprob_bwd(z, targets, lse, dlogprob=lse, dlogits=torch.zeros(100, 4, device="cuda").t())
