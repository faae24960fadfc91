"""The operators around a state-space layer's scan, as cases to be measured.

Three operators, each with the directions that a program uses:

  conv  causal depthwise convolution over the last few tokens, with bias and SiLU: prompts, gradient, one token
  scan  selective scan with a decay per channel and state (h = exp(dt A) h + dt x B, y = C h + D x, gated by
        silu(z)): prompts, gradient, one token
  norm  RMS norm fused with the gate before or after it and the scaled residual: forward, gradient

`own` False runs the formulas as elementary torch operations in fp32; `own`
True runs the calls a user makes.  Batches are either `batch` sequences of
`seqlen` tokens, or `nseq` sequences of unequal lengths packed back to back
into `seqlen` tokens (`cut` draws the offsets).
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token of four conversations: the convolution of a 130M-shaped Mamba-2 layer (1536 + 2*128 channels), where
        # only latency counts
        dict(name="conv_token_small", op="conv_step", dtype="bf16", batch=4, channels=1792, width=4, row=3352, bias=True),
        # the same layer's prompt: four prompts of 2048 tokens, read in place out of the projection's rows (z | x B C | dt)
        # and written as the x, B and C that the chunked scan takes
        dict(name="conv_prompt", op="conv", dtype="bf16", batch=4, seqlen=2048, nseq=0, cut=0, channels=1792, width=4,
             row=3352, parts="1536,128,128", bias=True, init=False),
        # a packed prefill of a 2.7B-shaped layer (5120 + 2*128 channels): 48 prompts of unequal lengths that continue
        # from cached states
        dict(name="conv_packed_large", op="conv", dtype="bf16", batch=1, seqlen=65537, nseq=48, cut=5, channels=5376, width=4,
             row=10576, parts="5120,128,128", bias=True, init=True),
        # one training step's gradient, odd length
        dict(name="conv_grad", op="conv_grad", dtype="bf16", batch=4, seqlen=4095, nseq=0, cut=0, channels=2560, width=4,
             row=2560, parts="2560", bias=True, init=False),
        # one token of 128 conversations: the state is read and written once
        dict(name="scan_token", op="scan_step", dtype="bf16", batch=128, channels=5120, dstate=16, gate=True),
        # a single prompt, few channels: little to run side by side
        dict(name="scan_prompt_one", op="scan", dtype="bf16", batch=1, seqlen=2048, nseq=0, cut=0, channels=1536, dstate=16,
             groups=1, gate=True, init=False),
        # a batch of long prompts: the largest scan
        dict(name="scan_prompt_large", op="scan", dtype="bf16", batch=8, seqlen=4096, nseq=0, cut=0, channels=5120, dstate=16,
             groups=1, gate=True, init=True),
        # ragged prompts in fp32 with states carried in, an odd number of channels
        dict(name="scan_packed_f32", op="scan", dtype="f32", batch=1, seqlen=9001, nseq=23, cut=3, channels=1001, dstate=16,
             groups=1, gate=False, init=True),
        # one training step's gradient
        dict(name="scan_grad", op="scan_grad", dtype="bf16", batch=4, seqlen=2048, nseq=0, cut=0, channels=1536, dstate=16,
             groups=1, gate=True, init=False),
        # the gradient over packed documents in fp32, with shared B and C in two groups
        dict(name="scan_grad_packed_f32", op="scan_grad", dtype="f32", batch=1, seqlen=4097, nseq=9, cut=7, channels=640,
             dstate=32, groups=2, gate=True, init=True),
        # the gated norm between scan and output projection, over a prefill of a 2.7B-shaped layer
        dict(name="norm_gate", op="norm", dtype="bf16", rows=16384, dim=5120, group=5120, gate="before", residual="none",
             scale=False),
        # the gradient of the norm that opens the next block, with the fp32 residual stream and its learned scale
        dict(name="norm_residual_grad", op="norm_grad", dtype="bf16", rows=8191, dim=2560, group=2560, gate="none",
             residual="f32", scale=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    c = _draw(rng)
    while 3072 in c.values() or "3072" in c.get("parts", ""):
        c = _draw(rng)
    return c


def _draw(rng):
    op = rng.choice(["conv", "conv", "conv_grad", "conv_step", "scan", "scan", "scan_grad", "scan_step", "norm", "norm_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    channels = _log(rng, 48, 5376)
    if rng.random() < 0.6:
        channels = -(-channels // 64) * 64
    if op == "conv_step":
        return dict(op=op, dtype=dtype, batch=_log(rng, 1, 512), channels=channels, width=rng.choice([2, 3, 4]),
                    row=channels + rng.choice([0, 8, 24, 129]), bias=rng.random() < 0.8)
    if op == "scan_step":
        return dict(op=op, dtype=dtype, batch=_log(rng, 1, 512), channels=channels, dstate=rng.choice([8, 16, 16, 32]),
                    gate=rng.random() < 0.7)
    if op in ("norm", "norm_grad"):
        groups = rng.choice([1, 1, 1, 2, 8])
        dim = -(-channels // groups) * groups
        return dict(op=op, dtype=dtype, rows=_log(rng, 1, 16384), dim=dim, group=dim // groups,
                    gate=rng.choice(["none", "before", "after"]), residual=rng.choice(["none", "same", "f32"]),
                    scale=rng.random() < 0.5)
    most = {"conv": 65536 * 4096, "conv_grad": 16384 * 2560, "scan": 32768 * 2560, "scan_grad": 8192 * 1280}[op]
    tokens = max(1, min(_log(rng, 1, 65536), most // channels))
    nseq, batch = (rng.randint(1, 40), 1) if rng.random() < 0.5 else (0, rng.choice([1, 1, 2, 3, 4, 8]))
    seqlen = tokens if nseq else max(1, tokens // batch)
    c = dict(op=op, dtype=dtype, batch=batch, seqlen=seqlen, nseq=nseq, cut=rng.randint(0, 999), channels=channels)
    if op in ("conv", "conv_grad"):
        side = rng.choice([0, 0, 16, 17]) if channels > 64 else 0
        parts = "%d,%d,%d" % (channels - 2 * side, side, side) if side else str(channels)
        c.update(width=rng.choice([2, 3, 4]), row=channels + rng.choice([0, 8, 24, 129]), parts=parts, bias=rng.random() < 0.8)
    else:
        groups = 2 if channels % 2 == 0 and rng.random() < 0.25 else 1
        dstate = rng.choice([8, 16, 16, 16, 32])
        if dstate == 32:
            c["seqlen"] = max(1, seqlen // 2)
        c.update(dstate=dstate, groups=groups, gate=rng.random() < 0.7)
    c["init"] = rng.random() < 0.5
    return c


def _offsets(case):
    """Sequence offsets of a packed batch; None for an equal-length one.  With four or more sequences one is empty and one
    holds a single token, where the tokens allow it."""
    if not case["nseq"]:
        return None
    r = random.Random(case["cut"] * 1000003 + case["seqlen"])
    total, n = case["seqlen"], case["nseq"]
    cu = [0] + sorted(r.randint(0, total) for _ in range(n - 1)) + [total]
    if n >= 4:
        cu[2] = cu[1]
        cu[3] = max(cu[2], min(cu[2] + 1, cu[4]))
    return cu


# ---------------------------------------------------------------------------
# the inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    dtype = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dtype):
        return (torch.randn(*shape, generator=g, device=DEV) * std + mean).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    op = case["op"]
    s = dict(case=case)
    f32 = torch.float32
    if op in ("conv", "conv_grad", "conv_step"):
        b, ch, w, row = case["batch"], case["channels"], case["width"], case["row"]
        at = (row - ch) // 16 * 8  # the columns sit inside a wider row
        s["weight"] = normal(ch, w, std=1 / math.sqrt(w), dtype=f32)
        s["bias"] = normal(ch, std=0.1, dtype=f32) if case["bias"] else None
        if op == "conv_step":
            s["x"] = normal(b, row)[:, at:at + ch]
            s["state"] = normal(b, w - 1, ch)
            return s
        s["cu"] = _offsets(case)
        s["parts"] = [int(v) for v in case["parts"].split(",")]
        s["x"] = normal(b, case["seqlen"], row)[:, :, at:at + ch]
        nst = case["nseq"] or b
        s["init"] = normal(nst, w - 1, ch) if case["init"] else None
        if op == "conv_grad":
            s["dy"] = [normal(b, case["seqlen"], p) for p in s["parts"]]
            s["dfinal"] = normal(nst, w - 1, ch) if case["init"] else None
        return s
    if op in ("scan", "scan_grad", "scan_step"):
        b, ch, n = case["batch"], case["channels"], case["dstate"]
        groups = case.get("groups", 1)
        tok = (b,) if op == "scan_step" else (b, case["seqlen"])
        s["x"], s["dt"] = normal(*tok, ch), normal(*tok, ch, std=0.5)
        s["z"] = normal(*tok, ch) if case["gate"] else None
        s["B"], s["C"] = (normal(*tok, groups, n) for _ in range(2))
        s["A"] = -torch.arange(1, n + 1, device=DEV, dtype=f32) * torch.exp(0.2 * normal(ch, n, dtype=f32))
        s["D"] = normal(ch, std=0.1, mean=1.0, dtype=f32)
        u = torch.exp(math.log(1e-3) + (math.log(1e-1) - math.log(1e-3)) * uniform(ch))
        s["dt_bias"] = u + torch.log(-torch.expm1(-u))
        if op == "scan_step":
            s["state"] = normal(b, ch, n, std=0.3, dtype=f32)
            return s
        s["cu"] = _offsets(case)
        nst = case["nseq"] or b
        s["init"] = normal(nst, ch, n, std=0.3, dtype=f32) if case["init"] else None
        if op == "scan_grad":
            s["dy"] = normal(*tok, ch)
            s["dfinal"] = normal(nst, ch, n, std=0.3, dtype=f32) if case["init"] else None
        return s
    rows, dim = case["rows"], case["dim"]
    rdtype = {"none": None, "same": dtype, "f32": f32}[case["residual"]]
    s["x"] = normal(rows, dim)
    s["weight"] = normal(dim, std=0.1, mean=1.0, dtype=f32)
    s["z"] = normal(rows, dim) if case["gate"] != "none" else None
    s["scale"] = normal(dim, std=0.1, mean=0.5, dtype=f32) if case["scale"] else None
    s["residual"] = normal(rows, dim, std=2.0, dtype=rdtype) if rdtype else None
    if op == "norm_grad":
        s["dout"] = normal(rows, dim)
        if rdtype:
            s["dresidual_out"] = normal(rows, dim, dtype=rdtype)
            v = s["x"].float()
            if case["gate"] == "before":
                zf = s["z"].float()
                v = v * zf * torch.sigmoid(zf)
            if case["scale"]:
                v = v * s["scale"]
            s["summed"] = (s["residual"].float() + v).to(rdtype)  # what the forward call returned beside its output
            del s["residual"]
    return s


# ---------------------------------------------------------------------------
# the plain forms: elementary operations in fp32
# ---------------------------------------------------------------------------
def _seq_index(cu, b, seqlen, dev):
    """For every flat token: its sequence, that sequence's first token and the token after its last."""
    if cu is None:
        cu = [seqlen * i for i in range(b + 1)]
    edges = torch.tensor(cu, device=dev)
    t = torch.arange(cu[-1], device=dev)
    seq = torch.searchsorted(edges, t, right=True) - 1
    return seq, edges[seq], edges[seq + 1], edges


def _silu(v):
    return v / (1 + torch.exp(-v))


def _silu_slope(v):
    s = 1 / (1 + torch.exp(-v))
    return s * (1 + v * (1 - s))


def _conv_rows(x, init, cu, width):
    """The input rows with every sequence's earlier rows behind them, and for each token and tap the row it reads."""
    b, seqlen, ch = x.shape
    seq, start, end, edges = _seq_index(cu, b, seqlen, x.device)
    nst, total = edges.numel() - 1, b * seqlen
    before = torch.zeros(nst * (width - 1), ch, device=x.device) if init is None else init.float().reshape(-1, ch)
    rows = torch.cat([x.float().reshape(total, ch), before])
    t = torch.arange(total, device=x.device)[:, None]
    at = t - (width - 1) + torch.arange(width, device=x.device)  # [total, width]
    at = torch.where(at >= start[:, None], at, total + seq[:, None] * (width - 1) + (width - 1) + at - start[:, None])
    j = torch.arange(width - 1, device=x.device)
    last = edges[1:, None] - (width - 1) + j  # the rows that a sequence leaves behind
    s = torch.arange(nst, device=x.device)[:, None]
    last = torch.where(last >= edges[:-1, None], last, total + s * (width - 1) + (width - 1) + last - edges[:-1, None])
    return rows, at, last


def _conv_pre(rows, at, weight, bias):
    p = sum(rows[at[:, k]] * weight[:, k] for k in range(weight.shape[1]))
    return p if bias is None else p + bias


def _plain_conv(x, weight, bias, init, cu, parts):
    rows, at, last = _conv_rows(x, init, cu, weight.shape[1])
    y = _silu(_conv_pre(rows, at, weight, bias)).to(x.dtype).reshape(x.shape)
    return [v.contiguous() for v in torch.split(y, parts, dim=-1)], rows[last].to(x.dtype)


def _plain_conv_grad(dy, x, weight, bias, init, cu, dfinal):
    b, seqlen, ch = x.shape
    width, total = weight.shape[1], b * seqlen
    rows, at, last = _conv_rows(x, init, cu, width)
    dp = torch.cat([v.float() for v in dy], dim=-1).reshape(total, ch) * _silu_slope(_conv_pre(rows, at, weight, bias))
    dweight = torch.stack([(dp * rows[at[:, k]]).sum(0) for k in range(width)], dim=1)
    drows = torch.zeros_like(rows)
    drows.index_add_(0, at.t().reshape(-1), torch.cat([dp * weight[:, k] for k in range(width)]))
    if dfinal is not None:
        drows.index_add_(0, last.reshape(-1), dfinal.float().reshape(-1, ch))
    dx = drows[:total].to(x.dtype).reshape(x.shape)
    dinit = None if init is None else drows[total:].to(init.dtype).reshape(init.shape)
    return dx, dweight, None if bias is None else dp.sum(0), dinit


def _plain_conv_step(x, weight, bias, state):
    win = torch.cat([state.float(), x.float()[:, None]], dim=1)  # [b, width, ch]
    p = (win * weight.t()).sum(1)
    state.copy_(win[:, 1:])
    return _silu(p if bias is None else p + bias).to(x.dtype)


def _softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(torch.minimum(v, torch.full_like(v, 20.0)))))


def _linear_scan(a, u):
    """h_t = a_t h_{t-1} + u_t along dim 0 in log2(length) doubling steps; a and u are used up."""
    step = 1
    while step < a.shape[0]:
        u[step:] += a[step:] * u[:-step]
        a[step:] = a[step:] * a[:-step]
        step *= 2
    return u


def _per_channel(v, ch):
    """[tokens, groups, n] to [tokens, channels, n]: the channels of a group share a row."""
    return v.float()[:, torch.arange(ch, device=v.device) * v.shape[1] // ch]


def _scan_parts(x, dt, A, B, C, dt_bias, init, cu):
    """Flat tokens: delta, decays, the states after every token."""
    b, seqlen, ch = x.shape
    total = b * seqlen
    seq, start, end, edges = _seq_index(cu, b, seqlen, x.device)
    pre = dt.float().reshape(total, ch) + dt_bias
    delta = _softplus(pre)
    xf = x.float().reshape(total, ch)
    Bf, Cf = (_per_channel(v.reshape(total, *v.shape[2:]), ch) for v in (B, C))
    a = torch.exp(delta[..., None] * A)
    u = (delta * xf)[..., None] * Bf
    first = start[:, None, None] == torch.arange(total, device=x.device)[:, None, None]
    if init is not None:
        u += torch.where(first, a * init[seq], 0.0)
    h = _linear_scan(torch.where(first, 0.0, a), u)
    return seq, start, end, edges, pre, delta, xf, Bf, Cf, a, h, first


def _final_states(h, init, edges):
    empty = (edges[1:] == edges[:-1])[:, None, None]
    last = h[(edges[1:] - 1).clamp(min=0)]
    return torch.where(empty, torch.zeros_like(last) if init is None else init, last)


def _plain_scan(x, dt, A, B, C, D, z, dt_bias, init, cu):
    seq, start, end, edges, pre, delta, xf, Bf, Cf, a, h, first = _scan_parts(x, dt, A, B, C, dt_bias, init, cu)
    y = (h * Cf).sum(-1) + D * xf
    if z is not None:
        y = y * _silu(z.float().reshape(y.shape))
    return y.to(x.dtype).reshape(x.shape), _final_states(h, init, edges)


def _plain_scan_grad(dy, x, dt, A, B, C, D, z, dt_bias, init, cu, dfinal):
    seq, start, end, edges, pre, delta, xf, Bf, Cf, a, h, first = _scan_parts(x, dt, A, B, C, dt_bias, init, cu)
    total, ch = xf.shape
    groups, n = B.shape[2], B.shape[3]
    g = dy.float().reshape(total, ch)
    dz = None
    if z is not None:
        zf = z.float().reshape(total, ch)
        dz = (g * ((h * Cf).sum(-1) + D * xf) * _silu_slope(zf)).to(z.dtype).reshape(z.shape)
        g = g * _silu(zf)
    final = (end - 1)[:, None, None] == torch.arange(total, device=x.device)[:, None, None]
    r = g[..., None] * Cf
    if dfinal is not None:
        r += torch.where(final, dfinal[seq], 0.0)
    after = torch.where(final, 0.0, torch.roll(a, -1, 0))  # the decay from t into t + 1
    dh = _linear_scan(after.flip(0), r.flip(0)).flip(0)
    per = ch // groups
    dC = (g[..., None] * h).reshape(total, groups, per, n).sum(2).to(C.dtype).reshape(C.shape)
    dB = (dh * (delta * xf)[..., None]).reshape(total, groups, per, n).sum(2).to(B.dtype).reshape(B.shape)
    before = torch.roll(h, 1, 0)
    before = torch.where(first, 0.0 if init is None else init[seq], before)
    w = dh * a * before
    du = (dh * Bf).sum(-1)
    ddelta = xf * du + (w * A).sum(-1)
    slope = 1 / (1 + torch.exp(-pre))
    ddt = ddelta * slope
    dA = (w * delta[..., None]).sum(0)
    dx = (delta * du + D * g).to(x.dtype).reshape(x.shape)
    dD = (g * xf).sum(0)
    dinit = None
    if init is not None:  # an empty sequence hands its state on as it is
        pushed = torch.where(first, a * dh, 0.0)
        dinit = pushed[edges[:-1].clamp(max=total - 1)]
        dinit = torch.where((edges[1:] == edges[:-1])[:, None, None], 0.0 if dfinal is None else dfinal, dinit)
    return dx, ddt.to(dt.dtype).reshape(dt.shape), dA, dB, dC, dD, dz, ddt.sum(0), dinit


def _plain_scan_step(x, dt, A, B, C, D, z, dt_bias, state):
    xf = x.float()
    delta = _softplus(dt.float() + dt_bias)
    ch = x.shape[1]
    h = torch.exp(delta[..., None] * A) * state + (delta * xf)[..., None] * _per_channel(B, ch)
    state.copy_(h)
    y = (h * _per_channel(C, ch)).sum(-1) + D * xf
    return (y if z is None else y * _silu(z.float())).to(x.dtype)


def _plain_norm(x, weight, z, residual, scale, group, gate, eps):
    v = x.float()
    if gate == "before":
        v = v * _silu(z.float())
    if scale is not None:
        v = v * scale
    if residual is not None:
        v = v + residual.float()
    q = v.reshape(v.shape[0], -1, group)
    out = (q * torch.rsqrt((q * q).mean(-1, keepdim=True) + eps)).reshape(v.shape) * weight
    if gate == "after":
        out = out * _silu(z.float())
    return out.to(x.dtype), None if residual is None else v.to(residual.dtype)


def _plain_norm_grad(dout, x, weight, z, scale, summed, dresidual_out, group, gate, eps):
    xf, zf = x.float(), None if z is None else z.float()
    v = xf * _silu(zf) if gate == "before" else xf
    s = (v if scale is None else v * scale) if summed is None else summed.float()
    q = s.reshape(s.shape[0], -1, group)
    rstd = torch.rsqrt((q * q).mean(-1, keepdim=True) + eps)
    hat = (q * rstd).reshape(s.shape)
    g = dout.float()
    dz = None
    if gate == "after":
        dz = g * hat * weight * _silu_slope(zf)
        g = g * _silu(zf)
    dweight = (g * hat).sum(0)
    gw = (g * weight).reshape(q.shape)
    ds = (rstd * (gw - hat.reshape(q.shape) * (gw * hat.reshape(q.shape)).mean(-1, keepdim=True))).reshape(s.shape)
    dres = None
    if summed is not None:
        ds = ds + dresidual_out.float()
        dres = ds.to(summed.dtype)
    dscale = None
    if scale is not None:
        dscale = (ds * v).sum(0)
        ds = ds * scale
    if gate == "before":
        dz = ds * xf * _silu_slope(zf)
        ds = ds * _silu(zf)
    return ds.to(x.dtype), dweight, None if dz is None else dz.to(z.dtype), dres, dscale


EPS = 1e-5


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    case, op = s["case"], s["case"]["op"]
    if own:
        import state_space_model_fwd_gb300 as ssd
        if op == "conv":
            return ssd.ssd_conv_fwd(s["x"], s["weight"], s["bias"], s["init"], cu_seqlens=s["cu"], split=s["parts"])
        if op == "conv_grad":
            return ssd.ssd_conv_bwd(s["dy"], s["x"], s["weight"], s["bias"], s["init"], cu_seqlens=s["cu"],
                                    dfinal_state=s["dfinal"])
        if op == "conv_step":
            return ssd.ssd_conv_step(s["x"], s["weight"], s["bias"], state=s["state"]), s["state"]
        if op == "scan":
            return ssd.ssd_channel_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], s["init"],
                                            cu_seqlens=s["cu"])
        if op == "scan_grad":
            return ssd.ssd_channel_scan_bwd(s["dy"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"],
                                            s["init"], cu_seqlens=s["cu"], dfinal_state=s["dfinal"])
        if op == "scan_step":
            return ssd.ssd_channel_scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"],
                                             state=s["state"]), s["state"]
        if op == "norm":
            return ssd.ssd_block_norm_fwd(s["x"], s["weight"], z=s["z"], residual=s["residual"], scale=s["scale"],
                                          group_size=case["group"], gate_after=case["gate"] == "after", eps=EPS)
        return ssd.ssd_block_norm_bwd(s["dout"], s["x"], s["weight"], z=s["z"], scale=s["scale"],
                                      residual_out=s.get("summed"), dresidual_out=s.get("dresidual_out"),
                                      group_size=case["group"], gate_after=case["gate"] == "after", eps=EPS)
    if op == "conv":
        return _plain_conv(s["x"], s["weight"], s["bias"], s["init"], s["cu"], s["parts"])
    if op == "conv_grad":
        return _plain_conv_grad(s["dy"], s["x"], s["weight"], s["bias"], s["init"], s["cu"], s["dfinal"])
    if op == "conv_step":
        return _plain_conv_step(s["x"], s["weight"], s["bias"], s["state"]), s["state"]
    if op == "scan":
        return _plain_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], s["init"], s["cu"])
    if op == "scan_grad":
        return _plain_scan_grad(s["dy"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], s["init"],
                                s["cu"], s["dfinal"])
    if op == "scan_step":
        return _plain_scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], s["state"]), s["state"]
    if op == "norm":
        return _plain_norm(s["x"], s["weight"], s["z"], s["residual"], s["scale"], case["group"], case["gate"], EPS)
    return _plain_norm_grad(s["dout"], s["x"], s["weight"], s["z"], s["scale"], s.get("summed"), s.get("dresidual_out"),
                            case["group"], case["gate"], EPS)


# ---------------------------------------------------------------------------
# the work that a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, e = case["op"], {"bf16": 2, "f32": 4}[case["dtype"]]
    if op.startswith("norm"):
        m, d = case["rows"], case["dim"]
        r = {"none": 0, "same": e, "f32": 4}[case["residual"]]
        z = e if case["gate"] != "none" else 0
        params = 4 * d * (2 if case["scale"] else 1)
        if op == "norm":
            return {"bytes": m * d * (2 * e + z + 2 * r) + params, "flops": m * d * (6 + (6 if z else 0))}
        return {"bytes": m * d * (3 * e + 2 * z + 3 * r) + 2 * params, "flops": m * d * (14 + (12 if z else 0))}
    b, ch = case["batch"], case["channels"]
    if op.startswith("conv"):
        w = case["width"]
        params = 4 * ch * (w + (1 if case["bias"] else 0))
        if op == "conv_step":
            return {"bytes": b * ch * e * 2 * w + params, "flops": b * ch * (2 * w + 5)}
        t, nst = b * case["seqlen"], case["nseq"] or b
        st = nst * (w - 1) * ch * e
        if op == "conv":
            return {"bytes": 2 * t * ch * e + params + st * (2 if case["init"] else 1), "flops": t * ch * (2 * w + 5)}
        return {"bytes": 3 * t * ch * e + 2 * params + (3 * st if case["init"] else 0), "flops": t * ch * (6 * w + 12)}
    n, gate = case["dstate"], case["gate"]
    params = 4 * ch * (n + 2)
    if op == "scan_step":
        return {"bytes": b * ch * (e * (3 + gate) + 8 * n) + 2 * b * n * e + params, "flops": b * ch * (8 * n + 12)}
    t, nst, gn = b * case["seqlen"], case["nseq"] or b, case["groups"] * n
    st = 4 * nst * ch * n
    if op == "scan":
        return {"bytes": t * (ch * e * (3 + gate) + 2 * gn * e) + params + st * (2 if case["init"] else 1),
                "flops": t * ch * (8 * n + 12)}
    return {"bytes": t * (ch * e * (5 + 2 * gate) + 4 * gn * e) + 2 * params + (3 * st if case["init"] else 0),
            "flops": t * ch * (24 * n + 30)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one token after another
# ---------------------------------------------------------------------------
def _d(v):
    return None if v is None else v.double()


def _spans(case):
    """(sequence, batch row, first token, token after the last) of every sequence."""
    cu = _offsets(case)
    if cu is None:
        return [(i, i, 0, case["seqlen"]) for i in range(case["batch"])]
    return [(i, 0, cu[i], cu[i + 1]) for i in range(len(cu) - 1)]


def _exact_conv(case, s, grad):
    x, weight, bias, init = (_d(s[k]) for k in ("x", "weight", "bias", "init"))
    w, ch = case["width"], case["channels"]
    dy = torch.cat([_d(v) for v in s["dy"]], dim=-1) if grad else None
    y, final = torch.empty_like(x), []
    dx, dinit, dw = torch.empty_like(x), [], torch.zeros_like(weight)
    db = torch.zeros(ch, device=x.device, dtype=torch.float64)
    for q, row, lo, hi in _spans(case):
        past = x.new_zeros(w - 1, ch) if init is None else init[q]
        line = torch.cat([past, x[row, lo:hi]])
        if hi > lo:
            win = line.unfold(0, w, 1)  # [tokens, ch, w]
            p = torch.einsum("tcw,cw->tc", win, weight) + (0 if bias is None else bias)
            y[row, lo:hi] = p * torch.sigmoid(p)
        final.append(line[hi - lo:])
        if grad:
            back = torch.zeros_like(line)
            if hi > lo:
                sg = torch.sigmoid(p)
                dp = dy[row, lo:hi] * (sg + p * sg * (1 - sg))
                dw += torch.einsum("tc,tcw->cw", dp, win)
                db += dp.sum(0)
                for k in range(w):
                    back[k:k + hi - lo] += dp * weight[:, k]
            if s["dfinal"] is not None:
                back[hi - lo:] += _d(s["dfinal"])[q]
            dx[row, lo:hi] = back[w - 1:]
            dinit.append(back[:w - 1])
    if grad:
        return dx, dw, None if bias is None else db, None if init is None else torch.stack(dinit)
    return [v.contiguous() for v in torch.split(y, s["parts"], dim=-1)], torch.stack(final)


def _exact_scan(case, s, grad):
    x, dt, A, B, C, D, z, dt_bias, init = (_d(s[k]) for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "init"))
    ch, n, groups = case["channels"], case["dstate"], case["groups"]
    group = torch.arange(ch, device=x.device) // (ch // groups)
    pre = dt + dt_bias
    delta = torch.nn.functional.softplus(pre, threshold=1e3)
    gate = None if z is None else z * torch.sigmoid(z)
    y = torch.empty_like(x)
    # sequences of one length go side by side
    spans = _spans(case)
    sets = [spans] if not case["nseq"] else [[v] for v in spans]
    final = x.new_zeros(len(spans), ch, n)
    out = {k: torch.zeros_like(v) for k, v in dict(x=x, dt=dt, A=A, B=B, C=C, D=D).items()}
    dz, dinit = torch.zeros_like(x), torch.zeros_like(final)
    dbias = torch.zeros_like(D)
    for each in sets:
        q = [v[0] for v in each]
        r = [v[1] for v in each]
        lo, hi = each[0][2], each[0][3]
        h = torch.zeros_like(final[q]) if init is None else init[q]
        kept = [h]
        for t in range(lo, hi):
            h = torch.exp(delta[r, t, :, None] * A) * h + (delta[r, t] * x[r, t])[..., None] * B[r, t][:, group]
            v = (h * C[r, t][:, group]).sum(-1) + D * x[r, t]
            y[r, t] = v if gate is None else v * gate[r, t]
            if grad:
                kept.append(h)
                if gate is not None:
                    sg = torch.sigmoid(z[r, t])
                    dz[r, t] = _d(s["dy"])[r, t] * v * (sg + z[r, t] * sg * (1 - sg))
        final[q] = h
        if not grad:
            continue
        back = torch.zeros_like(h) if s["dfinal"] is None else _d(s["dfinal"])[q]
        for t in range(hi - 1, lo - 1, -1):
            g = _d(s["dy"][r, t])
            g = g if gate is None else g * gate[r, t]
            a = torch.exp(delta[r, t, :, None] * A)
            Bt, Ct = B[r, t][:, group], C[r, t][:, group]
            back = back + g[..., None] * Ct
            out["C"][r, t] = (g[..., None] * kept[t - lo + 1]).reshape(len(r), groups, -1, n).sum(2)
            out["B"][r, t] = (back * (delta[r, t] * x[r, t])[..., None]).reshape(len(r), groups, -1, n).sum(2)
            da = back * kept[t - lo] * a
            du = (back * Bt).sum(-1)
            dpre = (x[r, t] * du + (da * A).sum(-1)) * torch.sigmoid(pre[r, t])
            out["A"] += (da * delta[r, t, :, None]).sum(0)
            out["x"][r, t] = delta[r, t] * du + D * g
            out["D"] += (g * x[r, t]).sum(0)
            out["dt"][r, t] = dpre
            dbias += dpre.sum(0)
            back = back * a
        dinit[q] = back
    if not grad:
        return y, final
    return (out["x"], out["dt"], out["A"], out["B"], out["C"], out["D"], None if z is None else dz, dbias,
            None if init is None else dinit)


def _exact_norm(case, s, grad):
    x, weight, z, scale = (_d(s[k]) for k in ("x", "weight", "z", "scale"))
    leaves = [v.requires_grad_(grad) for v in (x, weight, z, scale) if v is not None]
    res = _d(s.get("residual"))
    gate = None if z is None else z * torch.sigmoid(z)
    v = x * gate if case["gate"] == "before" else x
    v = v if scale is None else v * scale
    summed = _d(s.get("summed"))
    if summed is not None:
        res = (summed - v.detach()).requires_grad_(True)  # the sum is given as it was stored
        leaves.append(res)
    v = v if res is None else v + res
    m = v.reshape(v.shape[0], -1, case["group"])
    out = (m / torch.sqrt(m.pow(2).mean(-1, keepdim=True) + EPS)).reshape(v.shape) * weight
    out = out * gate if case["gate"] == "after" else out
    if not grad:
        return out, None if res is None else v
    pairs = [(out, _d(s["dout"]))] + ([] if res is None else [(v, _d(s["dresidual_out"]))])
    got = torch.autograd.grad([p[0] for p in pairs], leaves, [p[1] for p in pairs])
    by = {id(k): g for k, g in zip(leaves, got)}
    return tuple(None if k is None else by[id(k)] for k in (x, weight, z, res, scale))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("conv", "conv_grad"):
        return _exact_conv(case, s, op == "conv_grad")
    if op in ("scan", "scan_grad"):
        if op == "scan_grad" and 3 * 8 * case["batch"] * case["seqlen"] * case["channels"] * case["dstate"] > 100 << 30:
            return None  # every state is kept in 64 bits
        if case["seqlen"] > 20000:
            return None  # one token after another would take too long
        return _exact_scan(case, s, op == "scan_grad")
    if op in ("norm", "norm_grad"):
        return _exact_norm(case, s, op == "norm_grad")
    if op == "conv_step":
        win = torch.cat([_d(s["state"]), _d(s["x"])[:, None]], dim=1)
        p = torch.einsum("bwc,cw->bc", win, _d(s["weight"])) + (0 if s["bias"] is None else _d(s["bias"]))
        return p * torch.sigmoid(p), win[:, 1:].contiguous()
    x, dt, A, D, z = (_d(s[k]) for k in ("x", "dt", "A", "D", "z"))
    delta = torch.nn.functional.softplus(dt + _d(s["dt_bias"]), threshold=1e3)
    h = torch.exp(delta[..., None] * A) * _d(s["state"]) + (delta * x)[..., None] * _d(s["B"])
    y = (h * _d(s["C"])).sum(-1) + D * x
    return (y if z is None else y * z * torch.sigmoid(z)), h
