"""The operators around the scan from their definitions, in float64 on the
CPU, one sequence and one token after another; gradients by autograd over the
same loops.  Inputs are torch tensors of any type, taken as the values they
hold."""
import torch


def d(v):
    return None if v is None else v.detach().double().cpu()


def spans(b, L, cu):
    """(sequence, batch row, first token, token after the last)."""
    if cu is None:
        return [(i, i, 0, L) for i in range(b)]
    return [(i, 0, cu[i], cu[i + 1]) for i in range(len(cu) - 1)]


def silu(v):
    return v * torch.sigmoid(v)


def conv(x, weight, bias, init, cu=None, act=True):
    b, L, C = x.shape
    W = weight.shape[1]
    rows, finals = {}, []
    for s, r, lo, hi in spans(b, L, cu):
        past = x.new_zeros(W - 1, C) if init is None else init[s]
        line = torch.cat([past, x[r, lo:hi]])
        for t in range(lo, hi):
            p = (line[t - lo:t - lo + W] * weight.t()).sum(0)
            p = p if bias is None else p + bias
            rows[r, t] = silu(p) if act else p
        finals.append(line[hi - lo:])
    y = torch.stack([rows[r, t] for r in range(b) for t in range(L)]).reshape(b, L, C) if b * L else x.clone()
    return y, (torch.stack(finals) if finals else x.new_zeros(0, W - 1, C))


def softplus(v):
    return torch.nn.functional.softplus(v, threshold=1e3)


def scan(x, dt, A, B, C, D, z, dt_bias, init, cu=None, soft=True):
    b, L, ch = x.shape
    G, N = B.shape[2], B.shape[3]
    grp = torch.arange(ch) // (ch // G)
    delta = dt if dt_bias is None else dt + dt_bias
    delta = softplus(delta) if soft else delta
    rows, finals = {}, []
    for s, r, lo, hi in spans(b, L, cu):
        h = x.new_zeros(ch, N) if init is None else init[s]
        for t in range(lo, hi):
            h = torch.exp(delta[r, t][:, None] * A) * h + (delta[r, t] * x[r, t])[:, None] * B[r, t][grp]
            y = (h * C[r, t][grp]).sum(-1)
            y = y if D is None else y + D * x[r, t]
            rows[r, t] = y if z is None else y * silu(z[r, t])
        finals.append(h)
    y = torch.stack([rows[r, t] for r in range(b) for t in range(L)]).reshape(b, L, ch) if b * L else x.clone()
    return y, (torch.stack(finals) if finals else x.new_zeros(0, ch, N))


def norm(x, weight, z, residual, scale, group, gate_after, eps):
    v = x
    if z is not None and not gate_after:
        v = v * silu(z)
    v = v if scale is None else v * scale
    v = v if residual is None else v + residual
    q = v.reshape(v.shape[0], v.shape[1] // group, group)
    out = (q / torch.sqrt((q * q).mean(-1, keepdim=True) + eps)).reshape(v.shape) * weight
    if z is not None and gate_after:
        out = out * silu(z)
    return out, v


def gradients(outputs, douts, leaves):
    """Gradients of sum(out * dout) for the leaves (None leaves give None)."""
    pairs = [(o, g) for o, g in zip(outputs, douts) if g is not None]
    live = [v for v in leaves if v is not None]
    got = torch.autograd.grad([p[0] for p in pairs], live, [p[1] for p in pairs], allow_unused=True)
    it = iter(got)
    return [None if v is None else (lambda g, v: torch.zeros_like(v) if g is None else g)(next(it), v) for v in leaves]


def check(got, want, what, rel=1e-5, scale=None):
    """|got - want| <= rel * scale elementwise, and half an ulp of the output
    type on top.  ``scale`` defaults to max(|want|, rms): fp32 arithmetic on
    sums whose terms are of the result's size.  Non-finite places must agree."""
    if want is None:
        assert got is None, what
        return
    half_ulp = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    assert tuple(got.shape) == tuple(want.shape), (what, got.shape, want.shape)
    g, w = got.detach().double().cpu(), want.detach().double()
    fine = torch.isfinite(w)
    assert torch.equal(fine, torch.isfinite(g)), f"{what}: non-finite values in other places"
    if not w.numel() or not bool(fine.any()):
        return
    g, w0 = g[fine], w[fine]
    rms = w0.pow(2).mean().sqrt()
    s = torch.maximum(w0.abs(), rms) if scale is None else scale[fine] if isinstance(scale, torch.Tensor) else scale
    bound = rel * s + half_ulp * w0.abs() * 1.01 + 1e-37
    worst = ((g - w0).abs() / bound).max().item()
    assert worst <= 1, f"{what}: off by {worst:.3g} times its bound"
