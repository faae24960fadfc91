"""A gated recurrence and the end of a language model, as cases to be measured.

Three operators, each with the directions that a program uses:

  gated    gated linear recurrence, one state a channel (log a = -c softplus(decay) sigmoid(r),
           h = a h + sqrt(1 - a^2) sigmoid(i) x, y = h silu(z)): prompts, training, one token
  logprob  from logits: the log-probability of a given token, the log of the sum, the entropy and the top
           alternatives of every row; training adds the gradient
  head     the same numbers (no alternatives) from hidden states and the output weights, without logits in memory;
           training adds the gradients of both

`own` False runs the formulas as elementary torch operations in fp32; `own`
True runs the calls a user makes.  Sequences are either `batch` rows of
`seqlen` tokens, or `nseq` of unequal lengths packed back to back into
`seqlen` tokens (`cut` draws the offsets).
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
RATE = 8.0


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token of 128 conversations through the recurrence of a 2560-wide layer: the state is read and written once
        dict(name="gated_token", op="gated_step", dtype="bf16", batch=128, channels=2560, igate=True, gate=True),
        # a single prompt, few channels: little to run side by side
        dict(name="gated_prompt_one", op="gated", dtype="bf16", batch=1, seqlen=2048, nseq=0, cut=0, channels=1536, row=1536,
             igate=True, gate=False, init=False),
        # a packed prefill: 48 prompts of unequal lengths that continue from cached states, read out of wider rows
        dict(name="gated_packed_large", op="gated", dtype="bf16", batch=1, seqlen=65537, nseq=48, cut=5, channels=2560,
             row=2568, igate=True, gate=True, init=True),
        # a training step's forward and gradient over a batch of long sequences
        dict(name="gated_train", op="gated_train", dtype="bf16", batch=8, seqlen=4096, nseq=0, cut=0, channels=2560, row=2560,
             igate=True, gate=True, init=False),
        # the same over packed documents in fp32, an odd number of channels
        dict(name="gated_train_packed_f32", op="gated_train", dtype="f32", batch=1, seqlen=4097, nseq=9, cut=7, channels=1001,
             row=1001, igate=True, gate=False, init=True),
        # one token of four conversations: its log-probability and eight alternatives, where only latency counts
        dict(name="logprob_token", op="logprob", dtype="bf16", rows=4, vocab=50280, top=8, given=True, masked=False),
        # scoring a batch of prompts with five alternatives a token; an odd vocabulary, so rows lie at every alignment
        dict(name="logprob_score", op="logprob", dtype="bf16", rows=2047, vocab=65537, top=5, given=True, masked=False),
        # the loss of a training step and its gradient, a part of the tokens not trained on
        dict(name="logprob_train", op="logprob_train", dtype="bf16", rows=8192, vocab=50280, entropy=False),
        # log-probabilities and entropy in fp32, both trained on (as where answers are sampled and rewarded)
        dict(name="logprob_train_f32", op="logprob_train", dtype="f32", rows=1023, vocab=32000, entropy=True),
        # scoring the tokens of 16 conversations straight from the hidden states: the weights are read once
        dict(name="head_token", op="head", dtype="bf16", rows=16, dim=2560, vocab=50280),
        # scoring a batch of prompts
        dict(name="head_score", op="head", dtype="bf16", rows=8192, dim=2560, vocab=32000),
        # the loss of a training step from hidden states, odd sizes, with the gradients of hidden states and weights
        dict(name="head_train", op="head_train", dtype="bf16", rows=4095, dim=2560, vocab=50277, entropy=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_train", "gated_train", "gated_step", "logprob", "logprob", "logprob_train",
                     "logprob_train", "head", "head", "head_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("gated"):
        channels = _log(rng, 48, 5120)
        if rng.random() < 0.6:
            channels = -(-channels // 64) * 64
        c = dict(op=op, dtype=dtype, channels=channels, igate=rng.random() < 0.8, gate=rng.random() < 0.5)
        if op == "gated_step":
            return dict(c, batch=_log(rng, 1, 512))
        most = {"gated": 65536 * 2560, "gated_train": 32768 * 1280}[op]
        tokens = max(1, min(_log(rng, 1, 65536), most // channels))
        c["nseq"], c["batch"] = (rng.randint(1, 60), 1) if rng.random() < 0.5 else (0, rng.choice([1, 1, 2, 4, 8, 33]))
        c["seqlen"] = tokens if c["nseq"] else max(1, tokens // c["batch"])
        return dict(c, cut=rng.randint(0, 999), row=channels + rng.choice([0, 0, 8, 129]), init=rng.random() < 0.5)
    vocab = _log(rng, 1000, 131072)
    if rng.random() < 0.5:
        vocab = -(-vocab // 8) * 8
    if op.startswith("logprob"):
        rows = max(1, min(_log(rng, 1, 8192), 8192 * 16384 // vocab))
        if op == "logprob":
            return dict(op=op, dtype=dtype, rows=rows, vocab=vocab, top=rng.choice([0, 1, 4, 8, 20, 64]),
                        given=rng.random() < 0.8, masked=rng.random() < 0.3)
        return dict(op=op, dtype=dtype, rows=rows, vocab=vocab, entropy=rng.random() < 0.5)
    dim = rng.choice([_log(rng, 8, 320) * 8, _log(rng, 1, 40) * 64])
    rows = max(1, min(_log(rng, 1, 8192), 4096 * 2560 * 32000 // (vocab * dim)))
    c = dict(op=op, dtype="bf16", rows=rows, dim=dim, vocab=vocab)
    return dict(c, entropy=rng.random() < 0.5) if op == "head_train" else c


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
    g.manual_seed(seed * 7919 + 29)
    dtype, op, f32 = TYPES[case["dtype"]], case["op"], torch.float32

    def normal(*shape, std=1.0, mean=0.0, dtype=dtype):
        return (torch.randn(*shape, generator=g, device=DEV) * std + mean).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    s = dict(case=case)
    if op.startswith("gated"):
        b, ch = case["batch"], case["channels"]
        tok = (b,) if op == "gated_step" else (b, case["seqlen"])
        row = case.get("row", ch)
        at = (row - ch) // 16 * 8  # the columns sit inside a wider row
        s["x"], s["r"] = (normal(*tok, row)[..., at:at + ch] for _ in range(2))
        s["i"] = normal(*tok, row)[..., at:at + ch] if case["igate"] else None
        s["z"] = normal(*tok, row)[..., at:at + ch] if case["gate"] else None
        # a^c between 0.9 and 0.999 where the gate is open: softplus(decay) = -log(a^c)
        sp = -torch.log(0.9 + 0.099 * uniform(ch))
        s["decay"] = sp + torch.log(-torch.expm1(-sp))
        if op == "gated_step":
            s["state"] = normal(b, ch, std=0.5, dtype=f32)
            return s
        s["cu"] = _offsets(case)
        nst = case["nseq"] or b
        s["init"] = normal(nst, ch, std=0.5, dtype=f32) if case["init"] else None
        if op == "gated_train":
            s["dy"] = normal(*tok, ch)
            s["dfinal"] = normal(nst, ch, std=0.3, dtype=f32) if case["init"] else None
        return s
    rows, vocab = case["rows"], case["vocab"]
    s["targets"] = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    if op.endswith("train"):
        trained = uniform(rows) < 0.85
        s["targets"] = torch.where(trained, s["targets"], torch.full_like(s["targets"], -100))
        s["dlogprob"] = -(0.5 + uniform(rows)) / rows
        s["dlse"] = 1e-3 * uniform(rows) / rows
        s["dentropy"] = -0.01 * (0.5 + uniform(rows)) / rows if case["entropy"] else None
    if op.startswith("head"):
        s["hidden"] = normal(rows, case["dim"])
        s["weight"] = normal(vocab, case["dim"], std=2.0 / math.sqrt(case["dim"]))
        return s
    s["logits"] = normal(rows, vocab, std=3.0)
    if op == "logprob":
        if not case["given"]:
            s["targets"] = None
        if case["masked"]:  # tokens that an answer's grammar rules out; in one row all of them
            s["logits"][uniform(rows, vocab) < 0.5] = -math.inf
            s["logits"][rows // 2] = -math.inf
    return s


# ---------------------------------------------------------------------------
# the plain forms: elementary operations in fp32
# ---------------------------------------------------------------------------
def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _edges(cu, b, seqlen, dev):
    """For every flat token whether it is its sequence's first, its sequence, and the offsets."""
    edges = torch.tensor([seqlen * i for i in range(b + 1)] if cu is None else cu, device=dev)
    t = torch.arange(b * seqlen, device=dev)
    seq = torch.searchsorted(edges, t, right=True) - 1
    return edges[seq] == t, seq, edges


def _linear_scan(a, u):
    """h_t = a_t h_{t-1} + u_t along dim 0 in log2(length) doubling steps; a and u are used up."""
    step = 1
    while step < a.shape[0]:
        u[step:] += a[step:] * u[:-step]
        a[step:] = a[step:] * a[:-step]
        step *= 2
    return u


def _gates(x, r, i, decay):
    """log a, a, sqrt(1 - a^2), the gates and what enters the state."""
    sr = _sigmoid(r.float())
    la = -RATE * torch.log1p(torch.exp(decay)) * sr
    beta = torch.sqrt(-torch.expm1(2 * la))
    si = torch.ones_like(sr) if i is None else _sigmoid(i.float())
    return sr, la, torch.exp(la), beta, si, beta * si * x.float()


def _plain_gated(x, r, i, decay, z, init, cu, dy=None, dfinal=None, grad=False):
    b, seqlen, ch = x.shape
    total = b * seqlen
    flat = lambda v: None if v is None else v.reshape(total, ch)
    xf, rf, jf, zf = (flat(v) for v in (x, r, i, z))
    sr, la, a, beta, si, u = _gates(xf, rf, jf, decay)
    first, seq, edges = _edges(cu, b, seqlen, x.device)
    first = first[:, None]
    before = torch.zeros(edges.numel() - 1, ch, device=x.device) if init is None else init
    start = torch.where(first, before[seq], 0.0)
    h = _linear_scan(torch.where(first, 0.0, a), u + a * start)
    gate = None if z is None else zf.float() * _sigmoid(zf.float())
    y = (h if z is None else h * gate).to(x.dtype).reshape(x.shape)
    empty = (edges[1:] == edges[:-1])[:, None]
    last = (edges[1:] - 1).clamp(min=0)
    final = torch.where(empty, before, h[last])
    if not grad:
        return y, final
    gy = dy.reshape(total, ch).float()
    dz = None
    if z is not None:
        s = _sigmoid(zf.float())
        dz = (gy * h * s * (1 + zf.float() * (1 - s))).to(x.dtype).reshape(x.shape)
        gy = gy * gate
    else:
        gy = gy.clone()
    if dfinal is not None:
        gy.index_add_(0, last, torch.where(empty, 0.0, dfinal))
    # towards earlier tokens: what reaches token t from t + 1 goes through a of t + 1
    ends = torch.cat([first[1:], first.new_ones(1, 1)])
    back = torch.where(ends, 0.0, torch.cat([a[1:], a[:1]]))
    gh = _linear_scan(back.flip(0), gy.flip(0)).flip(0)
    prev = torch.where(first, start, torch.cat([h[:1], h[:-1]]))
    dla = gh * prev * a - torch.where(beta > 0, gh * si * xf.float() * a * a / beta, 0.0)
    dx = (gh * beta * si).to(x.dtype).reshape(x.shape)
    dr = (dla * la * (1 - sr)).to(x.dtype).reshape(x.shape)
    di = None if i is None else (gh * beta * xf.float() * si * (1 - si)).to(x.dtype).reshape(x.shape)
    ddecay = (dla * sr).sum(0) * -RATE * _sigmoid(decay)
    dinit = None
    if init is not None:
        at = edges[:-1].clamp(max=total - 1)
        dinit = torch.where(empty, torch.zeros_like(init) if dfinal is None else dfinal, (gh * a)[at])
    return y, final, dx, dr, di, ddecay, dz, dinit


def _plain_gated_step(x, r, i, decay, z, state):
    _, _, a, _, _, u = _gates(x, r, i, decay)
    state.copy_(a * state + u)
    y = state if z is None else state * z.float() * _sigmoid(z.float())
    return y.to(x.dtype)


def _row_numbers(zf, targets):
    """The log of the sum, the entropy, the given tokens' log-probabilities (0 where none is given) and the probabilities.
    A row that is masked throughout has no probabilities: minus infinity, an entropy of 0 and zeros."""
    top = zf.max(-1, keepdim=True).values
    top = torch.where(torch.isinf(top), 0.0, top)
    e = torch.exp(zf - top)
    total = e.sum(-1, keepdim=True)
    p = torch.where(total > 0, e / total, 0.0)
    lse = top + torch.log(total)
    entropy = -torch.where(p > 0, p * (zf - lse), 0.0).sum(-1)
    logprob = None
    if targets is not None:
        at = zf.gather(1, targets.clamp(min=0)[:, None])
        logprob = torch.where(torch.isinf(at), at, at - lse)[:, 0]
        logprob = torch.where(targets < 0, 0.0, logprob)
    return logprob, lse[:, 0], entropy, p


def _plain_logprob(logits, targets, top):
    zf = logits.float()
    logprob, lse, entropy, _ = _row_numbers(zf, targets)
    if not top:
        return logprob, lse, entropy, None, None
    value, index = torch.sort(zf, dim=-1, descending=True, stable=True)  # equal values: the lowest index first
    value, index = value[:, :top], index[:, :top].contiguous()
    return logprob, lse, entropy, torch.where(torch.isinf(value), value, value - lse[:, None]), index


def _plain_dlogits(zf, targets, lse, entropy, p, dlogprob, dlse, dentropy):
    glp = torch.where(targets < 0, 0.0, dlogprob)
    coef = (dlse - glp)[:, None]
    if dentropy is not None:
        coef = coef - dentropy[:, None] * (zf - lse[:, None] + entropy[:, None])
    d = p * coef
    d.scatter_add_(1, targets.clamp(min=0)[:, None], glp[:, None])
    return d


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        return _run_own(s, case, op)
    if op == "gated_step":
        return _plain_gated_step(s["x"], s["r"], s["i"], s["decay"], s["z"], s["state"]), s["state"]
    if op == "gated":
        return _plain_gated(s["x"], s["r"], s["i"], s["decay"], s["z"], s["init"], s["cu"])
    if op == "gated_train":
        return _plain_gated(s["x"], s["r"], s["i"], s["decay"], s["z"], s["init"], s["cu"], s["dy"], s["dfinal"], grad=True)
    if op == "logprob":
        return _plain_logprob(s["logits"], s["targets"], case["top"])
    if op == "logprob_train":
        zf = s["logits"].float()
        logprob, lse, entropy, p = _row_numbers(zf, s["targets"])
        d = _plain_dlogits(zf, s["targets"], lse, entropy, p, s["dlogprob"], s["dlse"], s["dentropy"])
        return logprob, lse, entropy, d.to(s["logits"].dtype)
    hf, wf = s["hidden"].float(), s["weight"].float()
    zf = hf @ wf.t()
    logprob, lse, entropy, p = _row_numbers(zf, s["targets"])
    if op == "head":
        return logprob, lse, entropy
    d = _plain_dlogits(zf, s["targets"], lse, entropy, p, s["dlogprob"], s["dlse"], s["dentropy"])
    return logprob, lse, entropy, (d @ wf).to(s["hidden"].dtype), (d.t() @ hf).to(s["weight"].dtype)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _run_own(s, case, op):
    import state_space_model_fwd_gb300 as ssd
    if op == "gated_step":
        return ssd.ssd_gated_scan_step(s["x"], s["r"], s["decay"], s["i"], s["z"], state=s["state"], rate=RATE), s["state"]
    if op == "gated":
        return ssd.ssd_gated_scan_fwd(s["x"], s["r"], s["decay"], s["i"], s["z"], s["init"], rate=RATE, cu_seqlens=s["cu"])
    if op == "gated_train":
        y, final, states = ssd.ssd_gated_scan_fwd(s["x"], s["r"], s["decay"], s["i"], s["z"], s["init"], rate=RATE,
                                                  cu_seqlens=s["cu"], return_chunk_states=True)
        dx, dr, ddecay, di, dz, dinit = ssd.ssd_gated_scan_bwd(s["dy"], s["x"], s["r"], s["decay"], s["i"], s["z"], s["init"],
                                                               rate=RATE, cu_seqlens=s["cu"], dfinal_state=s["dfinal"],
                                                               chunk_states=states)
        return y, final, dx, dr, di, ddecay, dz, dinit
    if op == "logprob":
        return ssd.ssd_token_logprob_fwd(s["logits"], s["targets"], top=case["top"])
    if op == "logprob_train":
        logprob, lse, entropy, _, _ = ssd.ssd_token_logprob_fwd(s["logits"], s["targets"])
        d = ssd.ssd_token_logprob_bwd(s["logits"], s["targets"], lse, entropy, dlogprob=s["dlogprob"], dlse=s["dlse"],
                                      dentropy=s["dentropy"])
        return logprob, lse, entropy, d
    logprob, lse, entropy = ssd.ssd_head_logprob_fwd(s["hidden"], s["weight"], s["targets"])
    if op == "head":
        return logprob, lse, entropy
    dhidden, dweight = ssd.ssd_head_logprob_bwd(s["hidden"], s["weight"], s["targets"], lse, entropy, dlogprob=s["dlogprob"],
                                                dlse=s["dlse"], dentropy=s["dentropy"])
    return logprob, lse, entropy, dhidden, dweight


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, es = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("gated"):
        ch, streams = case["channels"], 2 + case["igate"] + case["gate"]
        if op == "gated_step":
            n = case["batch"] * ch
            return {"bytes": n * (es * (streams + 1) + 8) + 4 * ch, "flops": 12 * n}
        n = case["batch"] * case["seqlen"] * ch
        states = 4 * (case["nseq"] or case["batch"]) * ch
        if op == "gated":
            return {"bytes": n * es * (streams + 1) + states * (1 + case["init"]) + 4 * ch, "flops": 12 * n}
        return {"bytes": n * es * (2 * streams + 2) + states * (1 + 3 * case["init"]) + 8 * ch, "flops": 40 * n}
    rows, vocab = case["rows"], case["vocab"]
    if op == "logprob":
        return {"bytes": rows * vocab * es + rows * (8 + 12 + 12 * case["top"]), "flops": 5 * rows * vocab}
    if op == "logprob_train":
        return {"bytes": 2 * rows * vocab * es + rows * 36, "flops": 9 * rows * vocab}
    dim = case["dim"]
    both = (rows + vocab) * dim * es
    if op == "head":
        return {"bytes": both + rows * 20, "flops": 2 * rows * vocab * dim}
    return {"bytes": 2 * both + rows * 36, "flops": 6 * rows * vocab * dim}


# ---------------------------------------------------------------------------
# the operators from their definitions in 64 bits
# ---------------------------------------------------------------------------
def _d(v):
    return None if v is None else v.double()


def _exact_gated(case, s, grad):
    """Token after token; the gradient of everything elementwise by differentiation, that of the recurrence by its adjoint."""
    x, r, i, z, decay = (_d(s[k]) for k in ("x", "r", "i", "z", "decay"))
    b, seqlen, ch = x.shape
    leaves = dict(x=x, r=r, i=i, decay=decay)
    leaves = {k: v.detach().requires_grad_(grad) for k, v in leaves.items() if v is not None}
    with torch.set_grad_enabled(grad):
        log_a = -RATE * torch.nn.functional.softplus(leaves["decay"], threshold=1e3) * torch.sigmoid(leaves["r"])
        a = torch.exp(log_a)
        u = torch.sqrt(-torch.expm1(2 * log_a)) * leaves["x"]
        if i is not None:
            u = u * torch.sigmoid(leaves["i"])
    av, uv = a.detach(), u.detach()
    spans = [(k, 0, seqlen) for k in range(b)] if s["cu"] is None else [(0, p, q) for p, q in zip(s["cu"], s["cu"][1:])]
    together = s["cu"] is None  # rows of one length go side by side
    sets = [list(range(b))] if together else [[k] for k in range(len(spans))]
    init = _d(s["init"]) if s["init"] is not None else x.new_zeros(len(spans), ch)
    h, prev, final = torch.empty_like(x), torch.empty_like(x), init.clone()
    for which in sets:
        lo, hi = spans[which[0]][1:]
        part = slice(None) if together else slice(0, 1)
        v = init[which]
        for t in range(lo, hi):
            prev[part, t] = v
            v = torch.addcmul(uv[part, t], av[part, t], v)
            h[part, t] = v
        final[which] = v
    gate = None if z is None else z * torch.sigmoid(z)
    y = h if z is None else h * gate
    if not grad:
        return y, final
    dy = _d(s["dy"])
    dz = None
    if z is not None:
        sz = torch.sigmoid(z)
        dz = dy * h * (sz + z * sz * (1 - sz))
        dy = dy * gate
    gh, dinit = torch.empty_like(x), torch.zeros_like(init)
    for which in sets:
        lo, hi = spans[which[0]][1:]
        part = slice(None) if together else slice(0, 1)
        v = torch.zeros_like(init[which]) if s["dfinal"] is None else _d(s["dfinal"])[which]
        for t in range(hi - 1, lo - 1, -1):
            v = v + dy[part, t]
            gh[part, t] = v
            v = v * av[part, t]
        dinit[which] = v
    got = torch.autograd.grad([a, u], list(leaves.values()), [gh * prev, gh])
    by = dict(zip(leaves, got))
    return y, final, by["x"], by["r"], by.get("i"), by["decay"], dz, None if s["init"] is None else dinit


def _exact_rows(z, targets, top):
    """Log-probabilities by logsumexp; a row with nothing left in it has none."""
    lse = torch.logsumexp(z, -1)
    alone = lse == -math.inf
    lp = torch.where(alone[:, None], -math.inf, z - torch.where(alone, 0.0, lse)[:, None])
    p = torch.exp(lp)
    entropy = torch.special.entr(p).sum(-1)
    logprob = None
    if targets is not None:
        logprob = torch.where(targets < 0, 0.0, lp[torch.arange(len(lp), device=lp.device), targets.clamp(min=0)])
    if not top:
        return lp, p, (logprob, lse, entropy, None, None)
    order = torch.argsort(lp, dim=-1, descending=True, stable=True)[:, :top].contiguous()
    return lp, p, (logprob, lse, entropy, lp.gather(1, order), order)


def _exact_dlogits(s, lp, p, entropy):
    """By the chain rule over dlogprob/dz = [v = target] - p, dlse/dz = p and dentropy/dz = -p (log p + entropy)."""
    d = p * s["dlse"].double()[:, None]
    rows = torch.nonzero(s["targets"] >= 0)[:, 0]
    g = s["dlogprob"].double()[rows]
    d[rows] -= g[:, None] * p[rows]
    d[rows, s["targets"][rows]] += g
    if s["dentropy"] is not None:
        d -= s["dentropy"].double()[:, None] * p * (lp + entropy[:, None])
    return d


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("gated", "gated_train"):
        return _exact_gated(case, s, op == "gated_train")
    if op == "gated_step":
        x, r, i, z, state = (_d(s[k]) for k in ("x", "r", "i", "z", "state"))
        log_a = -RATE * torch.nn.functional.softplus(_d(s["decay"]), threshold=1e3) * torch.sigmoid(r)
        h = torch.exp(log_a) * state + torch.sqrt(-torch.expm1(2 * log_a)) * x * (1 if i is None else torch.sigmoid(i))
        return (h if z is None else h * z * torch.sigmoid(z)), h
    if op == "logprob":
        return _exact_rows(s["logits"].double(), s["targets"], case["top"])[2]
    if op == "logprob_train":
        lp, p, (logprob, lse, entropy, _, _) = _exact_rows(s["logits"].double(), s["targets"], 0)
        return logprob, lse, entropy, _exact_dlogits(s, lp, p, entropy)
    h, w = s["hidden"].double(), s["weight"].double()
    lp, p, (logprob, lse, entropy, _, _) = _exact_rows(h @ w.t(), s["targets"], 0)
    if op == "head":
        return logprob, lse, entropy
    d = _exact_dlogits(s, lp, p, entropy)
    return logprob, lse, entropy, d @ w, d.t() @ h
