"""Small recurrent models built from the library's operators.

ChannelModel: blocks of [norm | projection | short convolution | channel scan
with its gate | projection], the norm that opens a block adding the previous
block's output to the residual stream.  It trains (the operators' gradients
as autograd functions below) on the given tokens' log-probabilities, which in
bf16 come straight from the hidden states (of a multiple of 8 columns), reads
prompts, continues token by token and lists the alternatives of an answer.

GatedModel: the same around the gated scan.

HeadBlock: a Mamba-2-shaped block around the chunked scan ssd_fwd: the
convolution writes x, B and C as the scan takes them, the norm gates its
output; tokens run through ssd_conv_step and ssd_decode_step.

    python examples/selective_layer.py
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import state_space_model_fwd_gb300 as ssd  # noqa: E402


# ---------------------------------------------------------------------------
# the operators as autograd functions
# ---------------------------------------------------------------------------
class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        ctx.save_for_backward(x, weight, bias)
        return ssd.ssd_conv_fwd(x, weight, bias, return_final_state=False)[0]

    @staticmethod
    def backward(ctx, dy):
        dx, dweight, dbias, _ = ssd.ssd_conv_bwd(dy.contiguous(), *ctx.saved_tensors)
        return dx, dweight, dbias


class ChannelScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias):
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias)
        return ssd.ssd_channel_scan_fwd(x, dt, A, B, C, D, z, dt_bias, return_final_state=False)[0]

    @staticmethod
    def backward(ctx, dy):
        return ssd.ssd_channel_scan_bwd(dy.contiguous(), *ctx.saved_tensors)[:8]


class AddNorm(torch.autograd.Function):
    """(norm(residual + x), residual + x)"""

    @staticmethod
    def forward(ctx, x, weight, residual):
        out, summed = ssd.ssd_block_norm_fwd(x, weight, residual=residual)
        ctx.save_for_backward(x, weight, summed)
        return out, summed

    @staticmethod
    def backward(ctx, dout, dsummed):
        x, weight, summed = ctx.saved_tensors
        dx, dweight, _, dres, _ = ssd.ssd_block_norm_bwd(dout.contiguous(), x, weight, residual_out=summed,
                                                         dresidual_out=dsummed.contiguous())
        return dx, dweight, dres


class GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, r, decay, i, z):
        y, _, states = ssd.ssd_gated_scan_fwd(x, r, decay, i, z, return_final_state=False, return_chunk_states=True)
        ctx.save_for_backward(x, r, decay, i, z, states)
        return y

    @staticmethod
    def backward(ctx, dy):
        *inputs, states = ctx.saved_tensors
        return ssd.ssd_gated_scan_bwd(dy.contiguous(), *inputs, chunk_states=states)[:5]


class TokenLogprob(torch.autograd.Function):
    """log-probabilities of the targets from logits"""

    @staticmethod
    def forward(ctx, logits, targets):
        logprob, lse, _, _, _ = ssd.ssd_token_logprob_fwd(logits, targets, return_entropy=False)
        ctx.save_for_backward(logits, targets, lse)
        return logprob

    @staticmethod
    def backward(ctx, dlogprob):
        logits, targets, lse = ctx.saved_tensors
        return ssd.ssd_token_logprob_bwd(logits, targets, lse, dlogprob=dlogprob.contiguous()), None


class HeadLogprob(torch.autograd.Function):
    """the same from hidden states and the output weights, without logits"""

    @staticmethod
    def forward(ctx, hidden, weight, targets):
        logprob, lse, _ = ssd.ssd_head_logprob_fwd(hidden, weight, targets, return_entropy=False)
        ctx.save_for_backward(hidden, weight, targets, lse)
        return logprob

    @staticmethod
    def backward(ctx, dlogprob):
        hidden, weight, targets, lse = ctx.saved_tensors
        return (*ssd.ssd_head_logprob_bwd(hidden, weight, targets, lse, dlogprob=dlogprob.contiguous(),
                                          need_dhidden=ctx.needs_input_grad[0], need_dweight=ctx.needs_input_grad[1]), None)


# ---------------------------------------------------------------------------
# a model of channel-scan blocks
# ---------------------------------------------------------------------------
class ChannelBlock(torch.nn.Module):
    def __init__(self, dim, inner, dstate=16, rank=16, width=4, dtype=torch.bfloat16):
        super().__init__()
        self.inner, self.dstate, self.rank = inner, dstate, rank
        lin = lambda i, o: torch.nn.Parameter((torch.randn(o, i) / math.sqrt(i)).to(dtype))
        f32 = lambda v: torch.nn.Parameter(v.float())
        self.norm = f32(torch.ones(dim))
        self.w_in, self.w_out = lin(dim, 2 * inner), lin(inner, dim)
        self.w_x, self.w_dt = lin(inner, rank + 2 * dstate), lin(rank, inner)
        self.conv_w, self.conv_b = f32(torch.randn(inner, width) / math.sqrt(width)), f32(torch.zeros(inner))
        u = torch.exp(torch.rand(inner) * math.log(100.0) + math.log(1e-3))
        self.dt_bias = f32(u + torch.log(-torch.expm1(-u)))
        self.log_A = f32(torch.log(torch.arange(1.0, dstate + 1)).repeat(inner, 1))
        self.D = f32(torch.ones(inner))

    def parts(self, x):
        """dt, B, C of the convolved x [..., inner]."""
        p = x @ self.w_x.t()
        dt = p[..., :self.rank] @ self.w_dt.t()
        n = self.dstate
        B, C = p[..., self.rank:self.rank + n], p[..., self.rank + n:]
        return dt, B.unsqueeze(-2), C.unsqueeze(-2)  # one group; strided views are read in place

    def forward(self, x, residual):
        h, residual = AddNorm.apply(x, self.norm, residual)
        xz = h @ self.w_in.t()
        x, z = xz[..., :self.inner], xz[..., self.inner:]
        x = Conv.apply(x, self.conv_w, self.conv_b)
        dt, B, C = self.parts(x)
        y = ChannelScan.apply(x, dt, -torch.exp(self.log_A), B, C, self.D, z, self.dt_bias)
        return y @ self.w_out.t(), residual

    @torch.no_grad()
    def prompt(self, x, residual):
        """The same, and the states to continue from."""
        h, residual = ssd.ssd_block_norm_fwd(x, self.norm.data, residual=residual)
        xz = h @ self.w_in.t()
        x, z = xz[..., :self.inner], xz[..., self.inner:]
        x, conv = ssd.ssd_conv_fwd(x, self.conv_w.data, self.conv_b.data)
        dt, B, C = self.parts(x)
        y, state = ssd.ssd_channel_scan_fwd(x, dt, -torch.exp(self.log_A.data), B, C, self.D.data, z, self.dt_bias.data)
        return y @ self.w_out.t(), residual, (conv, state)

    @torch.no_grad()
    def token(self, x, residual, cache):
        conv, state = cache
        h, residual = ssd.ssd_block_norm_fwd(x, self.norm.data, residual=residual, residual_out=residual)
        xz = h @ self.w_in.t()
        x, z = xz[..., :self.inner], xz[..., self.inner:]
        x = ssd.ssd_conv_step(x, self.conv_w.data, self.conv_b.data, state=conv)
        dt, B, C = self.parts(x)
        y = ssd.ssd_channel_scan_step(x, dt, -torch.exp(self.log_A.data), B, C, self.D.data, z, self.dt_bias.data,
                                      state=state)
        return y @ self.w_out.t(), residual


class GatedBlock(torch.nn.Module):
    def __init__(self, dim, inner, width=4, dtype=torch.bfloat16):
        super().__init__()
        self.inner = inner
        lin = lambda i, o: torch.nn.Parameter((torch.randn(o, i) / math.sqrt(i)).to(dtype))
        f32 = lambda v: torch.nn.Parameter(v.float())
        self.norm = f32(torch.ones(dim))
        self.w_in, self.w_gates, self.w_out = lin(dim, 2 * inner), lin(inner, 2 * inner), lin(inner, dim)
        self.conv_w, self.conv_b = f32(torch.randn(inner, width) / math.sqrt(width)), f32(torch.zeros(inner))
        sp = -torch.log(0.9 + 0.099 * torch.rand(inner))  # a^rate between 0.9 and 0.999
        self.decay = f32(sp + torch.log(-torch.expm1(-sp)))

    def parts(self, h):
        xz = h @ self.w_in.t()
        return xz[..., :self.inner], xz[..., self.inner:]

    def gates(self, x):
        g = x @ self.w_gates.t()
        return g[..., :self.inner], g[..., self.inner:]

    def forward(self, x, residual):
        h, residual = AddNorm.apply(x, self.norm, residual)
        x, z = self.parts(h)
        x = Conv.apply(x, self.conv_w, self.conv_b)
        r, i = self.gates(x)
        return GatedScan.apply(x, r, self.decay, i, z) @ self.w_out.t(), residual

    @torch.no_grad()
    def prompt(self, x, residual):
        h, residual = ssd.ssd_block_norm_fwd(x, self.norm.data, residual=residual)
        x, z = self.parts(h)
        x, conv = ssd.ssd_conv_fwd(x, self.conv_w.data, self.conv_b.data)
        r, i = self.gates(x)
        y, state = ssd.ssd_gated_scan_fwd(x, r, self.decay.data, i, z)
        return y @ self.w_out.t(), residual, (conv, state)

    @torch.no_grad()
    def token(self, x, residual, cache):
        conv, state = cache
        h, residual = ssd.ssd_block_norm_fwd(x, self.norm.data, residual=residual, residual_out=residual)
        x, z = self.parts(h)
        x = ssd.ssd_conv_step(x, self.conv_w.data, self.conv_b.data, state=conv)
        r, i = self.gates(x)
        return ssd.ssd_gated_scan_step(x, r, self.decay.data, i, z, state=state) @ self.w_out.t(), residual


class ChannelModel(torch.nn.Module):
    block = ChannelBlock

    def __init__(self, vocab=128, dim=64, inner=128, blocks=2, dtype=torch.bfloat16):
        super().__init__()
        self.embed = torch.nn.Parameter((0.5 * torch.randn(vocab, dim)).to(dtype))
        self.blocks = torch.nn.ModuleList(self.block(dim, inner, dtype=dtype) for _ in range(blocks))
        self.norm = torch.nn.Parameter(torch.ones(dim))

    def start(self, ids):
        x = self.embed[ids]
        return x, torch.zeros(x.shape, device=x.device)  # the residual stream in fp32

    def hidden(self, ids):
        x, residual = self.start(ids)
        for block in self.blocks:
            x, residual = block(x, residual)
        return AddNorm.apply(x, self.norm, residual)[0]

    def forward(self, ids):
        return (self.hidden(ids) @ self.embed.t()).float()

    def logprobs(self, ids, targets):
        """Of targets [b, L] (negative: none, 0) after each of ids [b, L]."""
        h = self.hidden(ids)
        if h.dtype == torch.bfloat16 and h.shape[-1] % 8 == 0:  # (rows on 16-byte boundaries)
            return HeadLogprob.apply(h, self.embed, targets)
        return TokenLogprob.apply(h @ self.embed.t(), targets)

    @torch.no_grad()
    def prompt(self, ids):
        x, residual = self.start(ids)
        caches = []
        for block in self.blocks:
            x, residual, cache = block.prompt(x, residual)
            caches.append(cache)
        h, _ = ssd.ssd_block_norm_fwd(x, self.norm.data, residual=residual)
        return (h @ self.embed.t()).float(), caches

    @torch.no_grad()
    def token(self, ids, caches):
        x, residual = self.start(ids)
        for block, cache in zip(self.blocks, caches):
            x, residual = block.token(x, residual, cache)
        h, _ = ssd.ssd_block_norm_fwd(x, self.norm.data, residual=residual)
        return (h @ self.embed.t()).float()


class GatedModel(ChannelModel):
    block = GatedBlock


def train(model, ids, steps=20, lr=0.02):
    """Next-token training on one batch; the losses."""
    opt = torch.optim.Adam(model.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        loss = -model.logprobs(ids[:, :-1].contiguous(), ids[:, 1:].contiguous()).mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


def generate(model, ids, count):
    """Greedy continuation: one prompt pass, then token by token."""
    logits, caches = model.prompt(ids)
    last = logits[:, -1].argmax(-1)
    out = [last]
    for _ in range(count - 1):
        last = model.token(last, caches).argmax(-1)
        out.append(last)
    return torch.stack(out, 1)


@torch.no_grad()
def answer(model, ids, count, top=4):
    """The greedy continuation [b, count] with every token's log-probability [b, count] and the `top` most probable tokens
    in its place, [b, count, top]."""
    if count < 1:
        raise ValueError(f"count must be at least 1, got {count}")
    logits, caches = model.prompt(ids)
    logits, out = logits[:, -1], []
    while True:
        _, _, _, value, index = ssd.ssd_token_logprob_fwd(logits, top=top, return_entropy=False)
        out.append((index[:, 0], value[:, 0], index))
        if len(out) == count:
            return tuple(torch.stack(v, 1) for v in zip(*out))
        logits = model.token(index[:, 0].contiguous(), caches)


# ---------------------------------------------------------------------------
# a block around the chunked scan
# ---------------------------------------------------------------------------
class HeadBlock:
    def __init__(self, dim=256, heads=8, headdim=64, dstate=128, dtype=torch.bfloat16, device="cuda"):
        g = torch.Generator(device=device).manual_seed(0)
        rnd = lambda *s: torch.randn(*s, generator=g, device=device)
        self.H, self.P, self.N, self.I = heads, headdim, dstate, heads * headdim
        self.split = [self.I, dstate, dstate]
        C = sum(self.split)
        self.w_in = (rnd(self.I + C + heads, dim) / math.sqrt(dim)).to(dtype)
        self.w_out = (rnd(dim, self.I) / math.sqrt(self.I)).to(dtype)
        self.conv_w, self.conv_b = rnd(C, 4) / 2, 0.1 * rnd(C)
        self.A, self.D = -torch.exp(torch.rand(heads, generator=g, device=device) * 2), torch.ones(heads, device=device)
        self.dt_bias = torch.full((heads,), -4.0, device=device)
        self.norm = torch.ones(self.I, device=device)

    def cut(self, u):
        p = u @ self.w_in.t()
        z, xbc, dt = p[..., :self.I], p[..., self.I:-self.H], p[..., -self.H:]
        return z, xbc, torch.nn.functional.softplus(dt.float() + self.dt_bias).to(u.dtype)

    def prompt(self, u):
        b, L, _ = u.shape
        z, xbc, dt = self.cut(u)
        (x, B, C), conv = ssd.ssd_conv_fwd(xbc, self.conv_w, self.conv_b, split=self.split)
        y, state = ssd.ssd_fwd(x.view(b, L, self.H, self.P), dt, self.A, B.unsqueeze(2), C.unsqueeze(2), self.D,
                               y_dtype=u.dtype)
        out, _ = ssd.ssd_block_norm_fwd(y.view(b, L, self.I), self.norm, z=z)
        return out @ self.w_out.t(), (conv, state)

    def token(self, u, cache):
        conv, state = cache
        b = u.shape[0]
        z, xbc, dt = self.cut(u)
        x, B, C = torch.split(ssd.ssd_conv_step(xbc, self.conv_w, self.conv_b, state=conv), self.split, dim=-1)
        y = ssd.ssd_decode_step(x.contiguous().view(b, self.H, self.P), dt.contiguous(), self.A,
                                B.contiguous().unsqueeze(1), C.contiguous().unsqueeze(1), self.D, state=state,
                                y_dtype=u.dtype)
        out, _ = ssd.ssd_block_norm_fwd(y.view(b, self.I), self.norm, z=z)
        return out @ self.w_out.t()


def main():
    torch.manual_seed(0)
    model = ChannelModel().cuda()
    ids = torch.randint(0, 128, (4, 65), device="cuda")
    losses = train(model, ids)
    print(f"training: loss {losses[0]:.3f} -> {losses[-1]:.3f}")
    print("continuation:", generate(model, ids[:1, :16].contiguous(), 8).tolist()[0])
    gated = GatedModel().cuda()
    losses = train(gated, ids)
    print(f"gated model: loss {losses[0]:.3f} -> {losses[-1]:.3f}")
    tokens, logprobs, others = answer(gated, ids[:1, :16].contiguous(), 8)
    print("answer:", tokens.tolist()[0], [round(v, 2) for v in logprobs.tolist()[0]], "instead of the last:", others[0, -1, 1:].tolist())
    block = HeadBlock()
    u = torch.randn(2, 100, 256, device="cuda").bfloat16()
    whole, _ = block.prompt(u)
    part, cache = block.prompt(u[:, :96].contiguous())
    tokens = torch.stack([block.token(u[:, t].contiguous(), cache) for t in range(96, 100)], 1)
    off = float((tokens - whole[:, 96:]).float().norm() / whole[:, 96:].float().norm())
    print(f"chunked block: tokens after a prompt against the whole prompt, relative difference {off:.1e}")


if __name__ == "__main__":
    main()
