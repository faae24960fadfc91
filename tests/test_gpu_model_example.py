"""The recurrent models of the example, from prompts to losses and answers: the
operators together, as a program uses them."""
import importlib.util
import math
import os

import pytest
import torch

import state_space_model_fwd_gb300 as ssd
from tests import layer_reference as ref
from tests.test_gpu_gated_scan import definition as gated_scan

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "selective_layer.py")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("selective_layer_models", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_logprobs(model, params, ids, targets):
    """The gated model from its formulas, in float64 on the CPU."""
    p = lambda name: params[name]
    x = p("embed")[ids]
    residual = torch.zeros_like(x)
    b, L, dim = x.shape
    norm = lambda x, w, res: [v.reshape(b, L, dim) for v in ref.norm(x.reshape(b * L, dim), w, None, res.reshape(b * L, dim), None,
                                                                      dim, False, 1e-5)]
    for k, block in enumerate(model.blocks):
        q = lambda name: p(f"blocks.{k}.{name}")
        h, residual = norm(x, q("norm"), residual)
        xz = h @ q("w_in").t()
        u, z = xz[..., :block.inner], xz[..., block.inner:]
        u, _ = ref.conv(u, q("conv_w"), q("conv_b"), None)
        g = u @ q("w_gates").t()
        y, _ = gated_scan(u, g[..., :block.inner], q("decay"), g[..., block.inner:], z, None)
        x = y @ q("w_out").t()
    h, _ = norm(x, p("norm"), residual)
    lp = torch.log_softmax(h @ p("embed").t(), -1)
    return torch.where(targets < 0, 0.0, lp.gather(-1, targets.clamp(min=0)[..., None])[..., 0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_loss_and_gradients(ex, dtype):
    torch.manual_seed(4)
    model = ex.GatedModel(vocab=96, dim=32, inner=64, dtype=dtype).cuda()
    ids = torch.randint(0, 96, (2, 20), device="cuda")
    targets = torch.randint(0, 96, (2, 20), device="cuda")
    targets[0, :7] = -100
    params = {k: v.detach().double().cpu().requires_grad_(True) for k, v in model.named_parameters()}
    want = plain_logprobs(model, params, ids.cpu(), targets.cpu())
    want.sum().backward()
    got = model.logprobs(ids, targets)
    got.sum().backward()
    # fp32: two blocks' products in fp32; bf16: every operator's output is rounded, 2^-8 each at most, a dozen in a row
    tol = 1e-4 if dtype == torch.float32 else 12 * 2.0 ** -8
    assert float((got.detach().double().cpu() - want.detach()).norm()) <= tol * float(want.detach().norm())
    for k, v in model.named_parameters():
        w = params[k].grad
        off = float((v.grad.double().cpu() - w).norm())
        assert off <= 3 * tol * float(w.norm()), (k, off / float(w.norm()))


@pytest.mark.parametrize("kind", ["ChannelModel", "GatedModel"])
def test_bf16_models_of_any_width(ex, kind):
    """Rows off 16-byte boundaries: through stored logits."""
    torch.manual_seed(9)
    model = getattr(ex, kind)(vocab=97, dim=36, inner=64).cuda()
    ids = torch.randint(0, 97, (2, 20), device="cuda")
    targets = torch.randint(0, 97, (2, 20), device="cuda")
    targets[1, 3:9] = -100
    got = model.logprobs(ids, targets)
    got.sum().backward()
    with torch.no_grad():
        lp = torch.log_softmax(model(ids).double(), -1).gather(-1, targets.clamp(min=0)[..., None])[..., 0]
    # of the same logits: fp32 sums of 97 terms
    assert torch.allclose(got.detach().double(), torch.where(targets < 0, 0.0, lp), rtol=1e-5, atol=1e-5)
    assert all(bool(torch.isfinite(p.grad).all()) and float(p.grad.abs().max()) > 0 for p in model.parameters())
    assert all(math.isfinite(v) for v in ex.train(model, ids, steps=2))


def test_only_the_gradients_that_are_asked_for(ex, monkeypatch):
    torch.manual_seed(10)
    model = ex.GatedModel(vocab=96, dim=32, inner=64).cuda()
    ids = torch.randint(0, 96, (2, 20), device="cuda")
    h = model.hidden(ids).detach()
    asked, real = [], ssd.ssd_head_logprob_bwd
    monkeypatch.setattr(ssd, "ssd_head_logprob_bwd", lambda *a, **kw: asked.append((kw["need_dhidden"], kw["need_dweight"])) or real(*a, **kw))
    w = model.embed.detach()
    both = [v.clone().requires_grad_(True) for v in (h, w)]
    ex.HeadLogprob.apply(*both, ids).sum().backward()
    for k in range(2):
        one = [v.clone().requires_grad_(i == k) for i, v in enumerate((h, w))]
        ex.HeadLogprob.apply(*one, ids).sum().backward()
        assert torch.equal(one[k].grad, both[k].grad) and one[1 - k].grad is None
    assert asked == [(True, True), (True, False), (False, True)]


def test_training_runs(ex):
    torch.manual_seed(5)
    model = ex.GatedModel().cuda()
    before = [p.detach().clone() for p in model.parameters()]
    losses = ex.train(model, torch.randint(0, 128, (2, 49), device="cuda"), steps=3)
    assert all(math.isfinite(v) for v in losses)
    assert all(p.grad is not None and bool(torch.isfinite(p.grad).all()) for p in model.parameters())
    assert any(not torch.equal(a, b) for a, b in zip(before, model.parameters()))


def test_tokens_continue_a_prompt(ex):
    torch.manual_seed(6)
    model = ex.GatedModel(dtype=torch.float32).cuda()
    ids = torch.randint(0, 128, (3, 40), device="cuda")
    whole, _ = model.prompt(ids)
    logits, caches = model.prompt(ids[:, :33].contiguous())
    rows = [logits[:, -1]] + [model.token(ids[:, t], caches) for t in range(33, 40)]
    got, want = torch.stack(rows, 1), whole[:, 32:]
    # two blocks of fp32 arithmetic in another order (the products' own rounding included)
    assert float((got - want).abs().max()) <= 1e-3 * float(want.abs().max())
    with torch.no_grad():
        assert torch.equal(model(ids), whole)  # the training path is the same calls


@pytest.mark.parametrize("kind", ["ChannelModel", "GatedModel"])
def test_answers_are_what_scoring_gives(ex, kind):
    """A greedy answer's log-probabilities, against scoring it as given tokens."""
    torch.manual_seed(7)
    model = getattr(ex, kind)(dtype=torch.float32).cuda()
    ids = torch.randint(0, 128, (2, 17), device="cuda")
    tokens, logprobs, others = ex.answer(model, ids, 6)
    assert torch.equal(tokens, others[..., 0]) and torch.equal(tokens, ex.generate(model, ids, 6))
    text = torch.cat([ids, tokens], 1)
    with torch.no_grad():
        scored = model.logprobs(text[:, :-1].contiguous(), text[:, 1:].contiguous())[:, -6:]
    assert float((scored - logprobs).abs().max()) <= 1e-3 * float(logprobs.abs().max() + 1)


def test_a_training_step_in_a_graph(ex):
    """Forward and gradient of a model captured on a stream of its own and replayed with other tokens."""
    torch.manual_seed(8)
    model = ex.GatedModel().cuda()
    ids = torch.randint(0, 128, (2, 70), device="cuda")
    targets = torch.randint(0, 128, (2, 70), device="cuda")
    params = list(model.parameters())

    def step():
        loss = -model.logprobs(ids, targets).mean()
        return (loss, *torch.autograd.grad(loss, params))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # (libraries prepare their workspaces)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    ids.copy_(torch.randint(0, 128, (2, 70)))
    graph.replay()
    for a, b in zip(out, step()):
        # the embedding's gradient is summed with atomics by the framework that holds it
        a, b = a.detach().float(), b.detach().float()
        assert torch.allclose(a, b, rtol=2e-2, atol=1e-3 * float(b.abs().max()))
    ssd.check_device_status()
