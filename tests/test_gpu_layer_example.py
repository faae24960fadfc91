"""The example's models: the operators together, as a program uses them."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "selective_layer.py")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("selective_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_training_learns_one_batch(ex):
    torch.manual_seed(1)
    model = ex.ChannelModel().cuda()
    ids = torch.randint(0, 128, (2, 49), device="cuda")
    losses = ex.train(model, ids, steps=25)
    assert losses[-1] < 0.5 * losses[0], losses
    assert all(p.grad is not None and bool(torch.isfinite(p.grad).all()) for p in model.parameters())


def test_tokens_continue_a_prompt(ex):
    """fp32: the logits of the whole sequence, against a prompt and then single tokens."""
    torch.manual_seed(2)
    model = ex.ChannelModel(dtype=torch.float32).cuda()
    ids = torch.randint(0, 128, (3, 40), device="cuda")
    whole, _ = model.prompt(ids)
    logits, caches = model.prompt(ids[:, :33].contiguous())
    rows = [logits[:, -1]] + [model.token(ids[:, t], caches) for t in range(33, 40)]
    got, want = torch.stack(rows, 1), whole[:, 32:]
    # two blocks of fp32 arithmetic in another order (the products' own rounding included)
    assert float((got - want).abs().max()) <= 1e-3 * float(want.abs().max())
    with torch.no_grad():
        assert torch.equal(model(ids), whole)  # the training path is the same calls


def test_block_around_the_chunked_scan(ex):
    torch.manual_seed(3)
    block = ex.HeadBlock()
    u = torch.randn(2, 140, 256, device="cuda").bfloat16()
    whole, _ = block.prompt(u)
    _, cache = block.prompt(u[:, :130].contiguous())
    tokens = torch.stack([block.token(u[:, t].contiguous(), cache) for t in range(130, 140)], 1)
    # bf16 operands in the chunked products and bf16 outputs of every operator: a few 2^-8
    assert float((tokens - whole[:, 130:]).float().norm()) <= 2e-2 * float(whole[:, 130:].float().norm())
