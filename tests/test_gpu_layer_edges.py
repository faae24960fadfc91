"""The operators around the scan at the edges of what they accept: broadcast
rows, non-finite values beside a sequence's end, very long sequences."""
import pytest
import torch

import state_space_model_fwd_gb300 as ssd

pytestmark = pytest.mark.gpu


# ---- block norm over broadcast rows ----------------------------------------
def norm_calls(t):
    """Forward and gradient over the operands in t, [b, L, dim] each."""
    fwd = ssd.ssd_block_norm_fwd(t["x"], t["weight"], z=t["z"], residual=t["residual"], scale=t["scale"])
    bwd = ssd.ssd_block_norm_bwd(t["dout"], t["x"], t["weight"], z=t["z"], scale=t["scale"], residual_out=t["residual"],
                                 dresidual_out=t["dresidual"])
    return fwd + bwd


@pytest.mark.parametrize("name", ["x", "z", "residual", "dout", "dresidual"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim", [64, 1001])
def test_broadcast_rows_of_the_norm(name, dtype, dim):
    b, L = 4, 8
    g = torch.Generator(device="cuda").manual_seed(dim)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)
    t = {k: rnd(b, L, dim).to(dtype) for k in ("x", "z", "residual", "dout", "dresidual")}
    t["weight"], t["scale"] = rnd(dim), rnd(dim)
    # a row a sequence, a row a token: two strides
    for wide in (rnd(b, 1, dim).to(dtype).expand(b, L, dim), rnd(1, L, dim).to(dtype).expand(b, L, dim)):
        assert 0 in wide.stride()
        with pytest.raises(ValueError, match="one stride"):
            norm_calls(dict(t, **{name: wide}))
        norm_calls(dict(t, **{name: wide.contiguous()}))
    # one row for all: read in place
    wide = rnd(dim).to(dtype).expand(b, L, dim)
    for u, v in zip(norm_calls(dict(t, **{name: wide})), norm_calls(dict(t, **{name: wide.contiguous()}))):
        assert torch.equal(u, v)
