"""Host side of the operators around the scan: what the binding makes of
strides, devices, workspaces and arguments.  No call here reaches a kernel."""
import pytest
import torch

from state_space_model_fwd_gb300 import _layer


# ---- rows of the block norm: every leading dimension at one stride ---------
def norm_rows(t):
    return _layer._norm_rows(t, "x", t.dtype, t.shape, t.get_device())


@pytest.mark.parametrize("t,rs", [
    (torch.zeros(5, 64), 64),
    (torch.zeros(4, 8, 64), 64),
    (torch.zeros(4, 8, 96)[:, :, 16:80], 96),                  # columns of wider rows
    (torch.zeros(4, 8, 64)[:, ::2], 128),                      # every other row: 4 x 2 rows of 64 lie 128 apart
    (torch.zeros(2, 3, 4, 8), 8),
    (torch.zeros(8, 64).as_strided((4, 1, 64), (64, 7, 1)), 64),    # a dimension of one row has no stride
    (torch.zeros(1, 1, 64), 0),
    (torch.zeros(64).expand(4, 8, 64), 0),                     # one row for all
    (torch.zeros(64).expand(32, 64), 0),
    (torch.zeros(3, 0, 64), 64),
    (torch.zeros(0, 5, 64), 64),
])
def test_norm_rows_at_one_stride(t, rs):
    r = norm_rows(t)
    assert r.row_stride == rs
    rows = t.numel() // t.shape[-1]
    if rows:  # the last row that the kernel reads lies in the tensor's memory
        end = t.storage_offset() + (rows - 1) * rs + t.shape[-1]
        assert end <= t.untyped_storage().nbytes() // t.element_size()


@pytest.mark.parametrize("t", [
    torch.zeros(4, 1, 64).expand(4, 8, 64),      # one row a sequence: strides (64, 0, 1)
    torch.zeros(1, 8, 64).expand(4, 8, 64),      # the same rows in every sequence: (0, 64, 1)
    torch.zeros(2, 1, 1, 64).expand(2, 3, 4, 64),
    torch.zeros(2, 3, 1, 64).expand(2, 3, 4, 64),
    torch.zeros(4, 8, 64)[:, :7],
    torch.zeros(8, 4, 64).transpose(0, 1),
], ids=lambda t: str(tuple(t.stride())))
def test_norm_rows_at_two_strides_are_refused(t):
    with pytest.raises(ValueError, match="one stride"):
        norm_rows(t)


def test_a_sums_gradient_is_such_a_tensor():
    """The gradient that autograd hands to what is summed over tokens."""
    out = torch.zeros(4, 8, 64, requires_grad=True)
    dout, = torch.autograd.grad(out.sum(1), out, torch.zeros(4, 64))
    assert dout.stride() == (64, 0, 1)
    with pytest.raises(ValueError, match="one stride"):
        norm_rows(dout)
