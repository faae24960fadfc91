"""Host side of the operators around the scan: what the binding makes of
strides, devices, workspaces and arguments.  No call here reaches a kernel."""
import ctypes
import os
import re

import pytest
import torch

import state_space_model_fwd_gb300 as ssd
from state_space_model_fwd_gb300 import _build, _layer


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return ssd.load_library()


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


# ---- devices ---------------------------------------------------------------
class OnCuda1(torch.Tensor):
    """A tensor that says it is on the second GPU."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 1))

    def get_device(self):
        return 1


def on_cuda1(*shape):
    return torch.zeros(*shape).as_subclass(OnCuda1)


t = on_cuda1
ENTRIES = {
    "ssd_conv_fwd": lambda: ssd.ssd_conv_fwd(t(1, 8, 16), t(16, 4)),
    "ssd_conv_bwd": lambda: ssd.ssd_conv_bwd(t(1, 8, 16), t(1, 8, 16), t(16, 4)),
    "ssd_conv_step": lambda: ssd.ssd_conv_step(t(1, 16), t(16, 4), state=t(1, 3, 16)),
    "ssd_channel_scan_fwd": lambda: ssd.ssd_channel_scan_fwd(t(1, 8, 32), t(1, 8, 32), t(32, 16), t(1, 8, 1, 16),
                                                             t(1, 8, 1, 16)),
    "ssd_channel_scan_bwd": lambda: ssd.ssd_channel_scan_bwd(t(1, 8, 32), t(1, 8, 32), t(1, 8, 32), t(32, 16),
                                                             t(1, 8, 1, 16), t(1, 8, 1, 16)),
    "ssd_channel_scan_step": lambda: ssd.ssd_channel_scan_step(t(1, 32), t(1, 32), t(32, 16), t(1, 1, 16), t(1, 1, 16),
                                                               state=t(1, 32, 16)),
    "ssd_block_norm_fwd": lambda: ssd.ssd_block_norm_fwd(t(4, 64), t(64)),
    "ssd_block_norm_bwd": lambda: ssd.ssd_block_norm_bwd(t(4, 64), t(4, 64), t(64)),
    "ssd_fwd": lambda: ssd.ssd_fwd(t(1, 64, 2, 16), t(1, 64, 2), t(2), t(1, 64, 1, 16), t(1, 64, 1, 16)),
    "ssd_fwd_varlen": lambda: ssd.ssd_fwd_varlen(t(1, 64, 2, 16), t(1, 64, 2), t(2), t(1, 64, 1, 16), t(1, 64, 1, 16),
                                                 cu_seqlens=[0, 64]),
    "selective_scan_fwd": lambda: ssd.selective_scan_fwd(t(1, 8, 2, 16), t(1, 8, 2), t(2), t(1, 8, 1, 16), t(1, 8, 1, 16)),
    "ssd_decode_step": lambda: ssd.ssd_decode_step(t(1, 2, 16), t(1, 2), t(2), t(1, 1, 16), t(1, 1, 16),
                                                   state=t(1, 2, 16, 16)),
}


@pytest.mark.parametrize("entry", ENTRIES)
def test_operands_on_another_than_the_current_device_are_refused(entry, monkeypatch):
    monkeypatch.setattr(_layer, "_current_device", lambda: 0, raising=False)
    with pytest.raises(ValueError, match="cuda:1, the current device is cuda:0"):
        ENTRIES[entry]()


# ---- workspaces ------------------------------------------------------------
def test_a_given_workspace_is_checked():
    x = torch.zeros(1)
    ws = torch.zeros(64, dtype=torch.uint8)
    assert _layer._workspace(ws, 64, x) is ws
    assert _layer._workspace(torch.zeros(16), 64, x).dtype == torch.float32  # any type: its bytes count
    assert _layer._workspace(ws, 65, x).numel() == 65                        # too small: a new one
    with pytest.raises(ValueError, match="contiguous"):
        _layer._workspace(torch.zeros(128, dtype=torch.uint8)[::2], 64, x)
    with pytest.raises(TypeError, match="workspace"):
        _layer._workspace(ws, 64, on_cuda1(1))
    with pytest.raises(TypeError, match="workspace"):
        _layer._workspace(on_cuda1(64), 64, x)
    with pytest.raises(TypeError, match="workspace"):
        _layer._workspace(1 << 20, 64, x)


class OnCuda0(OnCuda1):
    device = property(lambda self: torch.device("cuda", 0))

    def get_device(self):
        return 0


@pytest.mark.parametrize("ws,error", [(torch.zeros(1 << 20, dtype=torch.uint8), TypeError),
                                      (torch.zeros(1 << 20, dtype=torch.uint8).as_subclass(OnCuda0)[::2], ValueError)],
                         ids=["host", "strided"])
def test_the_scans_workspace_is_checked(ws, error, monkeypatch):
    monkeypatch.setattr(_layer, "_current_device", lambda: 0)
    monkeypatch.setattr(ssd, "load_library", NoLaunch)
    z = lambda *shape: torch.zeros(*shape).as_subclass(OnCuda0)
    x, dt, A, B, y = z(1, 64, 2, 16), z(1, 64, 2), z(2), z(1, 64, 1, 16), z(1, 64, 2, 16)
    with pytest.raises(error, match="workspace"):
        ssd.ssd_fwd(x, dt, A, B, B, y=y, return_final_state=False, workspace=ws)
    with pytest.raises(error, match="workspace"):
        ssd.ssd_fwd_varlen(x, dt, A, B, B, cu_seqlens=[0, 64], y=y, return_final_states=False, workspace=ws)
    with pytest.raises(error, match="workspace"):
        ssd.ssd_chunk_scan(x, dt, B, B, z(1, 2, 1, 64), z(1, 1, 2, 16, 16), out=y, workspace=ws)


class NoLaunch:
    """Stands for the library: sizes, and no call that would launch."""
    def __getattr__(self, name):
        if name.endswith("_workspace_size"):
            return lambda *args: 1024
        raise AssertionError(f"{name} reached")


# ---- the library is rebuilt after any change of what it is made from ---------
def test_every_included_file_is_an_input_of_the_build():
    inputs = {os.path.realpath(f) for f in _build._inputs()}
    seen, todo = set(), [f for f in inputs if f.endswith(".cu")]
    assert todo
    while todo:
        path = todo.pop()
        if path in seen:
            continue
        seen.add(path)
        for name in re.findall(r'^\s*#\s*include\s+"([^"]+)"', open(path, encoding="utf-8").read(), re.M):
            found = [os.path.realpath(os.path.join(d, name)) for d in (_build.CSRC, _build.INCLUDE)
                     if os.path.exists(os.path.join(d, name))]
            assert found, (path, name)
            todo.append(found[0])
    assert seen <= inputs, seen - inputs


def test_a_newer_header_makes_the_library_stale(monkeypatch):
    assert _build.up_to_date()
    newest = os.path.getmtime(_build.LIB) + 10
    true = os.path.getmtime
    header = os.path.join(_build.CSRC, "ssd_channel.h")
    monkeypatch.setattr(os.path, "getmtime", lambda f: newest if os.path.realpath(f) == header else true(f))
    assert not _build.up_to_date()


# ---- groups of the block norm ----------------------------------------------
@pytest.mark.parametrize("group", [0, -64, 48])
def test_a_group_size_that_does_not_divide_the_columns_is_refused(group, monkeypatch):
    x = torch.zeros(4, 64).as_subclass(OnCuda0)
    monkeypatch.setattr(_layer, "_current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0)
    with pytest.raises(ssd.SSDError, match="INVALID"):
        ssd.ssd_block_norm_fwd(x, torch.ones(64).as_subclass(OnCuda0), out=x, group_size=group)


def test_without_a_group_size_all_columns_are_one_group(monkeypatch):
    monkeypatch.setattr(_layer, "_current_device", lambda: 0)
    shape, _ = _layer._norm_shape(torch.zeros(4, 64).as_subclass(OnCuda0), None, 1e-5, None, False)
    assert shape.group_size == 64


# ---- gradients of absent operands ------------------------------------------
FAKE = 1 << 20  # never read


@pytest.mark.parametrize("given", ["dz", "dresidual", "dscale"])
def test_the_norms_gradient_of_an_absent_operand_is_refused(lib, given):
    """Workspace too small on purpose: what passes the checks ends there."""
    shape, r = _layer._norm_shape_t(4, 64, 64, 1e-5, 1, 1, 0), _layer._rows_t(FAKE, 0, 64)
    ref = ctypes.byref(r)
    call = lambda **kw: lib.ssd_block_norm_bwd(
        ctypes.byref(shape), ref, ref, FAKE, kw.get("z"), kw.get("scale"), kw.get("residual_out"), None, ref, FAKE,
        kw.get("dz"), kw.get("dresidual"), kw.get("dscale"), None, 0, None)
    operand = {"dz": "z", "dresidual": "residual_out", "dscale": "scale"}[given]
    value = FAKE if given == "dscale" else ref
    INVALID, WORKSPACE = 1, 4
    assert call() == WORKSPACE
    assert call(**{operand: value, given: value}) == WORKSPACE
    assert call(**{given: value}) == INVALID
