"""Host side of the gated scan and of the log-probabilities: what the binding
makes of devices, strides and workspaces.  No call here reaches a kernel."""
import importlib.util
import os

import pytest
import torch

import state_space_model_fwd_gb300 as ssd
from state_space_model_fwd_gb300 import _build, _layer
from tests.test_layer_binding import on_cuda1 as t


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return ssd.load_library()


ENTRIES = {
    "ssd_gated_scan_fwd": lambda: ssd.ssd_gated_scan_fwd(t(1, 8, 16), t(1, 8, 16), t(16)),
    "ssd_gated_scan_bwd": lambda: ssd.ssd_gated_scan_bwd(t(1, 8, 16), t(1, 8, 16), t(1, 8, 16), t(16)),
    "ssd_gated_scan_step": lambda: ssd.ssd_gated_scan_step(t(1, 16), t(1, 16), t(16), state=t(1, 16)),
    "ssd_token_logprob_fwd": lambda: ssd.ssd_token_logprob_fwd(t(4, 64)),
    "ssd_token_logprob_bwd": lambda: ssd.ssd_token_logprob_bwd(t(4, 64), None, t(4)),
    "ssd_head_logprob_fwd": lambda: ssd.ssd_head_logprob_fwd(t(4, 64), t(100, 64)),
    "ssd_head_logprob_bwd": lambda: ssd.ssd_head_logprob_bwd(t(4, 64), t(100, 64), None, t(4)),
}


@pytest.mark.parametrize("entry", ENTRIES)
def test_operands_on_another_than_the_current_device_are_refused(entry, monkeypatch):
    monkeypatch.setattr(_layer, "_current_device", lambda: 0, raising=False)
    with pytest.raises(ValueError, match="cuda:1, the current device is cuda:0"):
        ENTRIES[entry]()


@pytest.mark.parametrize("entry", ENTRIES)
def test_cpu_tensors_are_refused(entry, monkeypatch):
    monkeypatch.setattr("tests.test_model_binding.t", torch.zeros)
    with pytest.raises(TypeError, match="CUDA tensor"):
        ENTRIES[entry]()


def test_entry_points_are_exported_and_documented():
    for name in ENTRIES:
        assert name in ssd.__all__ and name in ssd.EXPORTED
        assert "Returns" in getattr(ssd, name).__doc__


def test_an_answer_of_no_tokens_is_refused():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "selective_layer.py")
    spec = importlib.util.spec_from_file_location("selective_layer_answers", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)

    class Model:  # gives up where a program would go on for ever
        def prompt(self, ids):
            raise AssertionError("asked for a prompt")
    for count in (0, -1):
        with pytest.raises(ValueError, match="count"):
            ex.answer(Model(), torch.zeros(1, 4, dtype=torch.int64), count)
