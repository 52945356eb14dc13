"""Which device is current while the differentiable products launch: that of
their tensors.  Without a GPU: the library is a stand-in that notes, at each
launch, whether the device guard was entered, and touches no memory."""

import contextlib

import pytest
import torch

import mxfp8_block_scaled_06_amd as mx
from mxfp8_block_scaled_06_amd import autograd


class Library:
    """Every entry point succeeds; workspaces take 256 bytes."""

    def __init__(self):
        self.guards, self.calls = 0, []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("workspace_bytes"):
                return 256
            self.calls.append((name, self.guards))
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    lib = Library()

    @contextlib.contextmanager
    def guard(device):
        assert device == torch.device("cpu")      # the tensors' device here
        lib.guards += 1
        yield
        lib.guards -= 1

    monkeypatch.setattr(mx, "_lib", lib)
    monkeypatch.setattr(mx, "_require", lambda t, dtype, name: None)
    monkeypatch.setattr(mx, "_stream", lambda device: 0)
    for module in (mx, autograd):
        if hasattr(module, "_on"):
            monkeypatch.setattr(module, "_on", guard)
    return lib


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("grads", [(True, True), (True, False), (False, True), (False, False)])
def test_forward_launches_on_the_tensors_device(library, fmt, grads):
    rows = lambda n, c: torch.zeros((n, c), dtype=torch.bfloat16)  # noqa: E731
    x = rows(64, 128).requires_grad_(grads[0])
    W = torch.zeros((2, 256, 128), dtype=torch.bfloat16, requires_grad=grads[1])
    offs = torch.tensor([32, 64], dtype=torch.int32)
    cache = autograd.WeightCache()
    ids = torch.zeros((64, 2), dtype=torch.int32)
    outs = [mx.mx_grouped_mm(x, W, offs, check_offsets=False, weight_format=fmt),
            mx.mx_grouped_mm(x, W, offs, check_offsets=False, cache=cache, weight_format=fmt),
            mx.mx_linear(x, W[0].detach().requires_grad_(grads[1]), weight_format=fmt),
            mx.mx_routed_experts(x, ids, W, check=False, weight_format=fmt),
            mx.mx_routed_experts(x, ids[:, 0].contiguous(), W, check=False, weight_format=fmt)]
    autograd.weight_cache().clear()
    assert [tuple(o.shape) for o in outs] == [(64, 256)] * 3 + [(64, 2, 256), (64, 256)]
    assert len(library.calls) >= 10
    assert not [name for name, guards in library.calls if guards == 0]
    assert library.guards == 0


def test_tensors_without_a_device_index_need_no_guard():
    """Refusals of CPU tensors read as before: no device is set for them."""
    with mx._on(torch.device("cpu")):
        pass
    A, W = torch.zeros((32, 128), dtype=torch.bfloat16), torch.zeros((1, 128, 128), dtype=torch.bfloat16)
    for fmt in ("mxfp8", "mxfp4"):
        with pytest.raises(ValueError, match="must be a GPU tensor"):
            mx.mx_grouped_mm(A, W, torch.tensor([32], dtype=torch.int32), weight_format=fmt)
