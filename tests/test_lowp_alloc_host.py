"""The tensor calls' new memory: a private call of torch where it does what is expected, the public one otherwise."""

import sys
import types

import pytest
import torch

from qwen3_decoder_forward_gb300 import binding


def _raises(*_):
    raise TypeError("another signature")


def _wrong(size, stride, dtype):
    return torch.empty_strided(size, stride, dtype=dtype)  # on the host


@pytest.mark.parametrize("short", [None, _raises, _wrong, lambda *a: None])
def test_another_form_of_the_private_call_is_not_used(short, monkeypatch):
    guards = types.ModuleType("torch._C._dynamo.guards")
    if short is not None:
        guards._empty_strided_cuda = short
    monkeypatch.setitem(sys.modules, "torch._C._dynamo.guards", guards)
    asked = []
    monkeypatch.setattr(torch, "empty_strided", lambda *a, **k: asked.append((a, k)))
    new = binding._TensorCalls._allocation(torch)
    asked.clear()
    new((4, 8), (8, 1), torch.float32)
    assert asked == [(((4, 8), (8, 1)), dict(dtype=torch.float32, device="cuda"))]


@pytest.mark.parametrize("short", [None, _raises, lambda ts: None])
def test_another_form_of_the_private_version_count_is_not_used(short, monkeypatch):
    if short is None:
        monkeypatch.delattr(torch._C, "_increment_version", raising=False)
        monkeypatch.setattr(torch.autograd.graph, "increment_version", lambda t: setattr(t, "told", True))
    else:
        told = torch._C._increment_version
        monkeypatch.setattr(torch._C, "_increment_version", short)
        monkeypatch.setattr(torch.autograd.graph, "increment_version", lambda t: (setattr(t, "told", True), told((t,))))
    t = torch.zeros(3)
    binding._TensorCalls._version_count(torch)((t,))
    assert t.told


def test_a_change_is_counted():
    t = torch.zeros(3)
    binding._TensorCalls._version_count(torch)((t,))
    assert t._version == 1
