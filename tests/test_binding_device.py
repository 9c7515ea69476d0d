"""Calls on tensors of a device that is not the current one: the library launches on the current device, so the binding makes the
tensors' device current for the call and goes back after it (no compute here: the library's functions and the devices are stand-ins)."""
from __future__ import annotations

import ast
import contextlib
import inspect

import pytest
import torch

from gated_delta_rule_70_amd import binding


class On:
    """as much of a tensor as a call's launch asks for"""

    def __init__(self, index):
        self.device = torch.device("cuda", index)


@pytest.fixture
def devices(monkeypatch):
    seen = {"at": 0, "streams": []}

    @contextlib.contextmanager
    def device(d):
        back, seen["at"] = seen["at"], torch.device(d).index
        try:
            yield
        finally:
            seen["at"] = back

    def stream(index):
        seen["streams"].append(index)
        return 100 + index

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: seen["at"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", stream, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    return seen


@pytest.mark.parametrize("index", [0, 1, 3])
def test_the_tensors_device_is_current_during_the_call(devices, index):
    calls = []
    binding._run(On(index), lambda *a: calls.append((devices["at"], a)) or 0, 1, None, 2.5)
    assert calls == [(index, (1, None, 2.5, 100 + index))] and devices["streams"] == [index] and devices["at"] == 0


def test_an_error_leaves_the_device_as_it_was(devices, monkeypatch):
    class Lib:
        gdr_last_error = staticmethod(lambda: b"why")

    monkeypatch.setattr(binding, "lib", Lib)
    for index in (0, 2):
        with pytest.raises(binding.GdrError, match="why"):
            binding._run(On(index), lambda *a: 2)
        assert devices["at"] == 0


def test_every_launch_goes_that_way():
    """No entry point hands a stream to the library by itself."""
    tree = ast.parse(inspect.getsource(binding))
    callers = [f.name for f in ast.walk(tree) if isinstance(f, ast.FunctionDef) for c in ast.walk(f)
               if isinstance(c, ast.Call) and isinstance(c.func, ast.Name) and c.func.id == "_stream"]
    assert set(callers) == {"_run"}
