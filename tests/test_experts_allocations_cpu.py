"""The experts' operators allocate past torch.empty, whose argument parsing takes
longer than a small kernel, unless something watches over allocations."""
import pytest
import torch
from torch.overrides import TorchFunctionMode
from torch.utils._python_dispatch import TorchDispatchMode

from mixture_experts_layer_mok_gb300 import experts, ops


class Dispatch(TorchDispatchMode):
    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        return func(*args, **(kwargs or {}))


class Function(TorchFunctionMode):
    def __torch_function__(self, func, types, args=(), kwargs=None):
        return func(*args, **(kwargs or {}))


@pytest.fixture
def way(monkeypatch):
    """Which way the last tensor came."""
    seen = []
    monkeypatch.setattr(experts, "_strided", lambda shape, stride, dtype: seen.append(("fast", tuple(shape), stride)))
    monkeypatch.setattr(ops, "_empty", lambda shape, dtype, device: seen.append(("empty", tuple(shape))))
    return seen


def test_modes_see_the_allocations(way):
    new = lambda: experts._new(torch.Size((2, 0, 3)), torch.float32, "cuda")  # noqa: E731
    new()
    for mode in (Dispatch(), Function()):
        with mode:
            new()
    with Dispatch(), Function():
        new()
    new()
    assert [w[0] for w in way] == ["fast", "empty", "empty", "empty", "fast"]
    assert way[0] == ("fast", (2, 0, 3), (3, 3, 1))


def test_deterministic_runs_fill_them(way):
    torch.use_deterministic_algorithms(True)
    try:
        experts._new((4,), torch.float32, "cuda")
    finally:
        torch.use_deterministic_algorithms(False)
    assert way == [("empty", (4,))]
