"""Workspace sizes are remembered per GPU, also where the caller names none."""
import pytest
import torch


class _Sizes:
    """A library whose sizes depend on the current GPU, and that counts its calls."""

    def __init__(self):
        self.current, self.calls = 0, 0

    def bitlinear_adapter_workspace_bytes(self, T, r):
        self.calls += 1
        return (1000, 2000)[self.current] + T * r


@pytest.fixture()
def two_gpus(monkeypatch):
    import bit_ternary_weight_b200 as bl
    lib = _Sizes()

    class On:
        def __init__(self, device):
            self.index, self.before = device.index, lib.current

        def __enter__(self):
            lib.current = self.index

        def __exit__(self, *exc):
            lib.current = self.before

    cached = next(f for f in vars(bl).values() if hasattr(f, "cache_clear") and f.__name__.startswith("_scratch"))
    cached.cache_clear()
    monkeypatch.setattr(bl, "_lib", lib)
    monkeypatch.setattr(bl, "_elsewhere", lambda d: d.type == "cuda" and d.index not in (None, lib.current))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: lib.current)
    monkeypatch.setattr(torch.cuda, "device", On)
    yield bl, lib
    cached.cache_clear()


def test_a_device_without_an_index_is_the_current_one(two_gpus):
    bl, lib = two_gpus
    name, anywhere = "bitlinear_adapter_workspace_bytes", torch.device("cuda")
    assert bl._scratch_bytes(name, anywhere, 4, 8) == 1032
    lib.current = 1
    assert bl._scratch_bytes(name, anywhere, 4, 8) == 2032
    assert bl._scratch_bytes(name, torch.device("cuda", 0), 4, 8) == 1032
    assert lib.current == 1
    calls = lib.calls
    assert [bl._scratch_bytes(name, d, 4, 8) for d in (anywhere, torch.device("cuda", 1))] == [2032, 2032]
    assert lib.calls == calls               # remembered
