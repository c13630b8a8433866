"""PagedKVCache's own checks, without a GPU: tensors that say they are on the cache's device, and a
library whose calls are only recorded."""
import importlib
import types

import pytest
import torch


class OnDevice(torch.Tensor):
    def get_device(self):
        return 0


def on(t):
    return t.as_subclass(OnDevice)


@pytest.fixture
def cache(monkeypatch):
    from compressed_attention_turboquantprod_b200 import build
    build.build()
    from compressed_attention_turboquantprod_b200 import PagedKVCache
    native = importlib.import_module("compressed_attention_turboquantprod_b200.native")
    c = PagedKVCache.__new__(PagedKVCache)
    c.desc = native.make_paged_desc(1, 2, 64, 16, 10, 4, 5, torch.bfloat16, 0)
    c.dtype, c._index, c._ws, c._cu = torch.bfloat16, 0, {}, {}
    c.buffer = types.SimpleNamespace(device=torch.device("cuda", 0))
    c.state = native.tq_paged_layout(c.desc)
    c.calls = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for name, f in list(vars(native).items()):
        if name.startswith("tq_paged_") and isinstance(f, types.FunctionType):
            monkeypatch.setattr(native, name, lambda *a, _n=name, **k: c.calls.append(_n))
    return c


def i32(x):
    return on(torch.tensor(x, dtype=torch.int32))


def test_a_workspace_of_another_device_is_refused(cache):
    Q, out = (on(torch.zeros(3, 4, 64, dtype=torch.bfloat16)) for _ in range(2))
    args = (Q, i32([0]), i32([0, 3]), 3)
    with pytest.raises(ValueError):
        cache.attend(*args, out=out, workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    assert cache.calls == []
    cache.attend(*args, out=out, workspace=on(torch.zeros(1 << 20, dtype=torch.uint8)))
    assert cache.calls == ["tq_paged_attention"]
