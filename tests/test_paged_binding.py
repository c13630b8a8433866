"""PagedKVCache's own checks, without a GPU: tensors that say they are on the cache's device, and a
library whose calls are only recorded."""
import ctypes
import importlib
import types

import pytest
import torch


class OnDevice(torch.Tensor):
    def get_device(self):
        return 0


def on(t):
    return t.as_subclass(OnDevice)


class Library:
    """Every call succeeds and is noted."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


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
    lib = Library()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(native, "raw_stream", lambda device: 0)
    monkeypatch.setattr(native, "lib", lib)
    c.calls = lib.calls
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


def test_an_append_is_checked_before_its_plan(cache):
    bf, z = torch.bfloat16, torch.zeros
    good, slots, cu = on(z(3, 2, 64, dtype=bf)), i32([0]), i32([0, 3])
    for K, V, s, o in ((good, good[:2], slots, cu), (on(z(3, 2, 32, dtype=bf)),) * 2 + (slots, cu),
                       (good, on(z(3, 64, 2, dtype=bf)).transpose(1, 2), slots, cu), (good, good, slots, i32([0])),
                       (good, good, slots, on(torch.tensor([0, 3]))), (good, on(z(3, 2, 64)), slots, cu),
                       (good, z(3, 2, 64, dtype=bf), slots, cu)):
        with pytest.raises(ValueError):
            cache.append(K, V, s, o)
        assert cache.calls == []
    cache.append(good, good, slots, cu)
    assert cache.calls == ["tq_paged_append"]


def test_a_decode_step_is_checked_before_its_append(cache):
    bf, z = torch.bfloat16, torch.zeros
    K, slots, cu, ws = on(z(1, 2, 64, dtype=bf)), i32([0]), i32([0, 1]), on(z(64, dtype=torch.uint8))
    Q, out = (on(z(1, 4, 64, dtype=bf)) for _ in range(2))
    for q, kw in ((on(z(1, 4, 32, dtype=bf)), {}), (on(z(1, 4, 64)), {}), (on(z(4, 64, dtype=bf)), {}),
                  (z(1, 4, 64, dtype=bf), {}), (Q, dict(out=on(z(1, 4, 64)))), (Q, dict(lse=on(z(1, 3)))),
                  (Q, dict(workspace=z(64))), (Q, dict(out=on(z(1, 4, 128, dtype=bf))[..., ::2])),
                  (on(z(1, 3, 64, dtype=bf)), dict(out=on(z(1, 3, 64, dtype=bf)))),
                  (on(z(1, 18, 64, dtype=bf)), dict(out=on(z(1, 18, 64, dtype=bf)))),
                  (on(z(260, dtype=bf))[4:].view(1, 4, 64), {}), (Q, dict(out=on(z(260, dtype=bf))[4:].view(1, 4, 64))),
                  (Q, dict(lse=on(z(1, 8))[:, ::2])), (Q, dict(softmax_scale=float("nan")))):
        with pytest.raises(ValueError):
            cache.decode_step(K, K, q, slots, cu, **{**dict(out=out, workspace=ws), **kw})
        assert cache.calls == []
    cache.decode_step(K, K, Q, slots, cu, out=out, workspace=ws)
    assert cache.calls == ["tq_paged_append", "tq_paged_attention"]


@pytest.mark.skipif(torch.cuda.is_available(), reason="uses fake device pointers")
def test_append_refusals_of_the_library():
    native = importlib.import_module("compressed_attention_turboquantprod_b200.native")
    L, bad, S = native.lib, native.TQ_ERR_INVALID_ARG, None
    fake, odd, w = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 4), 2 * 64
    c = native.tq_paged_layout(native.make_paged_desc(1, 2, 64, 16, 10, 4, 5, torch.bfloat16, 0))
    c.base = 1 << 20

    def append(c=c, slots=fake, cu=fake, n=1, K=fake, V=fake, ks=w, vs=w, total=5):
        return L.tq_paged_append(ctypes.byref(c), slots, cu, n, K, V, ks, vs, total, S)
    for kw in (dict(slots=None), dict(cu=ctypes.c_void_p(3)), dict(n=0), dict(n=5), dict(K=None), dict(V=odd), dict(ks=w - 8),
               dict(vs=w + 4), dict(total=-1), dict(total=1 << 31)):
        assert append(**kw) == bad, kw
        assert c.plan_rows == 0
    two = native.tq_paged_layout(native.make_paged_desc(2, 2, 64, 16, 10, 4, 5, torch.bfloat16, 0))
    two.base = 1 << 20
    assert append(c=two) == bad
    assert L.tq_paged_extend_within(ctypes.byref(c), fake, fake, 1, -1, S) == bad
    for name, args in (("tq_paged_append", (fake, fake, 1, fake, fake, w, w, 5, S)), ("tq_paged_extend_within", (fake, fake, 1, 5, S))):
        native.tq_debug_fail_next(name)
        assert getattr(L, name)(ctypes.byref(c), *args) == native.TQ_ERR_CUDA
        assert L.tq_last_error() == b"injected fault"


@pytest.mark.skipif(torch.cuda.is_available(), reason="uses fake device pointers")
def test_attention_without_queries():
    """The longest of no rows is 0."""
    native = importlib.import_module("compressed_attention_turboquantprod_b200.native")
    fake = ctypes.c_void_p(1 << 20)
    c = native.tq_paged_layout(native.make_paged_desc(1, 2, 64, 16, 10, 4, 5, torch.bfloat16, 0))
    c.base = 1 << 20

    def attention(max_q, total):
        return native.lib.tq_paged_attention(ctypes.byref(c), 0, None, 256, 4, fake, fake, 1, max_q, total, 1, 0.1, None, None,
                                             fake, 1 << 40, None)
    assert attention(0, 0) == native.TQ_OK and attention(5, 0) == native.TQ_OK
    assert attention(-1, 0) == native.TQ_ERR_INVALID_ARG and attention(0, 1) == native.TQ_ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="uses fake device pointers")
def test_arrays_that_overlap():
    """Apart, the calls come as far as the missing GPU; over one another they are refused before."""
    native = importlib.import_module("compressed_attention_turboquantprod_b200.native")
    L, bad = native.lib, native.TQ_ERR_INVALID_ARG
    c = native.tq_paged_layout(native.make_paged_desc(1, 2, 64, 16, 10, 4, 5, torch.bfloat16, 0))
    c.base = 1 << 30
    ws = L.tq_paged_workspace_bytes(ctypes.byref(c))
    at = dict(base=1 << 30, q=2 << 30, out=3 << 30, lse=4 << 30, ws=5 << 30, k=6 << 30, v=7 << 30)
    row = 4 * 64 * 2

    def attention(**kw):
        a = {**at, **kw}
        c.base = a["base"]
        return L.tq_paged_attention(ctypes.byref(c), 0, a["q"], 512, 4, at["k"], at["v"], 1, 9, 9, 1, 0.1, a["out"], a["lse"],
                                    a["ws"], ws, None)

    def read(**kw):
        a = {**at, **kw}
        c.base = a["base"]
        return L.tq_paged_read(ctypes.byref(c), 0, at["q"], at["q"], 1, 9, a["k"], a["v"], None)
    end = {"base": (1 << 30) + c.bytes, "q": (2 << 30) + 8 * 1024 + row, "out": (3 << 30) + 9 * row, "lse": (4 << 30) + 9 * 16,
           "ws": (5 << 30) + ws, "k": (6 << 30) + 9 * 256}
    assert attention() == native.TQ_ERR_CUDA and attention(lse=None) == native.TQ_ERR_CUDA
    for a, b in (("out", "q"), ("out", "lse"), ("out", "ws"), ("out", "base"), ("lse", "q"), ("lse", "ws"), ("lse", "base"),
                 ("ws", "q"), ("ws", "base")):
        up = lambda x: -(-x // 256) * 256
        assert attention(**{a: at[b]}) == bad, (a, b)
        assert attention(**{a: up(end[b] - 255) if a != "lse" else end[b] - 4}) == bad or up(end[b] - 255) >= end[b], (a, b)
        assert attention(**{a: up(end[b])}) == native.TQ_ERR_CUDA, (a, b)
    assert read() == native.TQ_ERR_CUDA and read(k=end["k"], v=at["k"]) == native.TQ_ERR_CUDA
    for kw in (dict(v=at["k"]), dict(v=end["k"] - 16), dict(k=at["base"]), dict(v=end["base"] - 256)):
        assert read(**kw) == bad, kw
