"""The paged 8-bit cache without a GPU: layout, host refusals, the oracle against brute force."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import paged as op

host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="host-only checks use fake device pointers")
FAKE = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 4)


@pytest.fixture(scope="module")
def nat():
    from compressed_attention_turboquantprod_b200 import build
    build.build()
    from compressed_attention_turboquantprod_b200 import native
    return native


def _desc(nat, **kw):
    p = dict(layers=1, Hkv=8, d=128, page=64, pages=100, slots=4, max_pages=30, dtype=2, code=0)
    p.update(kw)
    return nat.make_paged_desc(*(p[k] for k in ("layers", "Hkv", "d", "page", "pages", "slots",
                                                "max_pages", "dtype", "code")))


@host_only
@pytest.mark.parametrize("page,d,es,dt", [(16, 64, 4, 0), (64, 128, 2, 2), (128, 256, 2, 1), (32, 128, 4, 0)])
def test_layout(nat, page, d, es, dt):
    c = nat.tq_paged_layout(_desc(nat, page=page, d=d, dtype=dt, layers=3))
    sub = min(page, 64)
    assert c.sub_bytes == sub * d + 32 and c.block_bytes == page // sub * c.sub_bytes
    assert c.page_bytes == 2 * 8 * c.block_bytes
    assert c.o_pool - c.o_tail == 3 * 4 * 2 * 8 * page * d * es
    assert c.bytes - c.o_pool >= 3 * 100 * c.page_bytes > c.bytes - c.o_pool - 256
    offs = [c.o_state, c.o_len, c.o_table, c.o_ref, c.o_claim, c.o_rows, c.o_scan, c.o_moves, c.o_remap,
            c.o_tail, c.o_pool]
    assert offs == sorted(set(offs)) and all(o % 256 == 0 for o in offs)
    assert nat.tq_paged_bytes(_desc(nat, page=page, d=d, dtype=dt, layers=3)) == c.bytes


@host_only
@pytest.mark.parametrize("kw,status", [
    (dict(d=96), 2), (dict(page=48), 2), (dict(page=256), 2), (dict(code=2), 2), (dict(layers=0), 1),
    (dict(Hkv=0), 1), (dict(pages=0), 1), (dict(pages=(1 << 20) + 1), 1), (dict(slots=0), 1),
    (dict(slots=65537), 1), (dict(max_pages=0), 1), (dict(max_pages=(1 << 24) + 1), 2), (dict(dtype=3), 1)])
def test_bad_descriptors(nat, kw, status):
    assert nat.tq_paged_bytes(_desc(nat, **kw)) == 0
    with pytest.raises(nat.TQError) as e:
        nat.tq_paged_layout(_desc(nat, **kw))
    assert e.value.status == status


@host_only
def test_host_refusals(nat):
    L, bad, S = nat.lib, nat.TQ_ERR_INVALID_ARG, None
    c = nat.tq_paged_layout(_desc(nat))
    r = ctypes.byref(c)
    assert L.tq_paged_extend(r, FAKE, FAKE, 1, S) == bad                     # no memory bound
    c.base = 1 << 20
    d = _desc(nat)
    assert L.tq_paged_init(r, ctypes.byref(d), FAKE, 1000, S) == bad
    assert L.tq_paged_init(r, ctypes.byref(d), ODD, 1 << 40, S) == bad
    assert L.tq_paged_init(r, ctypes.byref(d), None, 1 << 40, S) == bad
    for n in (0, -1, 5):
        assert L.tq_paged_extend(r, FAKE, FAKE, n, S) == bad
    assert L.tq_paged_extend(r, None, FAKE, 1, S) == bad
    assert L.tq_paged_extend(r, FAKE, ctypes.c_void_p((1 << 20) + 2), 1, S) == bad
    w = 8 * 128
    assert L.tq_paged_write(r, 0, FAKE, FAKE, w, w, 10, S) == bad            # nothing extended
    c.plan_rows = 1
    assert L.tq_paged_write(r, 1, FAKE, FAKE, w, w, 10, S) == bad            # layer
    assert L.tq_paged_write(r, 0, FAKE, FAKE, w - 8, w, 10, S) == bad        # tokens overlap
    assert L.tq_paged_write(r, 0, FAKE, FAKE, w, w + 4, 10, S) == bad        # not 16 bytes
    assert L.tq_paged_write(r, 0, FAKE, ODD, w, w, 10, S) == bad
    assert L.tq_paged_write(r, 0, FAKE, FAKE, w, w, -1, S) == bad
    assert L.tq_paged_write(r, 0, None, None, w, w, 0, S) == nat.TQ_OK       # nothing to do
    assert L.tq_paged_read(r, 0, FAKE, FAKE, 1, 5, FAKE, None, S) == bad
    assert L.tq_paged_read(r, -1, FAKE, FAKE, 1, 5, FAKE, FAKE, S) == bad
    assert L.tq_paged_read(r, 0, FAKE, FAKE, 1, 0, None, None, S) == nat.TQ_OK
    ws = L.tq_paged_workspace_bytes(r)
    assert ws > 0

    def attn(layer=0, Q=FAKE, qs=32 * 128, Hq=32, n=1, mq=1, total=1, scale=0.1, out=FAKE, wsp=FAKE, wsb=ws):
        return L.tq_paged_attention(r, layer, Q, qs, Hq, FAKE, FAKE, n, mq, total, 1, scale, out, None, wsp, wsb, S)
    assert attn(Hq=30) == nat.TQ_ERR_UNSUPPORTED and attn(Hq=72, qs=72 * 128) == nat.TQ_ERR_UNSUPPORTED
    assert attn(Hq=4) == nat.TQ_ERR_UNSUPPORTED
    for kw in (dict(layer=1), dict(Q=None), dict(Q=ODD), dict(qs=31 * 128), dict(qs=32 * 128 + 4), dict(n=0),
               dict(mq=0), dict(total=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(out=None),
               dict(wsp=None), dict(wsp=ODD), dict(wsb=ws - 1)):
        assert attn(**kw) == bad, kw
    assert attn(total=0) == nat.TQ_OK
    over = ctypes.c_void_p((1 << 20) + 64 * 1024)                             # the output over the queries
    assert attn(total=9, out=over) == bad and attn(total=9, Q=over, out=FAKE) == bad
    o = nat.tq_paged_layout(_desc(nat, Hkv=4))
    o.base = 1 << 21
    assert L.tq_paged_copy(r, ctypes.byref(o), FAKE, FAKE, 1, S) == bad
    assert L.tq_paged_fork(r, FAKE, None, 1, S) == bad and L.tq_paged_fork(r, FAKE, FAKE, 5, S) == bad
    assert L.tq_paged_free(r, None, 1, S) == bad and L.tq_paged_table(r, FAKE, 1, None, S) == bad
    c.page_bytes += 1                                                         # not the layout of its descriptor
    assert L.tq_paged_compact(r, S) == bad


@host_only
def test_faults_are_injected(nat):
    c = nat.tq_paged_layout(_desc(nat))
    c.base = 1 << 20
    for name, args in (("tq_paged_extend", (FAKE, FAKE, 1, None)), ("tq_paged_compact", (None,)),
                       ("tq_paged_free", (FAKE, 1, None)), ("tq_paged_check", (None, None))):
        nat.tq_debug_fail_next(name)
        assert getattr(nat.lib, name)(ctypes.byref(c), *args) == nat.TQ_ERR_CUDA
        assert nat.lib.tq_last_error() == b"injected fault"


@host_only
def test_binding_checks(nat):
    x = torch.zeros(4, 2, 64)
    assert nat._tokens(x, 2, 64)[1] == 128
    assert nat._tokens(torch.zeros(4, 6, 64)[:, 2:4], 2, 64)[1] == 384
    assert nat._tokens(torch.zeros(4, 6, 64)[:1, 2:4], 2, 64)[1] == 128
    for bad in (torch.zeros(4, 2, 32), torch.zeros(4, 64, 2).transpose(1, 2), torch.zeros(4, 128)):
        with pytest.raises(ValueError):
            nat._tokens(bad, 2, 64)
    with pytest.raises(ValueError):
        nat._i32(torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        nat._rows(torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        nat._pairs(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


# ---------------------------------------------------------------------------- the oracle itself
def _e4m3_values():
    v = []
    for e in range(16):
        for m in range(8):
            if e == 15 and m == 7:
                continue
            v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(v)


def test_oracle_rounds_to_the_nearest_code():
    vals = _e4m3_values()
    assert vals[-1] == 448.0 and (np.diff(vals) > 0).all()
    y = np.concatenate([np.linspace(0, 448, 4001), (vals[1:] + vals[:-1]) / 2, vals])
    got = op.round_e4m3(y)
    for a, b in zip(y, got):
        d = np.abs(vals - a)
        near = np.flatnonzero(d == d.min())
        want = vals[near[0]] if len(near) == 1 else vals[[i for i in near if i % 2 == 0][0]]
        assert b == want, a
    rng = np.random.default_rng(1)
    x = rng.standard_normal((16, 64)).astype(np.float32)
    v, s = op.block_values(x, "int8")
    a = np.abs(x).max().astype(np.float64)
    assert np.abs(v / s - 127.0 * x / a).max() <= 0.5 + 1e-9 and np.abs(v / s).max() == 127
    v, s = op.block_values(x, "e4m3")
    assert s == 2.0 ** np.round(np.log2(s)) and a / s <= 448 < 2 * a / s
    assert op.block_values(np.full((4, 4), 2.0 ** -101), "int8")[1] == 0.0


def test_oracle_attention_by_hand():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((5, 2, 8)), rng.standard_normal((5, 2, 8))
    out, lse, _, _ = op.attention(q, k, v, True, 0.3)
    for i in range(3):
        for h in range(4):
            w = [np.exp(0.3 * float(q[i, h] @ k[t, h // 2])) for t in range(5 - 3 + i + 1)]
            want = sum(a * v[t, h // 2] for t, a in enumerate(w)) / sum(w)
            assert np.allclose(out[i, h], want, atol=1e-12) and np.isclose(lse[i, h], np.log(sum(w)))
    assert (op.attention(q, k[:0], v[:0], False, 0.3)[0] == 0).all()
    out, lse, _, _ = op.attention(q, k[:1], v[:1], True, 0.3)
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.allclose(out[2], np.repeat(v[0], 2, 0))


def test_model_of_the_pages():
    m = op.PagedModel(1, 4, 8, 4, 4, 2, "int8")
    m.append(0, [(np.ones((5, 1, 4)),) * 2])
    m.fork(0, 1)
    assert m.table[1] == [0, 1, 3] and m.ref[:5] == [2, 2, 1, 1, 0]
    m.free(0)
    assert m.ref[:4] == [1, 1, 0, 1]
    m.compact()
    assert m.table[1] == [0, 1, 2] and m.ref[:4] == [1, 1, 1, 0]
    with pytest.raises(RuntimeError):
        m.append(2, [(np.ones((12, 1, 4)),) * 2])
