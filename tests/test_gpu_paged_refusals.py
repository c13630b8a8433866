"""Calls on the paged cache that are refused, or that come in an order or at a time that other tests do
not try: what they leave behind."""
import numpy as np
import pytest
import torch

from gpu_common import host, nat
from test_gpu_paged import check_attention, fill, i32, make, offsets, same_tables, same_values, tokens

pytestmark = pytest.mark.gpu


def dirty(c, m, dtype):
    """Every page and tail filled with large values of a sequence that is gone."""
    n = min(c.desc.pages // c.desc.slots, c.desc.max_pages) * c.desc.page
    big = 1e3 + tokens(n * c.desc.slots, m.Hkv, m.d, dtype, 900)
    slots = i32(range(c.desc.slots))
    c.extend(slots, offsets([n] * c.desc.slots))
    for l in range(m.layers):
        c.write(big, big, layer=l)
    c.free(slots)
    c.check()


def refused(c, m, dtype, status, call):
    from compressed_attention_turboquantprod_b200 import TQError
    call()
    with pytest.raises(TQError) as e:
        c.check()
    assert e.value.status == status
    same_tables(c, m)
    for l in range(m.layers):
        same_values(c, m, dtype, layer=l)


@pytest.mark.parametrize("code,page", [("int8", 16), ("e4m3", 64)])
def test_an_append_past_its_tokens_is_refused_whole(code, page):
    bad = nat().TQ_ERR_INVALID_ARG
    c, m = make(2, 64, 32, 4, 8, page, code, "f16")
    dirty(c, m, "f16")
    fill(c, m, [20, 16], "f16", 71)
    K = tokens(80, 2, 64, "f16", 72)
    for given, rows, cu in ((3, [3], [0, 9]), (0, [3], [0, 9]), (0, [0], [0, 1]), (3, [0, 3], [0, 2, 4]),
                            (3, [2, 0, 1], [1, 2, 3, 60]), (9, [0], [9, 10])):
        refused(c, m, "f16", bad, lambda: c.append(K[:given], K[:given], i32(rows), i32(cu)))
    # past the tokens, but of no row: padding, and a row without tokens
    c.append(K[:3], K[:3], i32([0, -1, 1]), i32([0, 3, 50, 50]))
    m.append(0, [(host(K[:3]), host(K[:3]))])
    same_tables(c, m)
    same_values(c, m, "f16")


def test_an_extend_that_knows_its_tokens_is_refused_whole():
    n = nat()
    c, m = make(1, 128, 20, 3, 8, 32, "int8", "bf16", layers=2)
    dirty(c, m, "bf16")
    fill(c, m, [40, 3], "bf16", 73)
    refused(c, m, "bf16", n.TQ_ERR_INVALID_ARG, lambda: c.extend(i32([1, 2]), i32([0, 5, 9]), total=8))
    with pytest.raises(n.TQError):
        c.extend(i32([1]), i32([0, 5]), total=-1)
    same_tables(c, m)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("code,d,page", [("int8", 128, 32), ("e4m3", 64, 128), ("int8", 256, 64)])
@pytest.mark.parametrize("counts", [(5, 1), (200, 40), (0, 300)])
def test_a_write_that_is_given_too_few_tokens_stores_zeros(dtype, code, d, page, counts):
    """Nothing of what the pages or tails held before shows, and later appends build on the zeros."""
    from compressed_attention_turboquantprod_b200 import TQError
    c, m = make(2, d, 40, 3, 12, page, code, dtype)
    dirty(c, m, dtype)
    fill(c, m, [page // 2 + 3, 1], dtype, 75)
    total = sum(counts)
    c.extend(i32([0, 2]), offsets(counts))
    short = tokens(total - 1 if total < 100 else 2, 2, d, dtype, 76)
    c.write(short, short)
    with pytest.raises(TQError) as e:
        c.check()
    assert e.value.status == nat().TQ_ERR_INVALID_ARG
    for s, n in zip((0, 2), counts):
        m.append(s, [(np.zeros((n, 2, d)),) * 2])
    same_tables(c, m)
    same_values(c, m, dtype)
    fill(c, m, [3, page, 2], dtype, 77)
    same_tables(c, m)
    same_values(c, m, dtype)


def test_a_captured_write_behind_another_plan():
    """A graph holds a write for one row; a plan of nine rows comes before its replay."""
    from compressed_attention_turboquantprod_b200 import TQError
    c, m = make(1, 64, 40, 10, 4, 16, "int8", "f16")
    dirty(c, m, "f16")
    K = tokens(400, 1, 64, "f16", 78)
    c.extend(i32([0]), i32([0, 1]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.write(K, K)
    g.replay()
    m.append(0, [(host(K[:1]),) * 2])
    c.check()
    c.extend(i32(range(1, 10)), offsets([30] * 9))
    g.replay()
    with pytest.raises(TQError):
        c.check()
    for s in range(1, 10):
        m.append(s, [(np.zeros((30, 1, 64)),) * 2])
    same_tables(c, m)
    same_values(c, m, "f16")


def test_a_slot_freed_before_its_write_is_left_out():
    """Its page has gone to another sequence's fork by then."""
    from compressed_attention_turboquantprod_b200 import TQError
    c, m = make(2, 64, 12, 4, 4, 16, "int8", "f16")
    fill(c, m, [1], "f16", 81, slots=[2])
    K = tokens(30, 2, 64, "f16", 82)
    c.extend(i32([0, 1]), i32([0, 20, 30]))
    c.free(i32([0]))
    c.fork(i32([2]), i32([3]))
    c.write(K, K)
    with pytest.raises(TQError) as e:
        c.check()
    assert e.value.status == nat().TQ_ERR_INVALID_ARG
    table = c.page_table(i32([1, 3])).cpu()
    assert table[1, 0] == 1 and table[0, 0] == 3          # pages 1 and 2 were slot 0's
    m.append(1, [(host(K[20:]),) * 2])
    m.fork(2, 3)
    same_values(c, m, "f16")


def test_check_reports_every_reason_once():
    from compressed_attention_turboquantprod_b200 import TQError
    n = nat()
    c, m = make(1, 64, 6, 4, 4, 16, "int8", "f16")
    fill(c, m, [20], "f16", 91)
    K = tokens(80, 1, 64, "f16", 92)
    c.append(K, K, i32([2, 2]), i32([0, 1, 2]))            # a slot twice
    c.append(K, K, i32([1, 2]), i32([0, 40, 80]))          # six pages, four are free
    c.fork(i32([1]), i32([0]))                             # not empty
    with pytest.raises(TQError) as e:
        c.check()
    assert e.value.status == n.TQ_ERR_CAPACITY
    for text in ("free pages", "named twice", "not empty"):
        assert text in e.value.message
    assert c.check() == 4
    same_tables(c, m)


@pytest.mark.parametrize("cu", [[0, 20, 10, 36], [0, 5, 5, 41], [-1, 5, 20, 36], [30, 20, 10, 0]])
def test_a_read_with_bad_offsets_is_reported(cu):
    from compressed_attention_turboquantprod_b200 import TQError
    c, m = make(1, 64, 6, 3, 4, 16, "int8", "f16")
    fill(c, m, [20, 16, 3], "f16", 95)
    c.read(i32([0, 1, 2]), i32(cu), 40)
    with pytest.raises(TQError) as e:
        c.check()
    assert e.value.status == nat().TQ_ERR_INVALID_ARG
    same_values(c, m, "f16")


def test_a_batch_without_queries():
    c, m = make(1, 64, 6, 2, 4, 16, "int8", "f16")
    fill(c, m, [20], "f16", 97)
    Q = tokens(1, 2, 64, "f16", 98)
    out = c.attend(Q[:0], i32([0, 1]), i32([0, 0, 0]), 0)
    assert out.shape == (0, 2, 64) and c.check() == 4
    c.append(Q[:0, :1], Q[:0, :1], i32([0, 1]), i32([0, 0, 0]))
    K, V = c.read(i32([0, 1]), i32([0, 0, 0]), 0)
    assert K.shape == V.shape == (0, 1, 64)
    same_tables(c, m)


@pytest.mark.parametrize("d,G,nq,lens", [(64, 1, 40, [700, 90]), (128, 4, 70, [9000, 300]), (256, 2, 33, [400, 17000])])
def test_chunks_at_once_and_captured(d, G, nq, lens):
    """Chunk calls on two streams at a time, and two graphs of them replayed on both: each has a workspace of
    its own; at d = 64 their CTAs share SMs, and so wait for each other's tensor memory."""
    c, m = make(2, d, 400, 2, 300, 64, "int8", "bf16")
    fill(c, m, lens, "bf16", 101)
    rows, cu = i32([0, 1]), offsets([nq, nq])
    Q = [tokens(2 * nq, 2 * G, d, "bf16", 102 + i, 0.3) for i in range(2)]

    def call(i):
        return c.attend(Q[i], rows, cu, nq, causal=i == 0)
    want = [call(0), call(1)]
    if d != 128:
        check_attention(c, m, Q[0], [0, 1], [nq, nq], True, "bf16", single_p=True)
    st, got, graphs = [torch.cuda.Stream() for _ in range(2)], [], []
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(st[i]):
                got.append((i, call(i)))
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call(i)
        graphs.append((g, out))
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(st[i]):
                graphs[i][1].zero_()
                graphs[i][0].replay()
        torch.cuda.synchronize()
        got += [(i, graphs[i][1].clone()) for i in range(2)]
    torch.cuda.synchronize()
    for i, g in got:
        assert torch.equal(g, want[i])
    c.check()


def test_captured_appends_with_padding_rows():
    """A padded batch: offsets and slots change between replays, rows come and go as padding."""
    c, m = make(2, 128, 60, 4, 12, 32, "e4m3", "bf16")
    dirty(c, m, "bf16")
    K, V = (torch.zeros(64, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots, cu = i32([-1] * 4), i32([0] * 5)
    c.append(K, V, slots, cu)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.append(K, V, slots, cu)
    for step, (s, counts) in enumerate((([2, -1, 0, 1], [30, 4, 1, 20]), ([3, 0, -1, -1], [33, 1, 9, 9]), ([-1] * 4, [0] * 4),
                                        ([1, 2, 3, 0], [1, 1, 1, 61]))):
        k, v = (tokens(64, 2, 128, "bf16", 110 + 2 * step + j) for j in range(2))
        K.copy_(k), V.copy_(v), slots.copy_(i32(s)), cu.copy_(offsets(counts))
        g.replay()
        at = 0
        for slot, n in zip(s, counts):
            if slot >= 0:
                m.append(slot, [(host(k[at:at + n]), host(v[at:at + n]))])
            at += n
        same_tables(c, m)
        same_values(c, m, "bf16")
