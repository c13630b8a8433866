"""The paged 8-bit cache on the GPU against the float64 oracle.

Tolerances.  Stored values: the codes are exact by definition (ties decided exactly), so a read
value differs from code * scale by the fp32 product (2^-24) and one rounding to the output type.
Attention: a logit is a sum of d products held in fp32, off by at most (d + 8) 2^-24 of
scale * sum |q k| (`reach`); a weight is then off by twice that relatively, plus the exponential
and the sums (2^-19 together: 2 ulp of exp2, the running sums, q and p split into two halves of
11 bits), or plus 2^-11 where p is rounded to one half (chunks of bf16 / f16).  The output is off by that
times sum p |v| (`mass`), plus its own rounding.
Halves also have a smallest step, 2^-24, so what is held of a tiny p is off absolutely: p (at most 1
against the running maximum, times its page's value scale over the largest one of the tile, at most
1) is held times 2^15, the last rounding is off by at most 2^-25, so p by 2^-40, times a code times
the tile's largest scale, at most max |v|.  Over the visible tokens that is 2^-40 n max |v| (`floor`): later
rescaling only shrinks it, and the sum it is divided by is at least 1.  Chunks of bf16 / f16 hold p
times 2^11 against a reference that may lag by 2^4, so 2^-36 there."""
import math

import numpy as np
import pytest
import torch

from gpu_common import TORCH_DT, host, nat
from oracle import paged as op

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}     # half the smallest step


def make(Hkv, d, pages, slots, max_pages, page=64, code="int8", dtype="bf16", layers=1):
    nat()
    from compressed_attention_turboquantprod_b200 import PagedKVCache
    c = PagedKVCache(Hkv, d, pages, slots, max_pages, page=page, code=code, dtype=TORCH_DT[dtype],
                     layers=layers)
    return c, op.PagedModel(Hkv, d, pages, slots, max_pages, page, code, layers)


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def offsets(counts):
    return i32(np.cumsum([0] + list(counts)))


def tokens(n, H, d, dtype, seed, spread=0.7):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, H, d, generator=g) * torch.exp(spread * torch.randn(n, H, 1, generator=g))
    return x.to(TORCH_DT[dtype]).cuda()


def fill(c, m, counts, dtype, seed=0, slots=None):
    """Append counts[i] tokens to slots[i] on both sides."""
    slots = list(range(len(counts))) if slots is None else slots
    KV = [(tokens(sum(counts), m.Hkv, m.d, dtype, seed + 2 * l), tokens(sum(counts), m.Hkv, m.d, dtype, seed + 2 * l + 1))
          for l in range(m.layers)]
    c.extend(i32(slots), offsets(counts))
    for l, (K, V) in enumerate(KV):
        c.write(K, V, layer=l)
    at = 0
    for s, n in zip(slots, counts):
        if s >= 0:
            m.append(s, [(host(K[at:at + n]), host(V[at:at + n])) for K, V in KV])
        at += n


def same_tables(c, m):
    n = len(m.table)
    got = c.page_table(i32(range(n))).cpu().tolist()
    want = [t + [-1] * (m.max_pages - len(t)) for t in m.table]
    assert got == want
    assert c.lengths.cpu().tolist() == m.len
    assert c.check() == sum(r == 0 for r in m.ref)


def same_values(c, m, dtype, slots=None, layer=0):
    slots = [s for s in range(len(m.len)) if m.len[s]] if slots is None else slots
    counts = [m.len[s] for s in slots]
    K, V = c.read(i32(slots), offsets(counts), sum(counts), layer=layer)
    at = 0
    for s, n in zip(slots, counts):
        for got, want in zip((K, V), m.values(s, layer)):
            g = host(got[at:at + n])
            # an input's infinity saturates at the top code, inside the type's range unless the
            # block itself reaches the type's largest value
            tol = np.abs(want) * (HALF[dtype] + 2.0 ** -23) + TINY[dtype]
            bad = np.abs(g - want) > tol
            assert not bad.any(), (s, int(bad.sum()), float(np.abs(g - want).max()))
        at += n


def check_attention(c, m, Q, rows, counts, causal, dtype, scale=None, single_p=False, layer=0, out=None, lse=None):
    d = m.d
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    got_lse = torch.full(Q.shape[:2], 7.0, device="cuda") if lse is None else lse
    got = c.attend(Q, i32(rows), offsets(counts), max(max(counts), 1), causal, scale, layer, out=out, lse=got_lse)
    at = 0
    q64 = host(Q)
    for s, n in zip(rows, counts):
        ok = 0 <= s < len(m.len)
        k, v = m.values(s, layer) if ok else (np.zeros((0, m.Hkv, d)),) * 2
        want, wl, mass, reach = op.attention(q64[at:at + n], k, v, causal, sc)
        ew = 2 * (d + 8) * 2.0 ** -24 * reach + 2.0 ** -19 + (2.0 ** -11 if single_p else 0.0)
        floor = 2.0 ** (-36 if single_p else -40) * len(v) * np.abs(v).max() if len(v) else 0.0
        tol = floor + ew[..., None] * mass + HALF[dtype] * (np.abs(want) + ew[..., None] * mass) + TINY[dtype]
        err = np.abs(host(got[at:at + n]) - want)
        assert (err <= tol).all(), (s, n, float((err / np.maximum(tol, 1e-300)).max()), float(err.max()))
        gl = got_lse[at:at + n].cpu().double().numpy()
        assert (np.isneginf(gl) == np.isneginf(wl)).all()
        f = np.isfinite(wl)
        assert (np.abs(gl[f] - wl[f]) <= ew[f] + 2.0 ** -22 * (1 + np.abs(wl[f]))).all()
        at += n
    return got


# ---------------------------------------------------------------------------- storage
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("d,page", [(64, 16), (64, 128), (128, 64), (128, 32), (256, 128), (256, 16)])
def test_append_read(dtype, code, d, page):
    c, m = make(3, d, 60, 6, 30, page, code, dtype)
    fill(c, m, [1, 0, page, page + 1, 3 * page - 1, 200], dtype, 1)
    same_tables(c, m)
    same_values(c, m, dtype)
    fill(c, m, [1, 5, 1, page], dtype, 2, slots=[3, 1, 0, 4])      # a second chunk, slots in another order
    same_tables(c, m)
    same_values(c, m, dtype)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_token_by_token_equals_one_append(code, d):
    """The bytes of the pages do not depend on how the tokens were split into appends."""
    a, m = make(2, d, 8, 1, 4, 32, code, "bf16")
    b, _ = make(2, d, 8, 1, 4, 32, code, "bf16")
    n = 71
    K, V = tokens(n, 2, d, "bf16", 5), tokens(n, 2, d, "bf16", 6)
    a.append(K, V, i32([0]), offsets([n]))
    for t in range(n):
        b.append(K[t:t + 1], V[t:t + 1], i32([0]), offsets([1]))
    assert torch.equal(a.page_table(i32([0])), b.page_table(i32([0])))
    for x, y in zip(a.read(i32([0]), offsets([n]), n), b.read(i32([0]), offsets([n]), n)):
        assert torch.equal(x, y)
    m.append(0, [(host(K), host(V))])
    same_values(b, m, "bf16")


def test_int8_ties_and_bad_entries():
    """127 x / a on a half in every binade (exact ties go to the even code); infinities saturate,
    NaN reads back as 0 and neither touches its block's scale; a block of zeros; a tiny block."""
    c, m = make(1, 64, 8, 1, 8, 16, "int8", "f32")
    x = torch.zeros(64, 1, 64)
    x[0:16, 0] = (torch.arange(1024).reshape(16, 64) % 127 + 0.5) / 127.0      # a = 1 below: near ties
    x[0, 0, 0] = 127.0 / 127.0
    x[16:32, 0] = (torch.arange(1024).reshape(16, 64) % 128).float() - 63.5    # a = 254: exact ties
    x[16, 0, 0] = 254.0
    x[32, 0, 0], x[32, 0, 1], x[33, 0, 5], x[33, 0, 6] = float("inf"), float("-inf"), float("nan"), 3.0
    x[48:64] = 2.0 ** -110
    x = x.cuda()
    c.append(x, x, i32([0]), offsets([64]))
    m.append(0, [(host(x), host(x))])
    same_values(c, m, "f32")
    K, _ = c.read(i32([0]), offsets([64]), 64)
    assert float(K[33, 0, 5]) == 0.0 and (K[48:] == 0).all() and float(K[32, 0, 0]) == pytest.approx(3.0)


def test_e4m3_borders():
    c, m = make(1, 64, 8, 1, 8, 16, "e4m3", "f32")
    x = torch.zeros(48, 1, 64)
    y = (torch.arange(1024).float() / 1024.0 * 448.0).reshape(16, 64)
    y[0, 0] = 448.0                              # a / scale = 448 exactly: scale 1
    x[0:16, 0] = y
    x[16:32, 0] = y * 2.0 ** -30
    x[16, 0, 0] = 448.0 * (1 + 2.0 ** -20) * 2.0 ** -30     # just above: the scale doubles
    x[32:48, 0] = 2.0 ** -9 * torch.arange(1024).reshape(16, 64) / 64
    x[32, 0, 0] = 400.0                          # subnormal codes, ties among them
    x = x.cuda()
    c.append(x, -x, i32([0]), offsets([48]))
    m.append(0, [(host(x), host(-x))])
    same_values(c, m, "f32")


def test_strided_projection_views_and_padding_rows():
    """K, V, Q as views into one fused projection; a padding row's tokens are left out; rows
    behind the last sequence stay as they were."""
    c, m = make(2, 128, 20, 4, 8, 64, "int8", "bf16")
    Hq, n = 8, 90
    qkv = tokens(n, Hq + 4, 128, "bf16", 9)
    Q, K, V = qkv[:, :Hq], qkv[:, Hq:Hq + 2], qkv[:, Hq + 2:]
    rows, counts = [2, -1, 0], [50, 10, 20]              # 10 tokens behind the last sequence
    c.append(K, V, i32(rows), offsets(counts))
    m.append(2, [(host(K[:50]), host(V[:50]))])
    m.append(0, [(host(K[60:80]), host(V[60:80]))])
    same_tables(c, m)
    same_values(c, m, "bf16")
    out = torch.full((n, Hq, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, Hq), 3.0, device="cuda")
    got = check_attention(c, m, Q, rows, counts, True, "bf16", single_p=True, out=out, lse=lse)
    assert (got[50:60] == 0).all() and (got[80:] == 3.0).all() and (lse[80:] == 3.0).all()
    assert torch.isneginf(lse[50:60]).all()


# ---------------------------------------------------------------------------- attention
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("d,page,G", [(64, 16, 1), (64, 32, 6), (128, 64, 4), (128, 16, 8), (128, 128, 3),
                                      (256, 128, 4), (256, 32, 8)])
def test_decode(dtype, code, d, page, G):
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 129, 700]
    c, m = make(2, d, 120, len(lens), 50, page, code, dtype)
    fill(c, m, lens, dtype, 3)
    rows = list(range(len(lens))) + [3, -1, 9]           # a slot named twice, a padding row
    Q = tokens(len(rows), 2 * G, d, dtype, 4, 0.3)
    check_attention(c, m, Q, rows, [1] * len(rows), True, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decode_long_and_scales_far_apart(dtype):
    """Thousands of tokens across many CTAs; pages whose magnitudes differ by 2^40."""
    c, m = make(1, 128, 400, 2, 400, 16, "int8", dtype)
    n = 6001
    K, V = tokens(n, 1, 128, dtype, 5), tokens(n, 1, 128, dtype, 6)
    V[100:160] *= 2.0 ** 20
    V[1000:1100] *= 2.0 ** -20
    K[2000:2100] *= 2.0 ** -20
    c.append(K, V, i32([1]), offsets([n]))
    m.append(1, [(host(K), host(V))])
    Q = tokens(1, 4, 128, dtype, 7)
    check_attention(c, m, Q, [1], [1], True, dtype)


def test_decode_large_logits_and_scales():
    """Logits of hundreds: one token takes all the weight; a negative and a zero scale."""
    c, m = make(1, 64, 40, 1, 40, 32, "e4m3", "f32")
    fill(c, m, [300], "f32", 8)
    Q = 40 * tokens(1, 5, 64, "f32", 9)
    for scale in (1.0, -0.5, 0.0):
        check_attention(c, m, Q, [0], [1], True, "f32", scale=scale)


CHUNKS = [
    # d, page, code, dtype, Hkv, G, lens, nq
    (128, 64, "int8", "bf16", 2, 4, [300, 64, 5, 129], [40, 64, 5, 1]),
    (128, 16, "e4m3", "f16", 1, 8, [257, 16], [100, 3]),
    (64, 32, "int8", "f16", 2, 1, [400, 1, 0, 90], [200, 1, 2, 90]),     # more queries than tokens: empty rows
    (256, 128, "e4m3", "bf16", 1, 3, [260, 130], [77, 130]),
    (256, 32, "int8", "f16", 1, 2, [200], [33]),
    (64, 16, "e4m3", "bf16", 1, 5, [333], [333]),
    (128, 128, "int8", "f32", 2, 2, [200, 30], [19, 30]),
    (64, 64, "e4m3", "f32", 1, 7, [150], [12]),
    (256, 64, "int8", "f32", 1, 1, [140], [70]),
]


@pytest.mark.parametrize("case", CHUNKS)
@pytest.mark.parametrize("causal", [True, False])
def test_chunk_and_cross(case, causal):
    d, page, code, dtype, Hkv, G, lens, nq = case
    c, m = make(Hkv, d, 100, len(lens), 40, page, code, dtype)
    fill(c, m, lens, dtype, 11)
    Q = tokens(sum(nq), Hkv * G, d, dtype, 12, 0.3)
    check_attention(c, m, Q, list(range(len(lens))), nq, causal, dtype, single_p=dtype != "f32")


def test_more_queries_than_tokens_causal():
    """Queries before the first token of a short sequence see nothing: 0 and -inf."""
    c, m = make(1, 128, 10, 1, 10, 64, "int8", "bf16")
    fill(c, m, [5], "bf16", 13)
    Q = tokens(200, 4, 128, "bf16", 14)
    got = check_attention(c, m, Q, [0], [200], True, "bf16", single_p=True)
    assert (got[:195] == 0).all()


def test_many_sequences():
    """More rows than the planning CTA has threads."""
    n = 1500
    c, m = make(1, 64, n + 10, n, 2, 16, "int8", "f16")
    counts = [1 + (7 * i) % 16 for i in range(n)]
    fill(c, m, counts, "f16", 15)
    same_tables(c, m)
    Q = tokens(n, 2, 64, "f16", 16)
    check_attention(c, m, Q, list(range(n)), [1] * n, True, "f16")


def test_layers_share_the_table():
    c, m = make(2, 64, 30, 3, 10, 32, "int8", "bf16", layers=3)
    fill(c, m, [40, 7, 33], "bf16", 17)
    fill(c, m, [1, 30], "bf16", 27, slots=[2, 1])
    Q = tokens(3, 4, 64, "bf16", 18)
    for l in range(3):
        same_values(c, m, "bf16", layer=l)
        check_attention(c, m, Q, [0, 1, 2], [1, 1, 1], True, "bf16", layer=l)


# ---------------------------------------------------------------------------- pages
@pytest.mark.parametrize("code,d,page", [("int8", 128, 64), ("e4m3", 64, 16), ("int8", 256, 128)])
def test_fork_copy_free_compact(code, d, page):
    c, m = make(2, d, 60, 12, 8, page, code, "bf16", layers=2)
    fill(c, m, [3 * page + 5, page, 1, 2 * page - 1], "bf16", 19)
    src, dst = [0, 0, 1, 3, 2], [4, 5, 6, 7, 8]
    c.fork(i32(src), i32(dst))
    for a, b in zip(src, dst):
        m.fork(a, b)
    same_tables(c, m)
    fill(c, m, [1, page, 2, 1, 1], "bf16", 29, slots=dst)          # the forks go their own ways
    same_tables(c, m)
    for l in range(2):
        same_values(c, m, "bf16", layer=l)
    c.copy(i32([5, 1]), i32([9, 10]))
    m.fork(5, 9, share=False)
    m.fork(1, 10, share=False)
    same_tables(c, m)
    c.free(i32([0, 5, 3, -1, 5]))                                   # a padding row, a slot twice
    for s in (0, 5, 3):
        m.free(s)
    same_tables(c, m)
    c.compact()
    m.compact()
    same_tables(c, m)
    fill(c, m, [1, 1], "bf16", 39, slots=[9, 4])                    # the tails moved along
    same_tables(c, m)
    for l in range(2):
        same_values(c, m, "bf16", layer=l)
    c.compact()                                                     # nothing left to move
    m.compact()
    same_tables(c, m)


def test_copy_to_another_cache():
    a, ma = make(1, 128, 20, 2, 10, 32, "e4m3", "f16")
    b, mb = make(1, 128, 30, 3, 8, 32, "e4m3", "f16")
    fill(a, ma, [70, 32], "f16", 41)
    fill(b, mb, [5], "f16", 42, slots=[1])
    a.copy(i32([0, 1]), i32([2, 0]), to=b)
    for s, t in ((0, 2), (1, 0)):
        mb.append(t, [tuple(x for x in ma.tok[s][0])])
    same_tables(b, mb)
    fill(b, mb, [3, 1], "f16", 43, slots=[2, 0])
    same_values(b, mb, "f16")
    same_tables(a, ma)


def test_a_run_together():
    """Prompts in, chunks and decode steps, a beam split, losers freed, the pool compacted,
    steps again: every output against the oracle."""
    c, m = make(2, 128, 40, 8, 6, 64, "int8", "bf16")
    fill(c, m, [150, 61], "bf16", 51)
    Q = tokens(211, 8, 128, "bf16", 52, 0.3)
    check_attention(c, m, Q, [0, 1], [150, 61], True, "bf16", single_p=True)
    live = [0, 1]
    for step in range(8):
        if step == 2:
            c.fork(i32([0, 1, 0]), i32([2, 3, 4]))
            for a, b in ((0, 2), (1, 3), (0, 4)):
                m.fork(a, b)
            live = [0, 1, 2, 3, 4]
        if step == 5:
            c.free(i32([0, 3]))
            m.free(0), m.free(3)
            c.compact()
            m.compact()
            live = [1, 2, 4]
        n = len(live)
        K, V, q = (tokens(n, h, 128, "bf16", 60 + 3 * step + j, 0.3) for j, h in enumerate((2, 2, 8)))
        out = c.decode_step(K, V, q, i32(live))
        for i, s in enumerate(live):
            m.append(s, [(host(K[i:i + 1]), host(V[i:i + 1]))])
        assert torch.equal(out, check_attention(c, m, q, live, [1] * n, True, "bf16"))
        same_tables(c, m)
    enc = tokens(30, 8, 128, "bf16", 99, 0.3)                       # and as an encoder's states
    check_attention(c, m, enc, [4, 1], [10, 20], False, "bf16", single_p=True)


# ---------------------------------------------------------------------------- refusals
def test_device_refusals_leave_the_cache_alone():
    from compressed_attention_turboquantprod_b200 import TQError
    n = nat()
    c, m = make(1, 64, 6, 4, 4, 16, "int8", "f16")
    fill(c, m, [20, 16], "f16", 71)
    K = tokens(80, 1, 64, "f16", 72)

    def refused(status, call):
        call()
        with pytest.raises(TQError) as e:
            c.check()
        assert e.value.status == status
        same_tables(c, m)                  # and the status was cleared
        same_values(c, m, "f16")

    def append(rows, cu):
        return lambda: c.append(K, K, i32(rows), i32(cu))
    refused(n.TQ_ERR_CAPACITY, append([2], [0, 64]))                  # 4 pages, 3 are free
    refused(n.TQ_ERR_CAPACITY, append([0], [0, 60]))                  # 5 pages of at most 4
    refused(n.TQ_ERR_INVALID_ARG, append([2, 2], [0, 1, 2]))          # a slot twice
    refused(n.TQ_ERR_INVALID_ARG, append([4], [0, 1]))
    refused(n.TQ_ERR_INVALID_ARG, append([-2], [0, 1]))
    refused(n.TQ_ERR_INVALID_ARG, append([2, 3], [0, 5, 3]))          # offsets decrease
    refused(n.TQ_ERR_INVALID_ARG, append([2], [-1, 3]))
    refused(n.TQ_ERR_INVALID_ARG, lambda: c.fork(i32([0]), i32([1])))         # not empty
    refused(n.TQ_ERR_INVALID_ARG, lambda: c.fork(i32([0, 1]), i32([2, 2])))
    refused(n.TQ_ERR_INVALID_ARG, lambda: c.fork(i32([0, 2]), i32([2, 3])))   # a destination as a source
    refused(n.TQ_ERR_INVALID_ARG, lambda: c.fork(i32([0]), i32([9])))
    refused(n.TQ_ERR_INVALID_ARG, lambda: c.free(i32([7])))
    refused(n.TQ_ERR_CAPACITY, lambda: c.copy(i32([0, 0]), i32([2, 3])))      # 4 pages, 3 free
    # offsets past the tokens given: the row exists, its missing tokens are not written
    c.append(K[:3], K[:3], i32([3]), i32([0, 9]))
    with pytest.raises(TQError):
        c.check()


def test_workspace_not_made_ready():
    from compressed_attention_turboquantprod_b200 import TQError
    c, m = make(1, 64, 6, 2, 4, 16, "int8", "f16")
    fill(c, m, [20], "f16", 73)
    Q = tokens(1, 2, 64, "f16", 74)
    ws = torch.full_like(c.make_workspace(), 5)
    c.attend(Q, i32([0]), i32([0, 1]), 1, workspace=ws)
    with pytest.raises(TQError):
        c.check()
    check_attention(c, m, Q, [0], [1], True, "f16")


def test_a_row_longer_than_max_q_is_reported():
    from compressed_attention_turboquantprod_b200 import TQError
    c, m = make(1, 64, 6, 2, 4, 16, "int8", "f16")
    fill(c, m, [20], "f16", 75)
    c.attend(tokens(40, 2, 64, "f16", 76), i32([0]), i32([0, 40]), 1)
    with pytest.raises(TQError):
        c.check()


# ---------------------------------------------------------------------------- graphs, streams
def test_captured_steps_replay():
    """Decode steps with growing lengths and a page taken on the way, replayed from one graph;
    two graphs of attention on the same cache replayed in turn."""
    c, m = make(2, 128, 20, 3, 8, 16, "int8", "bf16")
    fill(c, m, [30, 14, 47], "bf16", 81)
    rows, cu = i32([0, 1, 2]), offsets([1, 1, 1])
    K, V, q = (tokens(3, h, 128, "bf16", 82 + h, 0.3) for h in (2, 2, 8))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = c.decode_step(K, V, q, rows, cu)
    torch.cuda.current_stream().wait_stream(side)
    for i in range(3):
        m.append(i, [(host(K[i:i + 1]), host(V[i:i + 1]))])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = c.decode_step(K, V, q, rows, cu)
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):
        out2 = c.decode(q, rows, cu=cu)
    for step in range(20):
        for t, s in ((K, 200), (V, 300), (q, 400)):
            t.copy_(tokens(3, t.shape[1], 128, "bf16", s + step, 0.3))
        g.replay()
        g2.replay()
        for i in range(3):
            m.append(i, [(host(K[i:i + 1]), host(V[i:i + 1]))])
        assert torch.equal(out, out2)
        assert torch.equal(out, check_attention(c, m, q, [0, 1, 2], [1, 1, 1], True, "bf16"))
    same_tables(c, m)
    same_values(c, m, "bf16")


def test_two_streams_read_one_cache():
    c, m = make(2, 128, 80, 2, 40, 64, "int8", "bf16")
    fill(c, m, [2000, 555], "bf16", 91)
    q = [tokens(2, 8, 128, "bf16", 92 + i, 0.3) for i in range(2)]
    want = [check_attention(c, m, x, [0, 1], [1, 1], True, "bf16") for x in q]
    rows, cu = i32([0, 1]), offsets([1, 1])
    st = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(st[i]):
                got[i].append(c.decode(q[i], rows, cu=cu))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert torch.equal(g, want[i])


def test_results_repeat_bit_for_bit():
    c, m = make(2, 128, 200, 3, 100, 64, "e4m3", "bf16")
    fill(c, m, [5000, 333, 1], "bf16", 95)
    q = tokens(3, 8, 128, "bf16", 96, 0.3)
    first = check_attention(c, m, q, [0, 1, 2], [1, 1, 1], True, "bf16")
    Q = tokens(150, 8, 128, "bf16", 97, 0.3)
    f2 = c.attend(Q, i32([0, 1]), offsets([100, 50]), 100)
    for _ in range(5):
        assert torch.equal(first, c.decode(q, i32([0, 1, 2])))
        assert torch.equal(f2, c.attend(Q, i32([0, 1]), offsets([100, 50]), 100))


def test_few_rows_of_a_chunk_many_times():
    """Warps without rows run ahead of those with rows: one row block, several tiles, again and again."""
    c, m = make(2, 128, 40, 2, 20, 64, "int8", "bf16")
    fill(c, m, [700, 65], "bf16", 101)
    Q = tokens(30, 8, 128, "bf16", 102, 0.3)
    first = check_attention(c, m, Q, [0, 1], [10, 20], False, "bf16", single_p=True)
    rows, cu = i32([0, 1]), offsets([10, 20])
    for _ in range(200):
        assert torch.equal(first, c.cross(Q, rows, cu, 20))


@pytest.mark.parametrize("scale", [-0.3, 0.0])
def test_chunk_with_a_negative_and_a_zero_scale(scale):
    c, m = make(1, 64, 20, 1, 20, 32, "int8", "bf16")
    fill(c, m, [150], "bf16", 111)
    Q = tokens(40, 4, 64, "bf16", 112, 0.3)
    check_attention(c, m, Q, [0], [40], True, "bf16", scale=scale, single_p=True)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (256, 128)])
def test_what_a_page_held_before_does_not_show(code, d, page):
    """Pages of freed sequences with entries near the type's largest, infinities and NaN are taken by
    short ones: the places behind a sequence's end hold those codes still."""
    c, m = make(1, d, 8, 2, 8, page, code, "bf16")
    big = tokens(8 * page, 1, d, "bf16", 121) * 1e36
    big[::7] = float("inf")
    big[3::11] = float("nan")
    c.append(big, big, i32([0]), offsets([8 * page]))
    c.free(i32([0]))
    fill(c, m, [page // 2 + 1, 1], "bf16", 122)
    same_values(c, m, "bf16")
    Q = tokens(2, 3, d, "bf16", 123, 0.3)
    check_attention(c, m, Q, [0, 1], [1, 1], True, "bf16")
    Q = tokens(41, 3, d, "bf16", 124, 0.3)
    check_attention(c, m, Q, [0, 1], [40, 1], False, "bf16", single_p=True)


def test_offsets_past_32_bits():
    """A pool of more than 4 GB: the last layer's pages lie past 2^32 bytes."""
    c, m = make(8, 128, 700, 2, 10, 64, "int8", "bf16", layers=56)
    assert c.state.o_pool + 55 * 700 * c.state.page_bytes > 2 ** 32
    counts = [130, 3]
    c.extend(i32([0, 1]), offsets(counts))
    K, V = tokens(133, 8, 128, "bf16", 131), tokens(133, 8, 128, "bf16", 132)
    c.write(K, V, layer=55)
    k, v = (op.cached_values(host(t[:130]), "int8", 64) for t in (K, V))
    rk, rv = c.read(i32([0]), offsets([130]), 130, layer=55)
    for got, want in ((rk, k), (rv, v)):
        assert (np.abs(host(got) - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -23) + 1e-30).all()
    assert (c.read(i32([0]), offsets([130]), 130, layer=54)[0] == 0).all()
    Q = tokens(41, 16, 128, "bf16", 133, 0.3)
    want, _, mass, reach = op.attention(host(Q), k, v, True, 128 ** -0.5)
    for got, lo, p_step in ((c.attend(Q, i32([0]), offsets([41]), 41, layer=55), 0, 2.0 ** -11),
                            (c.decode(Q[40:].contiguous(), i32([0]), layer=55), 40, 0.0)):
        ew = (2 * (128 + 8) * 2.0 ** -24 * reach[lo:] + 2.0 ** -19 + p_step)[..., None] * mass[lo:]
        tol = 2.0 ** -36 * 130 * np.abs(v).max() + ew + 2.0 ** -8 * (np.abs(want[lo:]) + ew)
        assert (np.abs(host(got) - want[lo:]) <= tol).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("G,nq", [(8, 3), (4, 5), (1, 24), (5, 4), (1, 25), (8, 4)])
def test_few_queries_on_either_side_of_the_rule(dtype, G, nq):
    """9 to 32 query rows of a KV head: several groups of 8 rows, a group that holds rows of two queries."""
    c, m = make(2, 128, 60, 2, 30, 32, "e4m3", dtype)
    fill(c, m, [500, nq + 1], dtype, 141)
    Q = tokens(2 * nq, 2 * G, 128, dtype, 142, 0.3)
    check_attention(c, m, Q, [0, 1], [nq, nq], True, dtype, single_p=nq * G > 24)


def test_the_largest_batch_and_pool():
    """65536 sequences in a pool of 2^20 pages: plans over many rounds, a compaction of the whole pool."""
    n = 65536
    c, _ = make(1, 64, 1 << 20, n, 4, 16, "int8", "f16")
    rows = torch.arange(n, dtype=torch.int32, device="cuda")
    counts = rows % 37
    cu = torch.cat([counts.new_zeros(1), counts.cumsum(0).int()])
    total = int(cu[-1])
    x = tokens(total, 1, 64, "f16", 151)
    c.append(x, x, rows, cu)
    assert torch.equal(c.lengths, counts)
    used = (counts + 15) // 16
    table = c.page_table(rows)
    have = torch.arange(4, device="cuda") < used[:, None]
    assert torch.equal(table[have], torch.arange(int(used.sum()), dtype=torch.int32, device="cuda"))
    assert (table[~have] == -1).all()
    K, _ = c.read(rows, cu, total)
    err = (K.float() - x.float()).abs()                  # at most half a step of the block's scale, and the type's
    assert float((err - x.float().abs().max() / 254 - x.float().abs() * 2.0 ** -11).max()) <= 0
    c.free(rows[: n // 2])
    c.compact()
    live = int(used[n // 2:].sum())
    assert c.check() == (1 << 20) - live
    table = c.page_table(rows)[n // 2:]
    got = table[have[n // 2:]]
    assert torch.equal(got.sort().values, torch.arange(live, dtype=torch.int32, device="cuda"))
    again, _ = c.read(rows[n // 2:], cu[n // 2:] - cu[n // 2], total - int(cu[n // 2]))
    assert torch.equal(again, K[int(cu[n // 2]):])
    q = tokens(n // 2, 2, 64, "f16", 152)
    out = c.decode(q, rows[n // 2:])
    assert torch.isfinite(out.float()).all() and (out[counts[n // 2:] == 0] == 0).all()
    one = counts[n // 2:] == 1                           # a single token: its value, rounded once more at most
    at = (cu[n // 2:-1] - cu[n // 2])[one].long()
    v = again[at][:, 0].float()                          # (K and V got the same tokens)
    assert ((out[one].float() - v[:, None]).abs() <= 2.0 ** -10 * v.abs()[:, None] + 2.0 ** -24).all()
