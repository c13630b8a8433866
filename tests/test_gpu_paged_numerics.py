"""What the paged cache's attention must not lose: long sums, value scales far apart (a block of zeros
among them), queries that are not finite, and what a mask hides.

The bounds are those of test_gpu_paged.py, taken over what a query sees: with p at most 1 against the
running maximum and b a visible block's largest |v|, a half keeps p b off by at most 2^-36 (chunks of bf16
and f16, against the largest p b in sight) or 2^-40 (decode, against the largest b in sight)."""
import math

import numpy as np
import pytest
import torch

from gpu_common import TORCH_DT, host
from oracle import paged as op
from test_gpu_paged import HALF, TINY, i32, make, offsets, tokens

pytestmark = pytest.mark.gpu


def reference(q, k, v, b, vis, scale):
    """One query [d] over its first `vis` tokens of one head, in float64; b: the largest |v| of each
    token's block.  (out, lse, sum p |v|, largest scale sum |q k|, largest p b, largest b)."""
    s = scale * (k[:vis] @ q)
    m = s.max()
    p = np.exp(s - m)
    l = p.sum()
    reach = (abs(scale) * (np.abs(k[:vis]) @ np.abs(q))).max()
    return p @ v[:vis] / l, m + math.log(l), p @ np.abs(v[:vis]) / l, reach, (p * b[:vis]).max() / l, b[:vis].max() / l


def check(c, page, K, V, Q, causal, dtype, scale=None, single_p=True, code="int8"):
    """Q over slot 0, which holds K and V, against the oracle; returns the output."""
    n, Hq, d = Q.shape
    Hkv, T, G = K.shape[1], K.shape[0], Hq // K.shape[1]
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    lse = torch.full((n, Hq), 7.0, device="cuda")
    got = c.attend(Q, i32([0]), offsets([n]), n, causal, sc, lse=lse)
    c.check()
    k, v = (op.cached_values(host(t), code, page) for t in (K, V))
    b = np.zeros((T, Hkv))
    for t in range(0, T, page):
        b[t:t + page] = np.abs(v[t:t + page]).max(axis=(0, 2))
    q64, g64, l64 = host(Q), host(got), lse.cpu().double().numpy()
    for i in range(n):
        vis = max(0, min(T, T - n + i + 1)) if causal else T
        for h in range(Hq):
            if vis == 0:
                assert (g64[i, h] == 0).all() and np.isneginf(l64[i, h])
                continue
            want, wl, mass, reach, pb, bb = reference(q64[i, h], k[:, h // G], v[:, h // G], b[:, h // G], vis, sc)
            ew = 2 * (d + 8) * 2.0 ** -24 * reach + 2.0 ** -19 + (2.0 ** -11 if single_p else 0.0)
            floor = vis * (2.0 ** -36 * pb if single_p else 2.0 ** -40 * bb)
            tol = floor + ew * mass + HALF[dtype] * (np.abs(want) + ew * mass) + TINY[dtype]
            err = np.abs(g64[i, h] - want)
            assert (err <= tol).all(), (i, h, vis, float((err / tol).max()), float(err.max()))
            assert abs(l64[i, h] - wl) <= ew + 2.0 ** -22 * (1 + abs(wl)), (i, h, l64[i, h], wl)
    return got


@pytest.mark.parametrize("d,G,rows", [(64, 1, 148), (64, 1, 100), (128, 8, 148), (256, 2, 148)])
def test_chunk_sums_of_a_long_sequence(d, G, rows):
    """Values around 1 over 400001 tokens: a sum that always rounds the same way would drift by 2^-24 of
    itself a step of 16 tokens (25000 of them).  Many rows name the one sequence, so that a CTA sums most
    or all of it.  Bound: p's rounding (2^-11), at most 512 steps that truncate (2^-23 each) before they are
    folded, a rounding for each of the folds (2^-24, at most 400) and for each joined part."""
    T, n, page = 400001, 26, 64
    c, _ = make(1, d, T // page + 2, 1, T // page + 1, page, "int8", "f16")
    g = torch.Generator().manual_seed(7)
    K = torch.randn(T, 1, d, generator=g).half()
    V = (1.0 + 0.25 * torch.randn(T, 1, d, generator=g)).half()
    c.append(K.cuda(), V.cuda(), i32([0]), offsets([T]))
    Q = tokens(n, G, d, "f16", 8, 0.3)
    got = c.cross(Q.repeat(rows, 1, 1), i32([0] * rows), offsets([n] * rows), n)
    c.check()
    k, v = (torch.from_numpy(op.cached_values(host(t), "int8", page)).cuda()[:, 0] for t in (K, V))
    q = Q.double().reshape(n * G, d)
    p = torch.softmax(q @ k.T / math.sqrt(d), -1)
    want, mass = p @ v, p @ v.abs()
    reach = (q.abs() @ k.abs().T).max() / math.sqrt(d)
    ew = float(2 * (d + 8) * 2.0 ** -24 * reach + 2.0 ** -19 + 2.0 ** -11 + 512 * 2.0 ** -23 + 410 * 2.0 ** -24)
    tol = ew * mass + 2.0 ** -11 * (want.abs() + ew * mass)
    err = (got.double().reshape(rows, n * G, d) - want).abs()
    assert float((err / tol).max()) <= 1, (float((err / tol).max()), float(err.max()))


@pytest.mark.parametrize("where", ["before", "between", "after", "all"])
@pytest.mark.parametrize("d,page,code", [(64, 16, "int8"), (128, 64, "e4m3"), (256, 128, "int8"), (128, 32, "int8")])
@pytest.mark.parametrize("size", [1.0, 1e-4, 1e-8])
def test_chunk_with_blocks_of_zero_values(where, d, page, code, size):
    """Padding tokens with values of zero: they take their weight and nothing else."""
    T = 4 * page + 150
    K, V = tokens(T, 1, d, "bf16", 11), size * tokens(T, 1, d, "bf16", 12)
    lo, hi = {"before": (0, 2 * page), "between": (page, 3 * page), "after": (3 * page, T), "all": (0, T)}[where]
    V[lo:hi] = 0
    c, _ = make(1, d, 40, 1, 40, page, code, "bf16")
    c.append(K, V, i32([0]), offsets([T]))
    for causal in (True, False):
        check(c, page, K, V, tokens(33, 3, d, "bf16", 13, 0.3), causal, "bf16", code=code)


@pytest.mark.parametrize("page", [16, 64])
def test_chunk_with_value_scales_far_apart(page):
    """Pages 2^40 apart, as the decode takes them; causal rows that see the small ones only."""
    T = 700
    K, V = tokens(T, 1, 128, "bf16", 21), tokens(T, 1, 128, "bf16", 22)
    V[128:192] *= 2.0 ** -20
    V[640:] *= 2.0 ** 20
    K[256:320] *= 2.0 ** -20
    c, _ = make(1, 128, 60, 1, 60, page, "int8", "bf16")
    c.append(K, V, i32([0]), offsets([T]))
    check(c, page, K, V, tokens(100, 2, 128, "bf16", 23, 0.3), True, "bf16")
    check(c, page, K, V, tokens(30, 2, 128, "bf16", 24, 0.3), False, "bf16")


@pytest.mark.parametrize("order", [(120, -95), (-95, 120), (0, 120), (120, 0), (0, -95), (-95, 0), (-95, -95)])
@pytest.mark.parametrize("heavy", [False, True])
@pytest.mark.parametrize("split", [False, True])
def test_chunk_over_the_whole_range_of_value_scales(order, heavy, split):
    """Values of 2^a in the first pages and 2^b in the last, zeros between; heavy: the larger ones get no
    weight (logits 300 below), so that the smaller ones decide the output.  split: over several CTAs."""
    page, d = 64, 64
    T = (40 if split else 6) * page
    third = T // 3 // page * page
    K, V = tokens(T, 1, d, "bf16", 31, 0.1), tokens(T, 1, d, "bf16", 32, 0.1)
    V = V.clamp(-8, 8)
    V[:third] *= 2.0 ** order[0]
    V[third:2 * third] = 0
    V[2 * third:] *= 2.0 ** order[1]
    Q = tokens(50, 1, d, "bf16", 33, 0.1)
    if heavy:
        big = slice(0, third) if order[0] > order[1] else slice(2 * third, T)
        K[..., 0], Q[..., 0] = 0, 8
        K[big][..., 0] = -300.0
    c, _ = make(1, d, 50, 1, 50, page, "int8", "bf16")
    c.append(K, V, i32([0]), offsets([T]))
    check(c, page, K, V, Q, False, "bf16", scale=0.125)
    check(c, page, K, V, Q, True, "bf16", scale=0.125)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [2, 40])
@pytest.mark.parametrize("T", [100, 6000])
def test_queries_that_are_not_finite(dtype, n, T):
    """A NaN or an infinity in a query gives NaN in that query's output and lse and nowhere else, in
    both kernels and in units of one CTA (100 tokens) or of several (6000); a query that sees nothing gives 0."""
    c, _ = make(1, 64, 120, 2, 100, 64, "int8", dtype)
    c.append(tokens(T, 1, 64, dtype, 41), tokens(T, 1, 64, dtype, 42), i32([0]), offsets([T]))
    Q = tokens(2 * n, 2, 64, dtype, 43, 0.3)
    rows, cu = i32([0, 1]), offsets([n, n])            # slot 1 is empty
    lse = [torch.zeros(2 * n, 2, device="cuda") for _ in range(2)]
    good = c.cross(Q, rows, cu, n, lse=lse[0])
    for value in (float("nan"), float("inf"), float("-inf")):
        bad = Q.clone()
        bad[0, 1, 5] = value
        bad[n - 1, 0, :] = value
        bad[n, 0, 3] = value
        out = c.cross(bad, rows, cu, n, lse=lse[1])
        hit = torch.zeros(2 * n, 2, dtype=torch.bool, device="cuda")
        hit[0, 1] = hit[n - 1, 0] = True
        assert torch.isnan(out[hit]).all() and torch.isnan(lse[1][hit]).all()
        assert torch.equal(out[~hit], good[~hit]) and torch.equal(lse[1][~hit], lse[0][~hit])
        assert (out[n:] == 0).all() and torch.isneginf(lse[1][n:]).all()
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page", [16, 32])
def test_what_a_mask_hides_does_not_coarsen_the_rest(dtype, page):
    """Two queries over a page of values near 1e-8 and a token of 1e8 behind it, which only the last one sees."""
    T = page + 1
    K, V = tokens(T, 1, 64, dtype, 51), 1e-8 * tokens(T, 1, 64, dtype, 52)
    V[page] = 1e8
    c, _ = make(1, 64, 8, 1, 8, page, "int8", dtype)
    c.append(K, V, i32([0]), offsets([T]))
    check(c, page, K, V, tokens(2, 2, 64, dtype, 53, 0.3), True, dtype, single_p=False)


