"""Small ragged runs of every paged path, in a child process of test_gpu_paged_bounds.py with either
library; writes outputs to an .npz file and, for the bounds-checked build, asserts that no device check
fired.

usage: python tests/paged_bounds_cases.py OUT.npz
"""
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from compressed_attention_turboquantprod_b200 import PagedKVCache, native  # noqa: E402

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

CASES = [  # d, page, code, dtype, Hkv, G, lengths, queries per sequence
    (128, 64, "int8", "bf16", 2, 4, [300, 64, 5, 0], [70, 64, 5, 2]),
    (64, 16, "e4m3", "f16", 3, 1, [33, 400, 1], [33, 150, 1]),
    (256, 128, "int8", "bf16", 1, 3, [260, 129], [77, 129]),
    (256, 32, "e4m3", "f32", 1, 2, [90, 31], [11, 3]),
    (64, 128, "int8", "f32", 2, 5, [200, 128], [7, 1]),
]


def run(path):
    res = {}
    for k, (d, page, code, dtype, Hkv, G, lens, nq) in enumerate(CASES):
        g = torch.Generator(device="cuda")
        g.manual_seed(k)

        def rand(n, h):
            return torch.randn(n, h, d, generator=g, device="cuda").to(DT[dtype])

        def i32(x):
            return torch.tensor(list(x), dtype=torch.int32, device="cuda")

        def off(x):
            return i32(np.cumsum([0] + list(x)))
        n = len(lens)
        # the pool holds just what the run needs at most, so that a stray page would leave it
        pages = 3 * sum(-(-x // page) for x in lens) + 2 * n
        c = PagedKVCache(Hkv, d, pages, 3 * n, max(-(-x // page) for x in lens) + 1, page=page, code=code,
                         dtype=DT[dtype], layers=2)
        a, b = range(n), range(n, 2 * n)
        c.extend(i32(a), off(lens))
        for l in range(2):
            c.write(rand(sum(lens), Hkv), rand(sum(lens), Hkv), layer=l)
        Q = rand(sum(nq), Hkv * G)
        for causal in (True, False):
            lse = torch.zeros(sum(nq), Hkv * G, device="cuda")
            o = c.attend(Q, i32(a), off(nq), max(nq), causal, layer=1, lse=lse)
            res[f"{k}_attend_{causal}"], res[f"{k}_lse_{causal}"] = o.float().cpu().numpy(), lse.cpu().numpy()
        c.fork(i32(a), i32(b))
        c.extend(i32(b), off([1] * n))
        for l in range(2):
            c.write(rand(n, Hkv), rand(n, Hkv), layer=l)
        res[f"{k}_decode"] = c.decode(rand(n, Hkv * G), i32(b)).float().cpu().numpy()
        c.copy(i32(b), i32(range(2 * n, 3 * n)))
        c.free(i32(a))
        c.compact()
        total = sum(lens) + n
        K, V = c.read(i32(range(2 * n, 3 * n)), off([x + 1 for x in lens]), total, layer=1)
        res[f"{k}_K"], res[f"{k}_V"] = K.float().cpu().numpy(), V.float().cpu().numpy()
        res[f"{k}_table"] = c.page_table(i32(range(3 * n))).cpu().numpy()
        res[f"{k}_free"] = np.array([c.check()])
    enabled = native.lib.tq_debug_bounds_enabled()
    native.tq_debug_bounds_check()          # raises TQError if any device check fired
    res["bounds_enabled"] = np.array([enabled])
    np.savez(path, **res)


if __name__ == "__main__":
    run(sys.argv[1])
