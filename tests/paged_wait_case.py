"""A decode whose copies never come, in a child process of test_gpu_paged_waits.py with the bounds-checked
library: its waits run out, the status says so, and cache, workspace and later calls are none the worse.

usage: python tests/paged_wait_case.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from compressed_attention_turboquantprod_b200 import PagedKVCache, TQError, native  # noqa: E402


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def main():
    g = torch.Generator(device="cuda").manual_seed(1)
    for d, page, lens in ((128, 64, [900, 3]), (64, 16, [4000, 70]), (256, 32, [33, 1])):
        c = PagedKVCache(2, d, 300, 2, 260, page=page)
        total = sum(lens)
        K, V = (torch.randn(total, 2, d, generator=g, device="cuda").bfloat16() for _ in range(2))
        rows = i32([0, 1])
        c.append(K, V, rows, i32([0, lens[0], total]))
        Q = torch.randn(2, 8, d, generator=g, device="cuda").bfloat16()
        want = c.decode(Q, rows)
        c.check()
        native.tq_debug_paged_lose_copies(True)
        try:
            c.decode(Q, rows)
            try:
                c.check()
                raise SystemExit("the check found nothing")
            except TQError as e:
                assert e.status == native.TQ_ERR_CUDA and "gave up" in e.message, e
        finally:
            native.tq_debug_paged_lose_copies(False)
        assert torch.equal(c.decode(Q, rows), want)
        c.check()
        native.tq_debug_bounds_check()
    print("waits ran out and were reported")


if __name__ == "__main__":
    main()
