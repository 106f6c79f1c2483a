"""Forks and releases of a large pool inside a captured graph."""
import numpy as np
import pytest
import torch

import paged_kv_cache_233_gb300 as pk
from test_gpu_pages import ALL, Cache, gpu  # noqa: F401  (gpu: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,length,width", [(3, 100000, 12600), (600, 1000, 130)])
def test_a_captured_release_of_a_large_pool(rows, length, width):
    """More than 32768 blocks, so that the push is a cluster's: step after step of a replayed
    fork and release in place, first of a pool's stack and table as they are, then as the
    steps left them."""
    block, rng = 8, np.random.default_rng(rows)
    c = Cache([length] * rows + [0] * rows, block, width, 40000, rows)
    assert c.blocks > 1 << 15
    d = c.device()
    S = 2 * rows
    dev = dict(dtype=torch.int32, device="cuda")
    parents, keep, pairs = torch.full((S,), -1, **dev), torch.full((S,), ALL, **dev), torch.zeros(S, 2, **dev)

    def step():
        pk.paged_kv_fork(parents, d["lens"], d["tables"], d["shared"], d["free"], d["count"], pairs, block)
        pk.paged_kv_release(keep, d["lens"], d["tables"], d["shared"], d["free"], d["count"], block)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):        # (captured first: what the launches ask of the host comes with it)
        step()
    for i in range(6):
        empty = [s for s in range(S) if c.lens[s] == 0]
        full = [s for s in range(S) if c.lens[s] > 0]
        of = [-1] * S
        for s in empty[:: 1 + i % 3]:
            if full:
                of[s] = int(rng.choice(full))
        want = c.fork(of)
        fate = rng.integers(0, 5, S)
        drop = [0 if f == 0 and s % 3 else max(0, n - int(rng.integers(0, 300))) if f == 1 else ALL
                for s, (f, n) in enumerate(zip(fate, c.lens))]
        parents.copy_(torch.tensor(of, dtype=torch.int32))
        keep.copy_(torch.tensor(drop, dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        c.release(drop)
        c.check(d, d["lens"], d["count"], pairs, want)
    assert pk.device_errors() == 0
