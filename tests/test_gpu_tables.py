"""paged_kv_build_tables against a request-by-request walk on the host."""
import numpy as np
import pytest
import torch

import paged_kv_cache_233_gb300 as pk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pk.load()
    torch.cuda.set_device(0)
    pk.device_errors()


def walk(new, ctx, tables, free, count, block, cap):
    """The definition, one request at a time."""
    tables = tables.copy()
    width = tables.shape[1]
    asked_blocks = asked_tokens = taken = 0
    lens, starts, seq, pos, slot = [], [0], [], [], []
    for s in range(len(new)):
        n, c = int(new[s]), int(ctx[s])
        ok = n >= 0 and c >= 0 and c + n <= width * block
        if ok:
            need = -(-(c + n) // block) - -(-c // block)
            asked_blocks += need
            asked_tokens += n
            ok = (need == 0 or asked_blocks <= count) and (n == 0 or asked_tokens <= cap)
        if ok:
            for j in range(need):
                tables[s, -(-c // block) + j] = free[count - 1 - taken]
                taken += 1
            for i in range(c, c + n):
                seq.append(s)
                pos.append(i)
                slot.append(int(tables[s, i // block]) * block + i % block)
        starts.append(len(seq))
        lens.append(c + n if ok else c)
    pad = cap - len(seq)
    return tables, lens, count - taken, starts, seq + [0] * pad, pos + [-1] * pad, slot + [-1] * pad


def make(S, block, seed, longest, chunk, extra_width=3, spare=1.0):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, longest + 1, S)
    new = np.where(rng.random(S) < 0.3, rng.integers(0, chunk + 1, S), 1)
    held = -(-ctx // block)
    width = int((longest + chunk) // block) + extra_width
    total = int(held.sum() + spare * (-(-(ctx + new) // block) - held).sum()) + 2
    ids = rng.permutation(total).astype(np.int32)
    tables = np.full((S, width), -1, np.int32)
    at = 0
    for s in range(S):
        tables[s, :held[s]] = ids[at:at + held[s]]
        at += held[s]
    return new.astype(np.int32), ctx.astype(np.int32), tables, ids[at:].copy(), total


def call(new, ctx, tables, free, count, block, blocks, cap, in_place=False, slots=True):
    t = lambda x: torch.tensor(np.asarray(x, np.int32)).cuda()  # noqa: E731
    a = dict(new=t(new), ctx=t(ctx), tables=t(tables), free=t(free), count=t([count]))
    o = dict(starts=t([-9] * (len(new) + 1)), seq=t([-9] * cap), pos=t([-9] * cap),
             slots=torch.full((cap,), -9, dtype=torch.int64).cuda() if slots else None,
             ctx_out=a["ctx"] if in_place else t([-9] * len(new)), count_out=a["count"] if in_place else t([-9]))
    pk.paged_kv_build_tables(a["new"], a["ctx"], a["tables"], a["free"], a["count"], block, blocks, o["starts"], o["seq"],
                             o["pos"], o["slots"], o["ctx_out"], o["count_out"])
    return (a["tables"].cpu().numpy(), o["ctx_out"].tolist(), int(o["count_out"]), o["starts"].tolist(), o["seq"].tolist(),
            o["pos"].tolist(), o["slots"].tolist() if slots else None)


def same(got, want):
    assert np.array_equal(got[0], want[0])
    for g, w in zip(got[1:], want[1:]):
        assert g is None or g == w


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("S,block,longest,chunk", [(1, 16, 40, 40), (3, 1, 5, 9), (33, 8, 100, 30), (257, 16, 500, 1),
                                                   (1000, 32, 90, 200), (1025, 7, 300, 50), (4096, 16, 64, 40)])
def test_tables(S, block, longest, chunk, in_place):
    new, ctx, tables, free, blocks = make(S, block, S, longest, chunk)
    cap = int(new.sum()) + S % 5
    want = walk(new, ctx, tables, free, len(free), block, cap)
    same(call(new, ctx, tables, free, len(free), block, blocks, cap, in_place), want)
    assert pk.device_errors() == 0
    assert want[3][-1] == new.sum()               # everything was granted


@pytest.mark.parametrize("S", [5, 130, 2000])
@pytest.mark.parametrize("short", ["blocks", "tokens", "both", "none left"])
def test_requests_wait_when_it_runs_short(S, short):
    new, ctx, tables, free, blocks = make(S, 16, S + 1, 200, 60)
    count = {"blocks": len(free) // 2, "tokens": len(free), "both": len(free) // 3, "none left": 0}[short]
    cap = int(new.sum()) // 2 if short in ("tokens", "both") else int(new.sum())
    want = walk(new, ctx, tables, free, count, 16, cap)
    same(call(new, ctx, tables, free, count, 16, blocks, cap), want)
    assert pk.device_errors() == 0


def test_nothing_to_do():
    empty = np.zeros((0, 4), np.int32)
    same(call([], [], empty, [], 0, 16, 8, 5), (empty, [], 0, [0], [0] * 5, [-1] * 5, [-1] * 5))
    new, ctx, tables, free, blocks = make(7, 16, 1, 50, 9)
    same(call(new * 0, ctx, tables, free, len(free), 16, blocks, 0), walk(new * 0, ctx, tables, free, len(free), 16, 0))
    same(call(new, ctx, tables, free, len(free), 16, blocks, 0), walk(new, ctx, tables, free, len(free), 16, 0))
    same(call(new, ctx, tables, free, len(free), 16, blocks, 40, slots=False),
         walk(new, ctx, tables, free, len(free), 16, 40))
    assert pk.device_errors() == 0


def test_bad_lengths_and_blocks_are_reported():
    new, ctx, tables, free, blocks = make(6, 16, 2, 50, 9)
    new[1], ctx[2], new[4] = -1, -5, 2 ** 31 - 1
    cap = 80
    got = call(new, ctx, tables, free, len(free), 16, blocks, cap)
    same(got, walk(new, ctx, tables, free, len(free), 16, cap))
    assert pk.device_errors() == 4 | 8            # CONTEXT_LEN, POSITION
    # ids outside the pool: the token has no slot
    new, ctx, tables, free, blocks = make(3, 16, 3, 50, 9)
    new[:], ctx[:] = [1, 1, 20], [3, 16, 0]
    free, blocks = np.concatenate([free, np.arange(blocks, blocks + 5, dtype=np.int32)]), blocks + 5
    tables[0, 0] = blocks + 5
    free[-1] = -3
    got = call(new, ctx, tables, free, len(free), 16, blocks, 30)
    assert pk.device_errors() == 2                # BLOCK_ID
    assert got[6][:2] == [-1, -1] and min(got[6][2:22]) >= 0
    # a count that is no count is taken as its nearest
    got = call(new, ctx, tables, free, len(free) + 9, 16, blocks, 30)
    assert pk.device_errors() == 2 | 8
    assert got[2] == len(free) - 3


def test_totals_past_32_bits_are_refused_not_wrapped():
    S, block = 4096, 1 << 20
    new = np.full(S, 1 << 20, np.int32)           # 2^32 tokens asked for in all
    ctx = np.zeros(S, np.int32)
    tables = np.full((S, 2), -1, np.int32)
    free = np.arange(S, dtype=np.int32)
    cap = (1 << 20) + 5
    got = call(new, ctx, tables, free, S, block, S, cap)
    assert got[3] == [0] + [1 << 20] * S          # the first request alone
    assert got[2] == S - 1 and got[1][:2] == [1 << 20, 0]
    assert pk.device_errors() == 0


def test_side_stream_and_graph_evolve_the_state():
    new, ctx, tables, free, blocks = make(40, 16, 9, 60, 1, extra_width=9, spare=1)
    free = np.concatenate([free, np.arange(blocks, blocks + 200, dtype=np.int32)])
    blocks += 200
    t = lambda x: torch.tensor(np.asarray(x, np.int32)).cuda()  # noqa: E731
    a, c, tab, fr, cnt = t(np.ones(40)), t(ctx), t(tables), t(free), t([len(free)])
    starts, seq, pos = t([0] * 41), t([0] * 40), t([0] * 40)
    slots = torch.zeros(40, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        pk.paged_kv_build_tables(a, c, tab, fr, cnt, 16, blocks, starts, seq, pos, slots)
    h_ctx, h_tab, h_cnt = ctx, tables, len(free)
    for _ in range(40):
        g.replay()
        w = walk(np.ones(40, int), h_ctx, h_tab, free, h_cnt, 16, 40)
        h_tab, h_ctx, h_cnt = w[0], np.array(w[1]), w[2]
    torch.cuda.synchronize()
    assert np.array_equal(tab.cpu().numpy(), h_tab) and c.tolist() == h_ctx.tolist() and int(cnt) == h_cnt
    assert slots.tolist() == w[6]
    assert pk.device_errors() == 0


def test_the_16_bit_path_right_behind():
    """paged_kv_append_tokens and paged_attention_decode on tables, lengths and token
    lists that the kernel before them writes, step after step in one graph."""
    S, heads, dim, block = 96, 4, 64, 16
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 50, (S,), generator=g)
    held = -(-lens // block)
    blocks, width, steps = int(held.sum()) + S * 3, 8, 30
    ids = torch.randperm(blocks, generator=g).to(torch.int32)
    tables = torch.full((S, width), -1, dtype=torch.int32)
    tables[torch.arange(width)[None] < held[:, None]] = ids[:int(held.sum())]
    i32 = dict(dtype=torch.int32, device="cuda")
    bt, ctx, free = tables.cuda(), lens.to(torch.int32).cuda(), ids[int(held.sum()):].cuda()
    count, new = torch.tensor([len(free)], **i32), torch.ones(S, **i32)
    starts, seq, pos = torch.zeros(S + 1, **i32), torch.zeros(S, **i32), torch.zeros(S, **i32)
    kc, vc = (torch.zeros(blocks, block, heads, dim, dtype=torch.float16, device="cuda") for _ in range(2))
    # every earlier token's rows are zero, so a step's output is its own V row times its weight
    k = torch.zeros(S, heads, dim, dtype=torch.float16, device="cuda")
    v = torch.ones(S, heads, dim, dtype=torch.float16, device="cuda")
    q = torch.zeros(S, heads, dim, dtype=torch.float16, device="cuda")
    out = torch.zeros(steps, S, heads, dim, dtype=torch.float16, device="cuda")

    def step(i):
        pk.paged_kv_build_tables(new, ctx, bt, free, count, block, blocks, starts, seq, pos)
        pk.paged_kv_append_tokens(k, v, bt, seq, pos, kc, vc)
        pk.paged_attention_decode(q, kc, vc, bt, ctx, 1.0, out[i])

    step(0)                                   # (first calls look up addresses: not in a capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(1, steps):
            step(i)
    graph.replay()
    torch.cuda.synchronize()
    assert pk.device_errors() == 0
    for i in range(steps):
        # i + 1 ones among lens + i + 1 tokens of equal weight, in fp16 (2^-11, and P's own)
        want = ((i + 1) / (lens + i + 1).double())[:, None, None]
        got = out[i].cpu().double()
        assert bool(((got - want).abs() <= want * 2.0 ** -9).all()), f"step {i}"
    assert ctx.tolist() == (lens + steps).tolist()


@pytest.mark.parametrize("S,chunk", [(130, 60), (2000, 60), (4096, 9)])
@pytest.mark.parametrize("short", ["blocks", "tokens", "both", "none left"])
def test_requests_wait_when_it_runs_short_in_place(S, chunk, short):
    """The lengths and the count updated in place by several blocks of threads."""
    new, ctx, tables, free, blocks = make(S, 16, S + 1, 200, chunk)
    count = {"blocks": len(free) // 2, "tokens": len(free), "both": len(free) // 3, "none left": 0}[short]
    cap = int(new.sum()) // 2 if short in ("tokens", "both") else int(new.sum())
    want = walk(new, ctx, tables, free, count, 16, cap)
    same(call(new, ctx, tables, free, count, 16, blocks, cap, in_place=True), want)
    assert pk.device_errors() == 0
    assert 0 <= want[3][-1] < new.sum()


@pytest.mark.parametrize("S", [6, 1500])
def test_bad_lengths_and_counts_in_place(S):
    new, ctx, tables, free, blocks = make(S, 16, 2, 50, 40)
    new[1], ctx[2], new[4] = -1, -5, 2 ** 31 - 1
    cap = 80 if S == 6 else 20000
    same(call(new, ctx, tables, free, len(free), 16, blocks, cap, in_place=True),
         walk(new, ctx, tables, free, len(free), 16, cap))
    assert pk.device_errors() == 4 | 8            # CONTEXT_LEN, POSITION
    new[:], ctx = np.maximum(new, 0) % 41, np.maximum(ctx, 0)
    # a count that is no count is taken as its nearest
    for count, taken in ((len(free) + 9, len(free)), (-7, 0)):
        same(call(new, ctx, tables, free, count, 16, blocks, cap, in_place=True),
             walk(new, ctx, tables, free, taken, 16, cap))
        assert pk.device_errors() == 8


@pytest.mark.parametrize("lengths", [False, True])
@pytest.mark.parametrize("short", [False, True])
@pytest.mark.parametrize("S", [40, 1800])
def test_one_of_the_two_in_place(S, short, lengths):
    """The lengths alone, or the count alone, updated in place."""
    new, ctx, tables, free, blocks = make(S, 16, 5, 90, 40)
    count, cap = len(free) // (2 if short else 1), int(new.sum())
    t = lambda x: torch.tensor(np.asarray(x, np.int32)).cuda()  # noqa: E731
    a, c, tab, n = t(new), t(ctx), t(tables), t([count])
    starts, seq, pos = t([-9] * (S + 1)), t([-9] * cap), t([-9] * cap)
    slots = torch.full((cap,), -9, dtype=torch.int64).cuda()
    c_out, n_out = (c, t([-9])) if lengths else (t([-9] * S), n)
    pk.paged_kv_build_tables(a, c, tab, t(free), n, 16, blocks, starts, seq, pos, slots, c_out, n_out)
    got = (tab.cpu().numpy(), c_out.tolist(), int(n_out), starts.tolist(), seq.tolist(), pos.tolist(), slots.tolist())
    same(got, walk(new, ctx, tables, free, count, 16, cap))
    assert c.tolist() == (got[1] if lengths else ctx.tolist()) and int(n) == (count if lengths else got[2])
    assert pk.device_errors() == 0
