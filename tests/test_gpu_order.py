"""Calls right behind one another on a stream and in a graph, each reading what the
one before it wrote: the kernels are chained by programmatic dependent launch, so a
kernel that may start early has to wait before it reads that. Every chain's results
are compared with those of the same calls with a synchronisation between them."""
import pytest
import torch

import paged_kv_cache_233_gb300 as pk

pytestmark = pytest.mark.gpu
F16 = torch.float16
TIMES = 6


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pk.load()
    torch.cuda.set_device(0)
    pk.device_errors()


class Cache:
    """S sequences of n tokens in shuffled blocks, 16-bit and 4-bit pools of the same rows."""

    def __init__(self, S, n, heads, dim=128, block=16, seed=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.dim, self.block = heads, dim, block
        per = -(-n // block)
        self.blocks = S * per
        self.tables = torch.randperm(self.blocks, generator=g, device="cuda").to(torch.int32).view(S, per)
        self.lens = torch.full((S,), n, dtype=torch.int32, device="cuda")
        self.kc, self.vc = (torch.randn(self.blocks, block, heads, dim, generator=g, device="cuda", dtype=F16) for _ in range(2))
        self.k4, self.v4 = (pk.new_q4_pool(self.blocks, heads, block, dim) for _ in range(2))
        slots = torch.arange(self.blocks * block, device="cuda")
        pk.paged_kv_append_q4(self.kc.flatten(0, 1), self.vc.flatten(0, 1), slots, self.k4, self.v4)
        torch.cuda.synchronize()

    def decode(self, bits, q, out, part, ws, lens=None):
        f = pk.paged_attention_decode_q4 if bits == 4 else pk.paged_attention_decode
        k, v = (self.k4, self.v4) if bits == 4 else (self.kc, self.vc)
        f(q, k, v, self.tables, self.lens if lens is None else lens, self.dim ** -0.5, out, part, ws)


def queries(S, heads, dim, seed):
    return torch.randn(S, heads, dim, generator=torch.Generator().manual_seed(seed)).to(F16).cuda()


def same_as_apart(steps, reset, results, graph):
    """steps: calls in order. The results of a run with a synchronisation after each,
    and of runs without any, are the same bits."""
    reset()
    for s in steps:
        s()
        torch.cuda.synchronize()
    want = [r.clone() for r in results]
    torch.cuda.synchronize()
    g = None
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for s in steps:
                s()
    for _ in range(TIMES):
        reset()
        torch.cuda.synchronize()
        if graph:
            g.replay()
        else:
            for s in steps:
                s()
        torch.cuda.synchronize()
        for r, w in zip(results, want):
            assert torch.equal(r, w)
    assert pk.device_errors() == 0


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("bits,part,S,n,heads", [
    (4, 512, 400, 500, 8), (16, 512, 400, 500, 8),      # every row within one partition
    (4, 2048, 30, 2000, 8), (16, 2048, 30, 2000, 8),
    (4, 32, 600, 32, 8),                                 # more than 32 partitions in the tables' width
    (16, pk.PARTITION_BALANCED, 38, 1024, 32),           # every pair within one share of 304
    (4, pk.PARTITION_BALANCED, 57, 1024, 32), (4, 512, 40, 1500, 8)])
def test_rows_taken_right_behind_a_decode(bits, part, S, n, heads, graph):
    """A decode whose merge has nothing to do for any row, and an append of its
    outputs, which waits for the merge alone."""
    c = Cache(S, n, heads)
    if part == 32:
        c.tables = torch.cat([c.tables, c.tables.repeat(1, 40)], 1).contiguous()
    q = queries(S, heads, c.dim, 2)
    out = torch.empty_like(q)
    ws = pk.new_workspace(q, c.tables, c.block, part)
    k4, v4 = (pk.new_q4_pool(-(-S // c.block), heads, c.block, c.dim) for _ in range(2))
    kc, vc = (torch.empty(-(-S // c.block), c.block, heads, c.dim, dtype=F16, device="cuda") for _ in range(2))
    slots = torch.arange(S, device="cuda")

    def reset():
        for x in (out, kc, vc):
            x.fill_(-1)
        for x in (k4, v4):
            x.fill_(0)

    for take, pools in ((lambda: pk.paged_kv_append_q4(out, out, slots, k4, v4), (k4, v4)),
                        (lambda: pk.paged_kv_append(out, out, slots, kc, vc), (kc, vc))):
        same_as_apart([lambda: c.decode(bits, q, out, part, ws), take], reset, [out, *pools], graph)


@pytest.mark.parametrize("graph", [False, True])
def test_lengths_moved_on_right_behind_a_decode(graph):
    """paged_kv_build_tables moves the lengths on in place behind a decode whose merge
    has nothing to do."""
    c = Cache(400, 500, 8)
    q = queries(400, 8, c.dim, 2)
    out, part = torch.empty_like(q), 512
    ws = pk.new_workspace(q, c.tables, c.block, part)
    i32 = dict(dtype=torch.int32, device="cuda")
    new, free, count = torch.ones(400, **i32), torch.zeros(1, **i32), torch.zeros(1, **i32)
    start, seq, pos = torch.empty(401, **i32), torch.empty(400, **i32), torch.empty(400, **i32)

    def reset():
        out.fill_(-1)
        c.lens.fill_(500)

    def tables():
        pk.paged_kv_build_tables(new, c.lens, c.tables, free, count, c.block, c.blocks, start, seq, pos)

    same_as_apart([lambda: c.decode(4, q, out, part, ws), tables, lambda: c.decode(4, q, out, part, ws), tables], reset,
                  [out, c.lens], graph)


def test_zero_rows_behind_a_decode_of_the_same_rows():
    """A balanced 16-bit decode of empty sequences alone, right behind a long decode
    into the same rows, and an append of them."""
    c = Cache(64, 4000, 8)
    q = queries(64, 8, c.dim, 2)
    out, part = torch.empty_like(q), pk.PARTITION_BALANCED
    ws = [pk.new_workspace(q, c.tables, c.block, part) for _ in range(2)]
    none = torch.zeros_like(c.lens)
    kc, vc = (torch.empty(4, 16, 8, c.dim, dtype=F16, device="cuda") for _ in range(2))
    slots = torch.arange(64, device="cuda")

    def reset():
        for x in (out, kc, vc):
            x.fill_(-1)

    same_as_apart([lambda: c.decode(16, q, out, part, ws[0]), lambda: c.decode(16, q, out, part, ws[1], none),
                   lambda: pk.paged_kv_append(out, out, slots, kc, vc)], reset, [out, kc, vc], False)
    assert bool((out == 0).all()) and bool((kc == 0).all())


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("part", [0, 512, pk.PARTITION_BALANCED])
@pytest.mark.parametrize("first,second", [(16, 16), (4, 16), (16, 4), (16, "prefill"), (4, "prefill")])
def test_outputs_as_the_next_queries(first, second, part, graph):
    """A call's outputs are the queries of the one right behind it, three in a row."""
    S, heads = 48, 8
    c = Cache(S, 1500, heads)
    q = queries(S, heads, c.dim, 2)
    xs = [torch.empty_like(q) for _ in range(3)]
    ws = [pk.new_workspace(q, c.tables, c.block, part) for _ in range(3)]
    starts = torch.arange(S + 1, dtype=torch.int32, device="cuda")

    def call(kind, q, out, w):
        if kind == "prefill":
            pk.paged_attention_prefill(q, c.kc, c.vc, c.tables, starts, c.lens, c.dim ** -0.5, out, 1)
        else:
            c.decode(kind, q, out, part, w)

    def reset():
        for x in xs:
            x.fill_(-1)

    same_as_apart([lambda: call(first, q, xs[0], ws[0]), lambda: call(second, xs[0], xs[1], ws[1]),
                   lambda: call(second, xs[1], xs[2], ws[2])], reset, xs, graph)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("part", [0, 64, pk.PARTITION_BALANCED])
def test_16_bit_calls_right_behind_the_tables(part, graph):
    """Tables, lengths and token lists in place, then the 16-bit append, decode and
    prefill that read them, two steps in a row."""
    S, heads, n = 300, 8, 95
    c = Cache(S, n, heads)
    more = S * 3
    tables = torch.full((S, 12), -1, dtype=torch.int32, device="cuda")
    tables[:, :c.tables.shape[1]] = c.tables
    kc, vc = (torch.cat([x, torch.zeros(more, *x.shape[1:], dtype=F16, device="cuda")]) for x in (c.kc, c.vc))
    i32 = dict(dtype=torch.int32, device="cuda")
    stack = torch.arange(c.blocks, c.blocks + more, **i32)
    new, T = (torch.arange(S, **i32) % 4 + 1), int((torch.arange(S) % 4 + 1).sum())
    t, lens, count = tables.clone(), c.lens.clone(), torch.tensor([more], **i32)
    start, seq, pos = torch.empty(S + 1, **i32), torch.empty(T, **i32), torch.empty(T, **i32)
    k, v = queries(T, heads, c.dim, 5), queries(T, heads, c.dim, 6)
    q, qp = queries(S, heads, c.dim, 7), queries(T, heads, c.dim, 8)
    outs = [torch.empty_like(q) for _ in range(2)]
    rows = [torch.empty_like(qp) for _ in range(2)]
    pools = [torch.empty_like(x) for x in (kc, vc)]
    ws = pk.new_workspace(q, t, c.block, part)

    def reset():
        t.copy_(tables), lens.copy_(c.lens), count.fill_(more)
        pools[0].copy_(kc), pools[1].copy_(vc)
        for x in (start, seq, pos, *outs, *rows):
            x.fill_(-1)

    def step(i):
        return [lambda: pk.paged_kv_build_tables(new, lens, t, stack, count, c.block, c.blocks + more, start, seq, pos),
                lambda: pk.paged_kv_append_tokens(k, v, t, seq, pos, *pools),
                lambda: pk.paged_attention_decode(q, *pools, t, lens, 0.09, outs[i], part, ws),
                lambda: pk.paged_attention_prefill(qp, *pools, t, start, lens, 0.09, rows[i], 4)]

    same_as_apart(step(0) + step(1), reset, [t, lens, count, start, seq, pos, *pools, *outs, *rows], graph)
    assert lens.tolist() == (c.lens + 2 * new).tolist()


def chunks(c, S, rows, heads):
    """S chunks of `rows` queries at the ends of their sequences, and their outputs."""
    q = queries(S * rows, heads, c.dim, 3)
    starts = (torch.arange(S + 1) * rows).to(torch.int32).cuda()
    return q, torch.zeros_like(q), starts


@pytest.mark.parametrize("bits", [4, 16])
def test_prefill_takes_its_workspace_on_the_calls_stream(bits, monkeypatch):
    """The workspace a split call allocates for itself goes back to the stream that
    the call runs on: memory given out next on another stream is not it."""
    c = Cache(2, 3000, 4)
    q, out, starts = chunks(c, 2, 40, 8)
    f = pk.paged_attention_prefill_q4 if bits == 4 else pk.paged_attention_prefill
    pools = (c.k4, c.v4) if bits == 4 else (c.kc, c.vc)
    want = torch.zeros_like(q)
    f(q, *pools, c.tables, starts, c.lens, 0.09, want, 40, workspace=pk.prefill_workspace(q), key_parts=8)
    torch.cuda.synchronize()
    taken = []
    make = pk.prefill_workspace

    def recording(q):
        w = make(q)
        taken.append((w.data_ptr(), w.numel()))
        return w

    monkeypatch.setattr(pk, "prefill_workspace", recording)
    side = torch.cuda.Stream()
    for _ in range(4):
        f(q, *pools, c.tables, starts, c.lens, 0.09, out, 40, stream=side, key_parts=8)
        at, size = taken[-1]
        mine = torch.empty(size, dtype=torch.uint8, device="cuda")
        assert mine.data_ptr() + size <= at or at + size <= mine.data_ptr()
        del mine
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("bits", [4, 16])
def test_prefill_reads_the_longest_chunk_on_the_calls_stream(bits):
    """query_start written on the call's own stream, which is behind."""
    c = Cache(3, 200, 4)
    q, out, starts = chunks(c, 3, 50, 8)
    f = pk.paged_attention_prefill_q4 if bits == 4 else pk.paged_attention_prefill
    pools = (c.k4, c.v4) if bits == 4 else (c.kc, c.vc)
    want = torch.zeros_like(q)
    f(q, *pools, c.tables, starts, c.lens, 0.09, want, 50)
    late = torch.zeros_like(starts)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(starts)
    f(q, *pools, c.tables, late, c.lens, 0.09, out, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and bool((want != 0).any())
