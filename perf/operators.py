"""Cases and plain forms of the operators around a paged KV cache held in 4 bits.

The operators, in the order a serving step calls them:

* ``tables``   block tables, token lists and slots of a step, from the requests' lengths
  and a stack of free blocks (``paged_kv_build_tables``);
* ``cache``    new tokens' K and V quantised into the 4-bit pools at their slots, and rows
  read back out of them (``paged_kv_append_q4``, ``paged_kv_gather_q4``);
* ``decode``   one query token per sequence over its 4-bit cache (``paged_attention_decode_q4``);
* ``prefill``  a chunk of query tokens per sequence over it (``paged_attention_prefill_q4``).

The 4-bit cache. 32 neighbouring channels of one token and kv head form a group with a
scale s and a middle m of the cache's 16-bit type; a channel is held as a code c of 0 .. 15
and stands for s * (c - 8) + m. A pool is uint8 [num_blocks][n_kv_heads][block_size][5 D / 8]:
the bytes of one (block, kv head) are first the codes, [D / 32 groups][block_size tokens][16
bytes] with channel 2 i of a group in the low half of byte i, then (s, m) pairs,
[block_size tokens][D / 32 groups][2].

``run`` computes the plain forms from elementary torch operations where ``own`` is false and
calls the framework's kernels where it is true.
"""
import math

import torch

own = False

GROUP = 32          # channels that share a scale and a middle
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # a decode step of a full batch: every request adds one token, some open a new block
        dict(name="tables decode step", kind="tables", seqs=256, chunk=1, chunks=0, context=4096,
             block=16, width=512, pad=0, short=0),
        # a step that admits prompts beside decoding requests, and has not blocks enough for all
        dict(name="tables mixed step", kind="tables", seqs=2048, chunk=511, chunks=256, context=8192,
             block=16, width=640, pad=1000, short=1),
        # the new tokens of a decode step: one per request
        dict(name="cache decode step", kind="cache", dtype="bf16", tokens=64, kv_heads=8, dim=128, block=16, pad=0),
        # a chunk of prompts, padded to a fixed token count
        dict(name="cache prompt chunk", kind="cache", dtype="f16", tokens=8192, kv_heads=8, dim=128, block=16, pad=57),
        # a long prompt of a model with many narrow kv heads, an odd count of tokens
        dict(name="cache narrow heads", kind="cache", dtype="bf16", tokens=16383, kv_heads=32, dim=64, block=32, pad=0),
        # one request answered alone: latency counts
        dict(name="decode one request", kind="decode", dtype="bf16", seqs=1, shortest=1999, longest=1999,
             kv_heads=8, group=4, dim=128, block=16),
        # a full batch of grouped heads, ragged lengths
        dict(name="decode grouped batch", kind="decode", dtype="bf16", seqs=256, shortest=200, longest=4000,
             kv_heads=8, group=4, dim=128, block=16),
        # one kv head per query head, small blocks
        dict(name="decode own heads", kind="decode", dtype="f16", seqs=64, shortest=1, longest=2048,
             kv_heads=32, group=1, dim=64, block=8),
        # few requests over long documents
        dict(name="decode long", kind="decode", dtype="f16", seqs=8, shortest=32768, longest=131072,
             kv_heads=8, group=8, dim=128, block=16),
        # a short follow-up question over a cached document
        dict(name="prefill follow-up", kind="prefill", dtype="bf16", seqs=1, chunk=33, cached=6001,
             kv_heads=8, group=4, dim=128, block=16),
        # several prompts' chunks together, ragged, nothing cached before some of them
        dict(name="prefill ragged batch", kind="prefill", dtype="f16", seqs=6, chunk=700, cached=900,
             kv_heads=8, group=3, dim=64, block=32),
        # a chunk of a long prompt
        dict(name="prefill long chunk", kind="prefill", dtype="bf16", seqs=1, chunk=2048, cached=16384,
             kv_heads=8, group=4, dim=128, block=16),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["tables", "cache", "cache", "decode", "decode", "decode", "prefill", "prefill"])
    block = rng.choice([8, 16, 32])
    if kind == "tables":
        seqs = _log(rng, 1, 4096)
        chunk = _log(rng, 1, 600)
        context = _log(rng, 1, 8192)
        return dict(kind=kind, seqs=seqs, chunk=chunk, chunks=rng.randint(0, max(1, min(seqs, 120000 // chunk))),
                    context=context, block=block, width=(context + chunk) // block + 2 + rng.randint(0, 9),
                    pad=rng.choice([0, rng.randint(1, 300)]), short=rng.choice([0, 0, 1]))
    dtype, dim = rng.choice(["f16", "bf16"]), rng.choice([64, 128, 128])
    if kind == "cache":
        heads = rng.choice([1, 2, 3, 4, 5, 8, 8, 16, 32])
        return dict(kind=kind, dtype=dtype, tokens=_log(rng, 1, max(1, (1 << 25) // (heads * dim))), kv_heads=heads,
                    dim=dim, block=block, pad=rng.choice([0, rng.randint(1, 40)]))
    heads = rng.choice([1, 2, 3, 4, 8, 8, 16])
    if kind == "decode":
        longest = _log(rng, 1, 65536)
        seqs = _log(rng, 1, max(1, min(256, (1 << 22) // (longest * heads))))
        return dict(kind=kind, dtype=dtype, seqs=seqs, shortest=rng.choice([0, 1, max(1, longest // 2), longest]),
                    longest=longest, kv_heads=heads, group=rng.choice([1, 2, 3, 4, 5, 6, 7, 8]), dim=dim, block=block)
    heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 6, 8, 16])
    chunk = _log(rng, 1, 1500)
    cached = rng.choice([0, _log(rng, 1, 12000)])
    seqs = _log(rng, 1, max(1, min(16, (1 << 29) // (chunk * (chunk + cached) * heads * group))))
    return dict(kind=kind, dtype=dtype, seqs=seqs, chunk=chunk, cached=cached, kv_heads=heads, group=group,
                dim=dim, block=block)


# ---------------------------------------------------------------------------
# What a program has in hand before the calls
# ---------------------------------------------------------------------------
def _generators(seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 11)
    h = torch.Generator()
    h.manual_seed(int(seed) * 104729 + 5)
    return dev, g, h


def _keys(shape, dtype, dev, g):
    """Keys as models make them: normal, with some channels that stand far off zero in every token."""
    heads, dim = shape[-2:]
    far = torch.randn(heads, dim, device=dev, generator=g) * (torch.rand(heads, dim, device=dev, generator=g) < 0.06) * 4
    return (torch.randn(shape, device=dev, generator=g) + far).to(dtype)


def _values(shape, dtype, dev, g):
    """Values: normal around a small mean of each channel."""
    return (torch.randn(shape, device=dev, generator=g) + 0.2 * torch.randn(shape[-2:], device=dev, generator=g)).to(dtype)


def _spread(low, high, n, h):
    """n whole numbers spaced evenly over [low, high], the same ones for every seed, in an order of the seed's."""
    return torch.linspace(low, high, n).round().long()[torch.randperm(n, generator=h)] if n > 1 else torch.tensor([high])


def _tables(lens, block, dev, h, spare=3):
    """Blocks for each sequence's tokens from one shuffled pool; unused entries hold -1."""
    need = (lens + block - 1) // block
    total = int(need.sum()) + spare
    ids = torch.randperm(total, generator=h)
    width = max(1, int(need.max()))
    held = torch.arange(width)[None] < need[:, None]
    tables = torch.full((len(lens), width), -1, dtype=torch.int64)
    tables[held] = ids[:int(need.sum())]
    return tables.to(torch.int32).to(dev), total


def prepare(case, seed):
    dev, g, h = _generators(seed)
    kind, block = case["kind"], case["block"]

    def filled_pool(blocks, heads, dim, dtype, make):
        pool = torch.empty(blocks, heads, block, dim * 5 // 8, dtype=torch.uint8, device=dev)
        step = max(1, (1 << 27) // (block * heads * dim))
        for b in range(0, blocks, step):
            n = min(step, blocks - b)
            _write(pool[b:b + n], torch.arange(n * block, device=dev), make((n * block, heads, dim), dtype, dev, g))
        return pool

    if kind == "tables":
        seqs, width = case["seqs"], case["width"]
        new = torch.ones(seqs, dtype=torch.int64)
        n = min(case["chunks"], seqs)
        new[torch.randperm(seqs, generator=h)[:n]] = _spread(1, case["chunk"], n, h)
        ctx = torch.randint(0, case["context"] + 1, (seqs,), generator=h)
        # blocks of a step's new tokens, with some to spare or too few of them
        held = (ctx + block - 1) // block
        need = (ctx + new + block - 1) // block - held
        free = int(need.sum()) * (3 if case["short"] else 5) // 4 + (0 if case["short"] else 1)
        total = int(held.sum()) + free
        ids = torch.randperm(total, generator=h)
        tables = torch.full((seqs, width), -1, dtype=torch.int64)
        tables[torch.arange(width)[None] < held[:, None]] = ids[:int(held.sum())]
        tokens = int(new.sum()) + case["pad"]
        i32 = lambda t: t.to(torch.int32).to(dev)  # noqa: E731
        return dict(case, new=i32(new), ctx=i32(ctx), tables=i32(tables), free=i32(ids[int(held.sum()):]),
                    count=torch.tensor([free], dtype=torch.int32, device=dev), blocks=total,
                    ctx_out=torch.zeros(seqs, dtype=torch.int32, device=dev),
                    count_out=torch.zeros(1, dtype=torch.int32, device=dev),
                    starts=torch.zeros(seqs + 1, dtype=torch.int32, device=dev),
                    seq=torch.zeros(tokens, dtype=torch.int32, device=dev),
                    pos=torch.zeros(tokens, dtype=torch.int32, device=dev),
                    slots=torch.zeros(tokens, dtype=torch.int64, device=dev))
    dtype, heads, dim = DTYPES[case["dtype"]], case["kv_heads"], case["dim"]
    if kind == "cache":
        tokens, pad = case["tokens"], case["pad"]
        blocks = (tokens + block - 1) // block + 2
        shape = (tokens + pad, heads, dim)
        slots = torch.randperm(blocks * block, device=dev, generator=g)[:tokens]
        slots = torch.cat([slots, torch.full((pad,), -1, dtype=torch.int64, device=dev)])
        pool = lambda: torch.zeros(blocks, heads, block, dim * 5 // 8, dtype=torch.uint8, device=dev)  # noqa: E731
        return dict(case, k=_keys(shape, dtype, dev, g), v=_values(shape, dtype, dev, g), slots=slots, k_cache=pool(),
                    v_cache=pool(), k_out=torch.zeros(shape, dtype=dtype, device=dev),
                    v_out=torch.zeros(shape, dtype=dtype, device=dev))
    seqs, group = case["seqs"], case["group"]
    scale = 1.0 / math.sqrt(dim)
    if kind == "decode":
        lens = _spread(case["shortest"], case["longest"], seqs, h)
        tables, blocks = _tables(lens, block, dev, h)
        rows, starts, most = seqs, None, 1
    else:
        chunk = _spread((case["chunk"] + 1) // 2, case["chunk"], seqs, h)
        cached = _spread(0, case["cached"], seqs, h)
        lens = chunk + cached
        tables, blocks = _tables(lens, block, dev, h)
        starts = torch.cat([torch.zeros(1, dtype=torch.int64), chunk.cumsum(0)]).to(torch.int32).to(dev)
        rows, most = int(chunk.sum()), int(chunk.max())
    q = torch.randn(rows, heads * group, dim, device=dev, generator=g).to(dtype)
    return dict(case, q=q, k_cache=filled_pool(blocks, heads, dim, dtype, _keys),
                v_cache=filled_pool(blocks, heads, dim, dtype, _values), tables=tables,
                lens=lens.to(torch.int32).to(dev), starts=starts, most=most, scale=scale, out=torch.zeros_like(q))


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _down(x, dtype):
    """Positive fp32 values to a 16-bit type, rounded towards zero."""
    y = x.to(dtype)
    return torch.where(y.float() > x, (y.view(torch.int16) - 1).view(dtype), y)


def _quantise(x):
    """[..., D] -> codes uint8 [..., D / 32, 16], (s, m) [..., D / 32, 2] of x's type."""
    y = x.unflatten(-1, (-1, GROUP)).float()
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    s = _down((hi - lo) / 15, x.dtype)
    m = (0.5 * lo + 0.5 * hi + 0.5 * s.float()).to(x.dtype)
    # the nearest code, ties to even; 64 bits, so that values next to a border fall on their side of it
    c = torch.round((y - m.float()).double() / s.double()).clamp(-8, 7) + 8
    c = torch.where((s > 0) & torch.isfinite(s), c, torch.full_like(c, 8)).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.cat([s, m], -1)


def _parts(pool, dim, dtype):
    """Views of a pool's codes [NB][Hkv][G][B][16] and (s, m) pairs [NB][Hkv][B][G][2]."""
    nb, heads, block, _ = pool.shape
    flat, groups = pool.flatten(2), dim // GROUP
    codes = flat[..., :groups * block * 16].unflatten(-1, (groups, block, 16))
    return codes, flat[..., groups * block * 16:].view(dtype).unflatten(-1, (block, groups, 2))


def _write(pool, slots, x):
    """Quantise rows [T][Hkv][D] into the pool's slots."""
    codes, pairs = _parts(pool, x.shape[-1], x.dtype)
    block = pool.shape[2]
    c, p = _quantise(x)
    codes[slots // block, :, :, slots % block] = c
    pairs[slots // block, :, slots % block] = p


def _stands_for(codes, pairs):
    """codes [..., 16] and (s, m) [..., 2] -> fp32 [..., 32]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8
    return c * pairs[..., 0:1].float() + pairs[..., 1:2].float()


def _read(pool, slots, dim, dtype):
    codes, pairs = _parts(pool, dim, dtype)
    block = pool.shape[2]
    return _stands_for(codes[slots // block, :, :, slots % block], pairs[slots // block, :, slots % block]).flatten(-2)


def _sequences(pool, tables, dim, dtype):
    """The sequences' rows through their tables, fp32 [S][Hkv][width * B][D]."""
    codes, pairs = _parts(pool, dim, dtype)
    ids = tables.long().clamp(min=0)
    x = _stands_for(codes[ids], pairs[ids].transpose(3, 4))        # [S][W][Hkv][G][B][32]
    return x.permute(0, 2, 1, 4, 3, 5).flatten(4).flatten(2, 3)


def _softmax(z, live):
    z = torch.where(live, z, torch.full_like(z, -math.inf))
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, torch.ones_like(total))


def _plain_tables(st):
    block, cap = st["block"], st["seq"].numel()
    new, ctx, tables = st["new"].long(), st["ctx"].long(), st["tables"].long()
    width = tables.shape[1]
    free = st["count"].long()
    held = (ctx + block - 1) // block
    valid = (new >= 0) & (ctx >= 0) & (ctx + new <= width * block)
    new = torch.where(valid, new, torch.zeros_like(new))
    need = torch.where(valid, (ctx + new + block - 1) // block - held, torch.zeros_like(new))
    # in order: a request that needs more than is left waits, and so does each later one that needs any
    go = valid & ((need == 0) | (need.cumsum(0) <= free)) & ((new == 0) | (new.cumsum(0) <= cap))
    new, need = new * go, need * go
    starts = torch.cat([new.new_zeros(1), new.cumsum(0)])
    nth = torch.arange(width, device=new.device)[None] - held[:, None]
    opened = (nth >= 0) & (nth < need[:, None])
    taken = (free - 1 - (need.cumsum(0) - need)[:, None] - nth).clamp(min=0, max=max(0, st["free"].numel() - 1))
    if st["free"].numel():
        tables = torch.where(opened, st["free"].long()[taken], tables)
    t = torch.arange(cap, device=new.device)
    live = t < starts[-1]
    s = torch.searchsorted(starts[1:], t, right=True) * live
    pos = torch.where(live, ctx[s] + t - starts[s], torch.full_like(t, -1))
    slot = torch.where(live, tables[s, pos.clamp(min=0) // block] * block + pos % block, torch.full_like(t, -1))
    i32 = torch.int32
    return (tables.to(i32), (ctx + new).to(i32), (free - need.sum()).to(i32), starts.to(i32), s.to(i32), pos.to(i32), slot)


def _plain_cache(st):
    dtype, dim, slots = st["k"].dtype, st["dim"], st["slots"]
    live = slots >= 0
    at = slots[live]
    _write(st["k_cache"], at, st["k"][live])
    _write(st["v_cache"], at, st["v"][live])
    at, keep = slots.clamp(min=0), live[:, None, None]
    k, v = _read(st["k_cache"], at, dim, dtype).to(dtype), _read(st["v_cache"], at, dim, dtype).to(dtype)
    return torch.where(keep, k, st["k_out"]), torch.where(keep, v, st["v_out"])


def _plain_decode(st):
    q, dim, dtype = st["q"], st["dim"], st["q"].dtype
    x = q.float().unflatten(1, (st["kv_heads"], st["group"]))
    k = _sequences(st["k_cache"], st["tables"], dim, dtype)
    z = (x @ k.transpose(2, 3)) * st["scale"]
    del k
    live = torch.arange(z.shape[-1], device=z.device)[None] < st["lens"].long()[:, None]
    p = _softmax(z, live[:, None, None])
    return (p @ _sequences(st["v_cache"], st["tables"], dim, dtype)).flatten(1, 2).to(dtype)


def _plain_prefill(st):
    q, dim, dtype = st["q"], st["dim"], st["q"].dtype
    starts, lens = st["starts"].long(), st["lens"].long()
    n = starts[1:] - starts[:-1]
    j = torch.arange(st["most"], device=q.device)[None]
    inside = j < n[:, None]                                           # [S][most]
    rows = torch.where(inside, starts[:-1, None] + j, torch.zeros_like(j))
    x = q.float()[rows].unflatten(2, (st["kv_heads"], st["group"])).permute(0, 2, 3, 1, 4)
    k = _sequences(st["k_cache"], st["tables"], dim, dtype)[:, :, None]
    z = (x @ k.transpose(3, 4)) * st["scale"]                         # [S][Hkv][g][most][L]
    del k
    key = torch.arange(z.shape[-1], device=z.device)
    live = inside[..., None] & (key <= ((lens - n)[:, None] + j)[..., None])
    p = _softmax(z, live[:, None, None])
    del z
    o = (p @ _sequences(st["v_cache"], st["tables"], dim, dtype)[:, :, None]).permute(0, 3, 1, 2, 4).flatten(2, 3)
    out = torch.zeros_like(q)
    out[rows[inside]] = o[inside].to(dtype)
    return out


def run(state):
    kind = state["kind"]
    if not own:
        if kind == "tables":
            return _plain_tables(state)
        if kind == "cache":
            return _plain_cache(state)
        return _plain_decode(state) if kind == "decode" else _plain_prefill(state)
    import paged_kv_cache_233_gb300 as pk
    st = state
    if kind == "tables":
        pk.paged_kv_build_tables(st["new"], st["ctx"], st["tables"], st["free"], st["count"], st["block"], st["blocks"],
                                 st["starts"], st["seq"], st["pos"], st["slots"], st["ctx_out"], st["count_out"])
        return st["tables"], st["ctx_out"], st["count_out"], st["starts"], st["seq"], st["pos"], st["slots"]
    if kind == "cache":
        pk.paged_kv_append_q4(st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"])
        pk.paged_kv_gather_q4(st["k_cache"], st["v_cache"], st["slots"], st["k_out"], st["v_out"])
        return st["k_out"], st["v_out"]
    if kind == "decode":
        if "workspace" not in st:     # a program makes it once, with its buffers
            st["workspace"] = pk.new_workspace(st["q"], st["tables"], st["block"], pk.PARTITION_BALANCED)
        pk.paged_attention_decode_q4(st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], st["scale"],
                                     st["out"], pk.PARTITION_BALANCED, st["workspace"])
        return st["out"]
    if "workspace" not in st:
        st["workspace"] = pk.prefill_workspace(st["q"])
    pk.paged_attention_prefill_q4(st["q"], st["k_cache"], st["v_cache"], st["tables"], st["starts"], st["lens"],
                                  st["scale"], st["out"], st["most"], workspace=st["workspace"], key_parts=0)
    return st["out"]


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    kind, block = case["kind"], case["block"]
    if kind == "tables":
        seqs = case["seqs"]
        tokens = seqs + min(case["chunks"], seqs) * (case["chunk"] - 1) / 2
        opened = tokens / block
        # lengths in and out, starts, the last partial block's entry, opened blocks in and out, each token's row
        return {"bytes": 4.0 * (4 * seqs + 2 * opened) + 16.0 * (tokens + case["pad"]), "flops": 0.0}
    heads, dim = case["kv_heads"], case["dim"]
    held = 2.0 * heads * dim * 5 / 8       # bytes of a token's K and V in 4 bits
    if kind == "cache":
        tokens = case["tokens"]
        rows = 2.0 * heads * dim * 2
        return {"bytes": tokens * (2 * rows + 2 * held + 16), "flops": tokens * 2.0 * heads * dim * 8}
    q_heads = heads * case["group"]
    if kind == "decode":
        keys = case["longest"] if case["seqs"] == 1 else case["seqs"] * (case["shortest"] + case["longest"]) / 2
        return {"bytes": keys * (held + 4 / block) + case["seqs"] * 4.0 * q_heads * dim,
                "flops": 4.0 * keys * q_heads * dim}
    chunk = case["chunk"] if case["seqs"] == 1 else 0.75 * case["chunk"]
    cached = case["cached"] if case["seqs"] == 1 else 0.5 * case["cached"]
    pairs = case["seqs"] * chunk * (cached + (chunk + 1) / 2)
    return {"bytes": case["seqs"] * ((chunk + cached) * held + chunk * 4.0 * q_heads * dim),
            "flops": 4.0 * pairs * q_heads * dim}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    def by_hand(st):
        new, ctx, free = st["new"].tolist(), st["ctx"].tolist(), st["free"].tolist()
        tables, left, block = st["tables"].cpu().clone(), int(st["count"]), st["block"]
        cap, blocks_asked, tokens_asked, tokens = st["seq"].numel(), 0, 0, 0
        start_count = left
        lens, starts, seq, pos, slot = [], [0], [], [], []
        for s, (n, c) in enumerate(zip(new, ctx)):
            held, after = -(-c // block), -(-(c + n) // block)
            ok = n >= 0 and c >= 0 and c + n <= tables.shape[1] * block
            if ok:
                blocks_asked += after - held
                tokens_asked += n
                ok = (after == held or blocks_asked <= start_count) and (n == 0 or tokens_asked <= cap)
            if ok:
                for j in range(held, after):
                    left -= 1
                    tables[s, j] = free[left]
                mine = tables[s].tolist()
                for i in range(c, c + n):
                    seq.append(s)
                    pos.append(i)
                    slot.append(mine[i // block] * block + i % block)
                tokens += n
            lens.append(c + n if ok else c)
            starts.append(tokens)
        rest = cap - tokens
        i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
        return (tables, i32(lens), i32([left]), i32(starts), i32(seq + [0] * rest), i32(pos + [-1] * rest),
                torch.tensor(slot + [-1] * rest, dtype=torch.int64))

    def row(x):
        """What 16-bit rows [..., D] stand for after 4 bits, in fp64, from the definition."""
        y = x.double().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
        low, high = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
        # a scale of the type: its spacing at this size, 11 or 8 significant bits, rounded down
        bits, least = (10, -24) if x.dtype == torch.float16 else (7, -133)
        width = (high - low) / 15
        grid = torch.exp2((torch.floor(torch.log2(width.clamp(min=1e-300))) - bits).clamp(min=least))
        s = torch.floor(width / grid) * grid
        m = ((low + high + s) / 2).to(x.dtype).double()
        c = torch.where(s > 0, torch.round((y - m) / s.clamp(min=1e-300)).clamp(-8, 7), torch.zeros_like(y))
        return (s * c + m).reshape(x.shape)

    def held_rows(pool, ids, n, dim, dtype):
        """A sequence's first n rows, fp64 [Hkv][n][D], byte by byte from its blocks."""
        _, heads, block, _ = pool.shape
        groups = dim // 32
        raw = pool[ids.long()].reshape(len(ids), heads, -1)
        split = block * dim // 2
        half = raw[..., :split].reshape(len(ids), heads, groups, block, 16).to(torch.int16)
        c = torch.empty(len(ids), heads, groups, block, 32, dtype=torch.float64, device=pool.device)
        c[..., 0::2], c[..., 1::2] = (half % 16).double(), (half // 16).double()
        pair = raw[..., split:].contiguous().view(dtype).double().reshape(len(ids), heads, block, groups, 2)
        s, m = (pair[..., i].permute(0, 1, 3, 2)[..., None] for i in (0, 1))
        x = (c - 8) * s + m
        return x.permute(1, 0, 3, 2, 4).reshape(heads, len(ids) * block, dim)[:, :n]

    def attention(st):
        q, out = st["q"].double(), torch.zeros_like(st["q"], dtype=torch.float64)
        lens = st["lens"].tolist()
        starts = st["starts"].tolist() if st["starts"] is not None else list(range(len(lens) + 1))
        heads, group, block, dtype = st["kv_heads"], st["group"], st["block"], st["q"].dtype
        for s, n in enumerate(lens):
            a, b = starts[s], starts[s + 1]
            if n == 0 or a == b:
                continue
            ids = st["tables"][s, :-(-n // block)]
            k, v = (held_rows(st[w], ids, n, st["dim"], dtype) for w in ("k_cache", "v_cache"))
            seen = torch.arange(n, device=q.device)[None] <= torch.arange(n - (b - a), n, device=q.device)[:, None]
            for h in range(heads):
                for i in range(h * group, (h + 1) * group):
                    z = (q[a:b, i] @ k[h].T) * st["scale"]
                    w = torch.softmax(z.masked_fill(~seen, -math.inf), -1)
                    out[a:b, i] = w @ v[h]
        return out

    st = prepare(case, seed)
    if case["kind"] == "tables":
        return by_hand(st)
    if case["kind"] == "cache":
        live = (st["slots"] >= 0)[:, None, None]
        return tuple(torch.where(live, row(st[w]), torch.zeros((), dtype=torch.float64, device=st[w].device))
                     for w in ("k", "v"))
    return attention(st)
