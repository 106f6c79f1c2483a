"""Cases and plain forms of the operators around a paged KV cache held in 8 bits.

The operators, in the order a serving step calls them:

* ``pages``    parallel samples forked off their prompts' rows, then blocks of finished and of
  shortened sequences given back to the free stack (``paged_kv_fork``, ``paged_kv_release``);
* ``cache``    a step's K and V rows quantised into the 8-bit pools behind each sequence's older
  tokens, and rows read back out of them (``paged_kv_append_q8``, ``paged_kv_gather_q8``);
* ``decode``   one query token per sequence over its 8-bit cache (``paged_attention_decode_q8``);
* ``prefill``  a chunk of query tokens per sequence over it (``paged_attention_prefill_q8``).

The 8-bit cache. The tokens of one block and kv head share a scale, a power of two 2^e, and a
channel is held as an e4m3 code c, which stands for c * 2^e. A pool is uint8 [num_blocks]
[n_kv_heads][block_size][D + tail], tail = 16 bytes (32 in blocks of 32) over block_size: the bytes
of one (block, kv head) are first the codes, [D / 16 panels][block_size tokens][16 bytes], then the
scale in fp32. An append sets 2^e to the smallest that holds the rows that it brings, at least 2^-64
and what the block's tokens before them had; their codes are then rounded anew where it grew.

``run`` computes the plain forms from elementary torch operations where ``own`` is false and
calls the framework's kernels where it is true.
"""
import math

import torch

own = False

PANEL = 16          # channels of a token that lie together
LEAST = -64         # the smallest scale's exponent
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
KEEP_ALL = 1 << 30


def listed():
    return [
        # a few requests, each sampled more than once, between two steps of a small server
        dict(name="pages few requests", kind="pages", seqs=24, children=8, context=1500, block=16, width=128, spare=300),
        # a large server's batch: many samples of long prompts, finished requests and drafts taken back
        dict(name="pages large batch", kind="pages", seqs=1024, children=1000, context=8192, block=16, width=520,
             spare=20000),
        # the new tokens of a decode step: one per request, mostly into started blocks
        dict(name="cache decode step", kind="cache", dtype="bf16", seqs=64, chunk=1, cached=4096, kv_heads=8, dim=128,
             block=16, pad=0),
        # chunks of prompts, padded to a fixed token count
        dict(name="cache prompt chunks", kind="cache", dtype="f16", seqs=12, chunk=1024, cached=700, kv_heads=8, dim=128,
             block=16, pad=57),
        # a long prompt of a model with many narrow kv heads, an odd count of tokens
        dict(name="cache narrow heads", kind="cache", dtype="bf16", seqs=1, chunk=16383, cached=5, kv_heads=32, dim=64,
             block=32, pad=0),
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
    kind = rng.choice(["pages", "cache", "cache", "decode", "decode", "decode", "prefill", "prefill"])
    block = rng.choice([8, 16, 32])
    if kind == "pages":
        seqs = _log(rng, 1, 2000)
        context = _log(rng, 1, max(1, min(8192, (1 << 22) // seqs)))
        return dict(kind=kind, seqs=seqs, children=rng.randint(0, min(seqs, 2000)), context=context, block=block,
                    width=context // block + 1 + rng.randint(0, 9), spare=_log(rng, 1, 20000))
    dtype, dim = rng.choice(["f16", "bf16"]), rng.choice([64, 128, 128])
    if kind == "cache":
        heads = rng.choice([1, 2, 3, 4, 5, 8, 8, 16, 32])
        chunk = rng.choice([1, 1, _log(rng, 2, max(2, (1 << 25) // (heads * dim)))])
        return dict(kind=kind, dtype=dtype, seqs=_log(rng, 1, max(1, min(512, (1 << 25) // (heads * dim * chunk)))),
                    chunk=chunk, cached=rng.choice([0, _log(rng, 1, 4000)]), kv_heads=heads, dim=dim, block=block,
                    pad=rng.choice([0, rng.randint(1, 40)]))
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


def _tail(block):
    """Bytes of a (block, kv head) behind its codes, per token."""
    return max(16, block) // block


def _pages(case, seed):
    dev, _, h = _generators(seed)
    seqs, children, block, width = case["seqs"], case["children"], case["block"], case["width"]
    rows = seqs + children
    lens = torch.cat([_spread(0, case["context"], seqs, h), torch.zeros(children, dtype=torch.int64)])
    held = (lens + block - 1) // block
    total = int(held.sum()) + case["spare"]
    ids = torch.randperm(total, generator=h)
    tables = torch.full((rows, width), -1, dtype=torch.int64)
    tables[torch.arange(width)[None] < held[:, None]] = ids[:int(held.sum())]
    shared = torch.zeros(total, dtype=torch.int64)
    # every fourth sequence holds the whole blocks of its left neighbour's prompt, its own go to the stack
    left = []
    for s in range(1, seqs, 4):
        n = int(min(lens[s - 1], lens[s]) // block) // 2
        left.append(tables[s, :n].clone())
        tables[s, :n] = tables[s - 1, :n]
        shared[tables[s, :n]] += 1
    stack = torch.cat([ids[int(held.sum()):], *left])
    stack = stack[torch.randperm(len(stack), generator=h)]
    parents = torch.full((rows,), -1, dtype=torch.int64)
    order = torch.randperm(rows, generator=h)                 # rows change places: children lie among the others
    place = torch.empty_like(order)
    place[order] = torch.arange(rows)
    parents[seqs:] = place[torch.randint(0, seqs, (children,), generator=h)]
    # a third of all sequences is finished, a third takes up to 8 tokens back
    fate = torch.randint(0, 3, (rows,), generator=h)
    after = torch.where(torch.arange(rows) < seqs, lens, lens[order[parents.clamp(min=0)]])
    keep = torch.where(fate == 0, torch.zeros_like(lens), torch.full_like(lens, KEEP_ALL))
    keep = torch.where(fate == 1, (after - torch.randint(0, 9, (rows,), generator=h)).clamp(min=0), keep)
    free = torch.zeros(total, dtype=torch.int64)
    free[:len(stack)] = stack
    i32 = lambda t: t.to(torch.int32).to(dev)  # noqa: E731
    kept = i32(torch.cat([shared, free]))          # what both calls change in place, and what it was
    work = kept.clone()
    return dict(case, lens=i32(lens[order]), tables=i32(tables[order]), parents=i32(parents[order]), keep=i32(keep[order]),
                kept=kept, work=work, shared=work[:total], free=work[total:],
                count=torch.tensor([len(stack)], dtype=torch.int32, device=dev),
                pairs=torch.zeros(rows, 2, dtype=torch.int32, device=dev), blocks=total,
                forked=i32(lens), forked_count=torch.zeros(1, dtype=torch.int32, device=dev),
                lens_out=i32(lens), count_out=torch.zeros(1, dtype=torch.int32, device=dev))


def prepare(case, seed):
    if case["kind"] == "pages":
        return _pages(case, seed)
    dev, g, h = _generators(seed)
    kind, block = case["kind"], case["block"]
    dtype, heads, dim = DTYPES[case["dtype"]], case["kv_heads"], case["dim"]

    def filled_pool(blocks, make):
        """Whole blocks of rows, as earlier steps left them, those past the sequences' ends stale."""
        pool = torch.zeros(blocks, heads, block, dim + _tail(block), dtype=torch.uint8, device=dev)
        step = max(1, (1 << 27) // (block * heads * dim))
        for b in range(0, blocks, step):
            n = min(step, blocks - b)
            codes, scale = _parts(pool[b:b + n], dim)
            x = make((n * block, heads, dim), dtype, dev, g).unflatten(0, (n, block)).transpose(1, 2).float()
            e = _exponent(x.abs().amax((-1, -2)))
            _put(codes, torch.ldexp(x, -e[..., None, None]))
            scale.copy_(torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)[..., None])
        return pool

    seqs = case["seqs"]
    i32 = lambda t: t.to(torch.int32).to(dev)  # noqa: E731
    if kind == "decode":
        lens = _spread(case["shortest"], case["longest"], seqs, h)
        chunk, starts, rows, most = None, None, seqs, 1
    else:
        low = (case["chunk"] + 1) // 2
        chunk = _spread(low, case["chunk"], seqs, h)
        cached = _spread(0, case["cached"], seqs, h)
        lens = chunk + cached
        starts = i32(torch.cat([torch.zeros(1, dtype=torch.int64), chunk.cumsum(0)]))
        rows, most = int(chunk.sum()), int(chunk.max())
    tables, blocks = _tables(lens, block, dev, h)
    pools = dict(k_cache=filled_pool(blocks, _keys), v_cache=filled_pool(blocks, _values))
    if kind == "cache":
        # rows to read back: every token of the blocks that the step writes into, some of them twice, and padding
        first = cached // block * block
        host = tables.cpu().long()
        slots = []
        for s in range(seqs):
            pos = torch.arange(int(first[s]), int(lens[s]))
            slots.append(host[s, pos // block] * block + pos % block)
        slots = torch.cat(slots + [slots[0][:3], torch.full((case["pad"],), -1, dtype=torch.int64)]).to(dev)
        shape = (rows + case["pad"], heads, dim)
        back = (len(slots), heads, dim)
        return dict(case, k=_keys(shape, dtype, dev, g), v=_values(shape, dtype, dev, g), tables=tables, starts=starts,
                    lens=i32(lens), most=most, slots=slots, k_out=torch.zeros(back, dtype=dtype, device=dev),
                    v_out=torch.zeros(back, dtype=dtype, device=dev), **pools)
    q = torch.randn(rows, heads * case["group"], dim, device=dev, generator=g).to(dtype)
    return dict(case, q=q, tables=tables, lens=i32(lens), starts=starts, most=most, scale=1.0 / math.sqrt(dim),
                out=torch.zeros_like(q), **pools)


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _exponent(top):
    """The smallest e with top <= 448 * 2^e, at least LEAST (int32)."""
    m, k = torch.frexp(top)
    return torch.where(m <= 0.875, k - 9, k - 8).clamp(min=LEAST).where(top > 0, torch.full_like(k, LEAST))


def _parts(pool, dim):
    """Views of a pool's codes [NB][Hkv][D / 16][B][16] and scales [NB][Hkv][1]."""
    block, flat = pool.shape[2], pool.flatten(2)
    codes = flat[..., :block * dim].unflatten(-1, (dim // PANEL, block, PANEL))
    return codes, flat[..., block * dim:block * dim + 4].view(torch.float32)


def _put(codes, x):
    """fp32 [..., B, D], at most 448, to codes [..., D / 16, B, 16]."""
    codes.copy_(x.to(torch.float8_e4m3fn).view(torch.uint8).unflatten(-1, (-1, PANEL)).transpose(-3, -2))


def _rows_of(codes):
    """Codes [..., D / 16, B, 16] as fp32 [..., B, D]."""
    return codes.transpose(-3, -2).flatten(-2).contiguous().view(torch.float8_e4m3fn).float()


def _append(pool, st, x):
    """Rows [T][Hkv][D] behind each sequence's older tokens."""
    block, dim, width = st["block"], st["dim"], st["tables"].shape[1]
    starts, lens = st["starts"].long(), st["lens"].long()
    n = starts[1:] - starts[:-1]
    old = lens - n
    j = (old // block)[:, None] + torch.arange(st["most"] // block + 2, device=x.device)[None]     # [S][M]
    touched = (j * block < lens[:, None]) & (n > 0)[:, None]
    s, m = touched.nonzero(as_tuple=True)
    ids = st["tables"].long()[s, j[s, m].clamp(max=width - 1)]
    pos = (j[s, m] * block)[:, None] + torch.arange(block, device=x.device)[None]                  # [U][B]
    fresh = (pos >= old[s][:, None]) & (pos < lens[s][:, None])
    held = pos < old[s][:, None]
    row = torch.where(fresh, starts[s][:, None] + pos - old[s][:, None], torch.zeros_like(pos))
    new = x.float()[row].transpose(1, 2)                                                           # [U][Hkv][B][D]
    codes, scale = _parts(pool, dim)
    fresh, held = fresh[:, None, :, None], held[:, None, :, None]
    top = torch.where(fresh, new.abs(), torch.zeros_like(new)).amax((-1, -2))
    before = torch.frexp(scale[ids][..., 0])[1] - 1
    e = torch.maximum(_exponent(top), before.where(held.any(2)[..., 0], torch.full_like(before, LEAST)))
    was = _rows_of(codes[ids])
    now = torch.where(held, torch.ldexp(was, (before - e).clamp(min=-126)[..., None, None]),
                      torch.ldexp(new, -e[..., None, None]))
    out = torch.empty_like(codes[ids])
    _put(out, torch.where(held | fresh, now, was))
    codes[ids] = out
    scale[ids] = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)[..., None]


def _read(pool, slots, dim):
    codes, scale = _parts(pool, dim)
    block = pool.shape[2]
    c = codes[slots // block, :, :, slots % block].flatten(-2)
    return c.view(torch.float8_e4m3fn).float() * scale[slots // block]


def _sequences(pool, tables, dim):
    """The sequences' rows through their tables, fp32 [S][Hkv][width * B][D]."""
    codes, scale = _parts(pool, dim)
    ids = tables.long().clamp(min=0)
    x = codes[ids].permute(0, 2, 1, 4, 3, 5).flatten(4).view(torch.float8_e4m3fn).float()   # [S][Hkv][W][B][D]
    x *= scale[ids].transpose(1, 2)[..., None]
    return x.flatten(2, 3)


def _softmax(z, live):
    z = torch.where(live, z, torch.full_like(z, -math.inf))
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, torch.ones_like(total))


def _plain_pages(st):
    block, tables, shared, free = st["block"], st["tables"], st["shared"], st["free"]
    st["work"].copy_(st["kept"])
    lens, parents, count = st["lens"].long(), st["parents"].long(), st["count"].long()
    width, blocks = tables.shape[1], st["blocks"]
    j = torch.arange(width, device=lens.device)[None]
    # fork: whole blocks are shared, a started one gets a copy's block, first come, first served
    child = parents >= 0
    of = parents.clamp(min=0)
    full, part = lens[of] // block, child & (lens[of] % block > 0)
    need = part.long()
    go = child & ((need == 0) | (need.cumsum(0) <= count))
    need = need * go
    entries = tables[of].long()
    at = (count - need.cumsum(0)).clamp(min=0)
    opened = free[at].long()
    take = go[:, None] & (j < full[:, None])
    start = go[:, None] & part[:, None] & (j == full[:, None])
    last = entries.gather(1, full.clamp(max=width - 1)[:, None])[:, 0]
    st["pairs"].copy_(torch.where((go & part)[:, None], torch.stack([last, opened], 1), torch.zeros_like(st["pairs"]).long()))
    tables.copy_(torch.where(take, entries, torch.where(start, opened[:, None], tables.long())))
    holders = shared.long()
    holders += torch.bincount(torch.where(take, entries, torch.full_like(entries, blocks)).flatten(), minlength=blocks + 1)[:blocks]
    lens = torch.where(go, lens[of], lens)
    st["forked"].copy_(lens)
    count = count - need.sum()
    st["forked_count"].copy_(count)
    # release: the blocks past what each sequence keeps
    left = torch.minimum(lens, st["keep"].long())
    drop = (j >= ((left + block - 1) // block)[:, None]) & (j < ((lens + block - 1) // block)[:, None])
    entries = tables.long()
    times = torch.bincount(torch.where(drop, entries, torch.full_like(entries, blocks)).flatten(), minlength=blocks + 1)[:blocks]
    holders = holders - times
    freed = (times > 0) & (holders < 0)
    shared.copy_(holders.clamp(min=0))
    ids = freed.nonzero()[:, 0]
    free[count + torch.arange(len(ids), device=lens.device)] = ids.to(torch.int32)
    st["lens_out"].copy_(left)
    st["count_out"].copy_(count + len(ids))
    return tables, shared, free, st["pairs"], st["forked"], st["forked_count"], st["lens_out"], st["count_out"]


def _plain_cache(st):
    dtype, dim, slots = st["k"].dtype, st["dim"], st["slots"]
    _append(st["k_cache"], st, st["k"])
    _append(st["v_cache"], st, st["v"])
    at, keep = slots.clamp(min=0), (slots >= 0)[:, None, None]
    k, v = _read(st["k_cache"], at, dim).to(dtype), _read(st["v_cache"], at, dim).to(dtype)
    return torch.where(keep, k, st["k_out"]), torch.where(keep, v, st["v_out"])


def _plain_decode(st):
    q, dim, dtype = st["q"], st["dim"], st["q"].dtype
    x = q.float().unflatten(1, (st["kv_heads"], st["group"]))
    k = _sequences(st["k_cache"], st["tables"], dim)
    z = (x @ k.transpose(2, 3)) * st["scale"]
    del k
    live = torch.arange(z.shape[-1], device=z.device)[None] < st["lens"].long()[:, None]
    p = _softmax(z, live[:, None, None])
    return (p @ _sequences(st["v_cache"], st["tables"], dim)).flatten(1, 2).to(dtype)


def _plain_prefill(st):
    q, dim, dtype = st["q"], st["dim"], st["q"].dtype
    starts, lens = st["starts"].long(), st["lens"].long()
    n = starts[1:] - starts[:-1]
    j = torch.arange(st["most"], device=q.device)[None]
    inside = j < n[:, None]                                           # [S][most]
    rows = torch.where(inside, starts[:-1, None] + j, torch.zeros_like(j))
    x = q.float()[rows].unflatten(2, (st["kv_heads"], st["group"])).permute(0, 2, 3, 1, 4)
    k = _sequences(st["k_cache"], st["tables"], dim)[:, :, None]
    z = (x @ k.transpose(3, 4)) * st["scale"]                         # [S][Hkv][g][most][L]
    del k
    key = torch.arange(z.shape[-1], device=z.device)
    live = inside[..., None] & (key <= ((lens - n)[:, None] + j)[..., None])
    p = _softmax(z, live[:, None, None])
    del z
    o = (p @ _sequences(st["v_cache"], st["tables"], dim)[:, :, None]).permute(0, 3, 1, 2, 4).flatten(2, 3)
    out = torch.zeros_like(q)
    out[rows[inside]] = o[inside].to(dtype)
    return out


def run(state):
    kind = state["kind"]
    if not own:
        return {"pages": _plain_pages, "cache": _plain_cache, "decode": _plain_decode, "prefill": _plain_prefill}[kind](state)
    import paged_kv_cache_233_gb300 as pk
    st = state
    if kind == "pages":
        st["work"].copy_(st["kept"])      # the calls change these: every pass starts from the same step
        pk.paged_kv_fork(st["parents"], st["lens"], st["tables"], st["shared"], st["free"], st["count"], st["pairs"],
                         st["block"], st["forked"], st["forked_count"])
        pk.paged_kv_release(st["keep"], st["forked"], st["tables"], st["shared"], st["free"], st["forked_count"],
                            st["block"], st["lens_out"], st["count_out"])
        return (st["tables"], st["shared"], st["free"], st["pairs"], st["forked"], st["forked_count"], st["lens_out"],
                st["count_out"])
    if kind == "cache":
        pk.paged_kv_append_q8(st["k"], st["v"], st["tables"], st["starts"], st["lens"], st["k_cache"], st["v_cache"])
        pk.paged_kv_gather_q8(st["k_cache"], st["v_cache"], st["slots"], st["k_out"], st["v_out"])
        return st["k_out"], st["v_out"]
    if kind == "decode":
        if "workspace" not in st:     # a program makes it once, with its buffers
            st["workspace"] = pk.new_workspace(st["q"], st["tables"], st["block"], pk.PARTITION_BALANCED)
        pk.paged_attention_decode_q8(st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], st["scale"],
                                     st["out"], pk.PARTITION_BALANCED, st["workspace"])
        return st["out"]
    if "workspace" not in st:
        st["workspace"] = pk.prefill_workspace(st["q"])
    pk.paged_attention_prefill_q8(st["q"], st["k_cache"], st["v_cache"], st["tables"], st["starts"], st["lens"],
                                  st["scale"], st["out"], st["most"], workspace=st["workspace"], key_parts=0)
    return st["out"]


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    kind, block = case["kind"], case["block"]
    if kind == "pages":
        rows, mean = case["seqs"] + case["children"], case["context"] / 2
        forked = case["children"] * mean / block             # entries read, written, their holders read and written
        given = rows * mean / block / 3                      # entries read, their holders read and written
        back = given * case["seqs"] / max(1, rows)           # blocks that no one holds any more
        return {"bytes": 16.0 * forked + 12.0 * given + 4.0 * back + 36.0 * rows, "flops": 0.0}
    heads, dim = case["kv_heads"], case["dim"]
    held = 2.0 * heads * (dim + 4 / block)       # bytes of a token's K and V in 8 bits, its share of a scale's too
    half = 1.0 if case["seqs"] == 1 else 0.5     # a mean of evenly spaced lengths from 0, from half
    three = 1.0 if case["seqs"] == 1 else 0.75
    if kind == "cache":
        tokens = case["seqs"] * (case["chunk"] if case["chunk"] == 1 else three * case["chunk"])
        back = tokens + case["seqs"] * min((block - 1) / 2, half * case["cached"])
        row = 2.0 * heads * dim * 2
        return {"bytes": tokens * (row + held) + back * (row + held + 8), "flops": (tokens + back) * 2.0 * heads * dim * 2}
    q_heads = heads * case["group"]
    if kind == "decode":
        keys = case["longest"] if case["seqs"] == 1 else case["seqs"] * (case["shortest"] + case["longest"]) / 2
        return {"bytes": keys * (held + 4 / block) + case["seqs"] * 4.0 * q_heads * dim,
                "flops": 4.0 * keys * q_heads * dim}
    chunk, cached = three * case["chunk"], half * case["cached"]
    pairs = case["seqs"] * chunk * (cached + (chunk + 1) / 2)
    return {"bytes": case["seqs"] * ((chunk + cached) * held + chunk * 4.0 * q_heads * dim),
            "flops": 4.0 * pairs * q_heads * dim}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    def by_hand(st):
        block, lens, parents = st["block"], st["lens"].tolist(), st["parents"].tolist()
        tables, shared, free = st["tables"].tolist(), st["shared"].tolist(), st["free"].tolist()
        top = start = int(st["count"])
        pairs, asked, before = [[0, 0] for _ in lens], 0, list(lens)
        for s, of in enumerate(parents):
            if of < 0:
                continue
            whole, rest = divmod(before[of], block)
            if rest:
                asked += 1
                if asked > start:
                    continue
            for i in range(whole):
                tables[s][i] = tables[of][i]
                shared[tables[of][i]] += 1
            if rest:
                top -= 1
                tables[s][whole] = free[top]
                pairs[s] = [tables[of][whole], free[top]]
            lens[s] = before[of]
        forked, forked_count, freed = list(lens), top, set()
        for s, keep in enumerate(st["keep"].tolist()):
            n = min(keep, lens[s])
            for i in range(-(-n // block), -(-lens[s] // block)):
                b = tables[s][i]
                if shared[b] == 0:
                    freed.add(b)
                else:
                    shared[b] -= 1
            lens[s] = n
        for b in sorted(freed):
            free[top] = b
            top += 1
        i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
        return i32(tables), i32(shared), i32(free), i32(pairs), i32(forked), i32([forked_count]), i32(lens), i32([top])

    def value(codes):
        """What e4m3 bytes stand for, fp64."""
        c = codes.to(torch.int16)
        sign, e, m = 1.0 - 2.0 * (c // 128).double(), (c // 8 % 16).double(), (c % 8).double()
        x = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m * 2.0 ** -9)
        return sign * torch.where((e == 15) & (m == 7), torch.full_like(x, math.nan), x)

    def nearest(x):
        """fp64 values to the nearest that e4m3 has, ties to even, at most 448."""
        step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
        return (torch.round(x / step) * step).clamp(-448, 448)

    def held_rows(pool, ids, n, dim):
        """A sequence's first n rows as code values and their scales, fp64 [Hkv][n][D] and [Hkv][n][1], byte by byte."""
        _, heads, block, _ = pool.shape
        raw = pool[ids.long()].reshape(len(ids), heads, -1)
        c = value(raw[..., :block * dim]).reshape(len(ids), heads, dim // 16, block, 16).permute(1, 0, 3, 2, 4)
        s = raw[..., block * dim:block * dim + 4].contiguous().view(torch.float32).double()
        s = s.permute(1, 0, 2).expand(-1, -1, block)
        return c.reshape(heads, len(ids) * block, dim)[:, :n], s.reshape(heads, len(ids) * block, 1)[:, :n]

    def cache(st, pool, x):
        """Each slot's row after the step, gathered: fp64 [slots][Hkv][D]."""
        block, dim, heads, n_slots = st["block"], st["dim"], st["kv_heads"], st[pool].shape[0] * st["block"]
        grid = torch.zeros(n_slots, heads, dim, dtype=torch.float64, device=x.device)
        starts, lens = st["starts"].tolist(), st["lens"].tolist()
        for s, L in enumerate(lens):
            n = starts[s + 1] - starts[s]
            first = (L - n) // block * block
            ids = st["tables"][s, first // block:-(-L // block)]
            old, count = L - n - first, len(ids) * block
            rows = torch.zeros(heads, count, dim, dtype=torch.float64, device=x.device)
            rows[:, old:old + n] = x[starts[s]:starts[s] + n].double().transpose(0, 1)
            blocks = rows.reshape(heads, len(ids), block * dim).abs().amax(-1)
            e = torch.ceil(torch.log2(blocks.clamp(min=1e-300) / 448)).clamp(min=-64)
            e += (blocks > 448 * torch.exp2(e)).double()                   # (where the logarithm was rounded)
            e -= ((blocks <= 448 * torch.exp2(e - 1)) & (e > -64)).double()
            if old:
                c, scale = held_rows(st[pool], ids[:1], old, dim)
                e[:, 0] = torch.maximum(e[:, 0], torch.log2(scale[:, 0, 0]).round())
                rows[:, :old] = c * scale
            unit = torch.exp2(e)[:, :, None].expand(-1, -1, block).reshape(heads, count, 1)
            at = (ids.long()[:, None] * block + torch.arange(block, device=x.device)).flatten()
            grid[at] = (nearest(rows / unit) * unit).transpose(0, 1)
        live = (st["slots"] >= 0)[:, None, None]
        return torch.where(live, grid[st["slots"].clamp(min=0)], torch.zeros((), dtype=torch.float64, device=x.device))

    def attention(st):
        q, out = st["q"].double(), torch.zeros_like(st["q"], dtype=torch.float64)
        lens = st["lens"].tolist()
        starts = st["starts"].tolist() if st["starts"] is not None else list(range(len(lens) + 1))
        heads, group, block = st["kv_heads"], st["group"], st["block"]
        for s, n in enumerate(lens):
            a, b = starts[s], starts[s + 1]
            if n == 0 or a == b:
                continue
            ids = st["tables"][s, :-(-n // block)]
            k, v = (torch.mul(*held_rows(st[w], ids, n, st["dim"])) for w in ("k_cache", "v_cache"))
            seen = torch.arange(n, device=q.device)[None] <= torch.arange(n - (b - a), n, device=q.device)[:, None]
            for h in range(heads):
                for i in range(h * group, (h + 1) * group):
                    z = (q[a:b, i] @ k[h].T) * st["scale"]
                    w = torch.softmax(z.masked_fill(~seen, -math.inf), -1)
                    out[a:b, i] = w @ v[h]
        return out

    st = prepare(case, seed)
    if case["kind"] == "pages":
        return by_hand(st)
    if case["kind"] == "cache":
        return cache(st, "k_cache", st["k"]), cache(st, "v_cache", st["v"])
    return attention(st)
