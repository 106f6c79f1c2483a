"""The 4-bit cache on the GPU against its definition in 64 bits."""
import math

import pytest
import torch

import paged_kv_cache_233_gb300 as pk
import q4_support as q4

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pk.load()
    torch.cuda.set_device(0)
    pk.device_errors()


def rows(shape, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * spread).to(dtype)


def append(k, v, slots, kc, vc):
    a, b = kc.cuda(), vc.cuda()
    pk.paged_kv_append_q4(k.cuda(), v.cuda(), slots.cuda(), a, b)
    return a, b


# ------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("tokens,heads,dim,block", [(1, 1, 64, 8), (5, 3, 128, 8), (70, 8, 128, 16), (33, 5, 64, 32),
                                                    (200, 2, 64, 16), (17, 32, 128, 32)])
def test_append_bytes(dtype, tokens, heads, dim, block):
    blocks = -(-tokens // block) + 3
    g = torch.Generator().manual_seed(tokens)
    slots = torch.randperm(blocks * block, generator=g)[:tokens]
    slots[::7] = -1 if tokens > 1 else slots[::7]
    k, v = rows((tokens, heads, dim), dtype, 1), rows((tokens, heads, dim), dtype, 2, 30.0)
    kc, vc = q4.new_pool(blocks, heads, block, dim, 5), q4.new_pool(blocks, heads, block, dim, 6)
    gk, gv = append(k, v, slots, kc, vc)
    assert pk.device_errors() == 0
    q4.write(kc, slots, k)
    q4.write(vc, slots, v)
    # the same bytes everywhere, those of no token included (no element of
    # these inputs lies within 2^-20 of a border between two codes but ties)
    assert torch.equal(gk.cpu(), kc) and torch.equal(gv.cpu(), vc)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_append_borders_and_odd_groups(dtype):
    """Ties between codes, flat groups, tiny and huge scales, far middles, NaN and infinities."""
    big = torch.finfo(dtype).max
    tiny = torch.finfo(dtype).smallest_normal
    base = torch.arange(32).float()
    groups = [base, base / 2, base * 0, base * 0 - 7, (base % 16) * 0.5, (base % 2) * big * 0.4, base * tiny,
              (base % 3) * tiny / 64, 1000 + base % 5, -300 + (base % 2), (base % 16) - 7.5, base * 1e-3 - 4]
    nan, inf = base.clone(), base.clone()
    nan[9], inf[30] = float("nan"), float("inf")
    groups += [nan, inf, -inf, torch.full((32,), big), -torch.full((32,), big), (base - 15.5) * big / 15.5 / 2.1]
    x = torch.cat(groups).reshape(-1, 1, 64).to(dtype)
    n = x.shape[0]
    kc = q4.new_pool(2, 1, 16, 64, 1)
    gk, _ = append(x, x, torch.arange(n), kc, kc)
    q4.write(kc, torch.arange(n), x)
    codes, pairs = q4.views(kc, 64, dtype)
    gcodes, gpairs = q4.views(gk.cpu(), 64, dtype)
    same = (gpairs == pairs) | (gpairs.isnan() & pairs.isnan())
    assert bool(same[0, 0, :n].all())
    assert torch.equal(gcodes[0, 0, :, :n], codes[0, 0, :, :n])


def test_append_slot_past_the_pool_is_reported():
    x = rows((3, 2, 64), F16, 1)
    kc = q4.new_pool(2, 2, 8, 64, 1)
    gk, gv = append(x, x, torch.tensor([1 << 40, 16, -5]), kc, kc)
    assert pk.device_errors() == 1            # PAGEDKV_DEVERR_SLOT_RANGE
    assert torch.equal(gk.cpu(), kc) and torch.equal(gv.cpu(), kc)


# ------------------------------------------------------------------- gather
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("tokens,heads,dim,block", [(1, 1, 64, 8), (65, 3, 128, 16), (40, 8, 64, 32)])
def test_gather_rows(dtype, tokens, heads, dim, block):
    kc, vc, _ = q4.filled([tokens], heads, block, dim, dtype, 3)
    tables, _ = q4.tables_for([tokens], block, 3)
    slots = q4.sequence_slots(tables, 0, tokens, block)
    slots = torch.cat([slots, slots[:1], torch.tensor([-1]), slots[-1:], torch.tensor([1 << 35])])
    k = torch.full((len(slots), heads, dim), 7.0, dtype=dtype, device="cuda")
    v = torch.full_like(k, -3.0)
    pk.paged_kv_gather_q4(kc.cuda(), vc.cuda(), slots.cuda(), k, v)
    assert pk.device_errors() == 1
    live = (slots >= 0) & (slots < kc.shape[0] * block)
    assert bool((k[~live.cuda()] == 7).all()) and bool((v[~live.cuda()] == -3).all())
    for got, pool in ((k, kc), (v, vc)):
        ref = q4.read(pool, slots[live], dim, dtype)
        err = (got.cpu()[live].double() - ref).abs()
        # one rounding to the type of an fp32 sum (2^-24)
        assert bool((err <= ref.abs() * (q4.HALF_STEP[dtype] + 2.0 ** -24) + q4.TINY[dtype]).all())


# ------------------------------------------------------------------- decode
def decode(q, kc, vc, tables, lens, scale, part, out=None):
    out = torch.full_like(q, float("nan")).cuda() if out is None else out
    q, tables = q.cuda(), tables.cuda()
    ws = pk.new_workspace(q, tables, kc.shape[2], part)
    if ws is not None:
        ws.fill_(255)                          # NaN
    pk.paged_attention_decode_q4(q, kc.cuda(), vc.cuda(), tables, torch.tensor(lens, dtype=torch.int32).cuda(), scale, out,
                                 part, ws)
    return out


def check_decode(dtype, lens, heads, group, dim, block, part, seed=0, spread=1.0, scale=None):
    kc, vc, tables = q4.filled(lens, heads, block, dim, dtype, seed + 10, spread, pad=seed % 3)
    q = rows((len(lens), heads * group, dim), dtype, seed + 1)
    scale = dim ** -0.5 if scale is None else scale
    got = decode(q, kc, vc, tables, lens, scale, part)
    assert pk.device_errors() == 0
    ref = q4.attention(q, (kc, vc), tables, range(len(lens) + 1), lens, scale, dim, dtype)
    empty = [s for s, n in enumerate(lens) if n == 0]
    assert bool((got[empty] == 0).all())
    # the output is rounded, and the probabilities may be
    q4.assert_near(got, ref, dtype, 2, f"{dtype} lens {lens} part {part}")


LENS = [1, 0, 7, 8, 9, 31, 32, 33, 64, 65, 100, 257, 1000]


@pytest.mark.parametrize("part", [0, 32, 96, pk.PARTITION_BALANCED])
@pytest.mark.parametrize("dtype,heads,group,dim,block", [
    (F16, 8, 4, 128, 16), (BF16, 8, 4, 128, 16), (F16, 2, 8, 64, 8), (BF16, 4, 1, 64, 32), (F16, 1, 3, 128, 8),
    (BF16, 3, 7, 64, 16), (F16, 5, 2, 128, 32), (BF16, 16, 1, 128, 8), (F16, 6, 5, 64, 32)])
def test_decode(dtype, heads, group, dim, block, part):
    check_decode(dtype, LENS, heads, group, dim, block, part, seed=heads)


@pytest.mark.parametrize("part", [0, 512, pk.PARTITION_BALANCED])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_decode_long_and_short_together(dtype, part):
    check_decode(dtype, [9000, 3, 1, 4097], 8, 4, 128, 16, part, seed=2)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_decode_scales(dtype, scale):
    check_decode(dtype, [50, 129], 2, 4, 64, 16, pk.PARTITION_BALANCED, scale=scale)


@pytest.mark.parametrize("dtype,spread", [(F16, 1e-3), (F16, 300.0), (BF16, 1e-6), (BF16, 1e5)])
def test_decode_small_and_large_values(dtype, spread):
    """V of any size the type holds (K's size goes into the scale)."""
    check_decode(dtype, [40, 700], 4, 2, 128, 16, pk.PARTITION_BALANCED, spread=spread, scale=128 ** -0.5 / spread)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_decode_values_that_grow_along_the_context(dtype):
    """Scales and scores far larger late than early, and the other way round."""
    for up in (False, True):
        n, heads, dim, block = 600, 2, 128, 16
        tables, nb = q4.tables_for([n], block, 4)
        kc, vc = q4.new_pool(nb, heads, block, dim, 1), q4.new_pool(nb, heads, block, dim, 2)
        ramp = torch.logspace(-3, 3, n) if up else torch.logspace(3, -3, n)
        slots = q4.sequence_slots(tables, 0, n, block)
        q4.write_fast(kc, slots, (rows((n, heads, dim), torch.float32, 5) * ramp.sqrt()[:, None, None] * 0.3).to(dtype))
        q4.write_fast(vc, slots, (rows((n, heads, dim), torch.float32, 6) * ramp[:, None, None]).to(dtype))
        q = rows((1, heads * 4, dim), dtype, 7)
        for part in (0, 64, pk.PARTITION_BALANCED):
            got = decode(q, kc, vc, tables, [n], dim ** -0.5, part)
            ref = q4.attention(q, (kc, vc), tables, [0, 1], [n], dim ** -0.5, dim, dtype)
            q4.assert_near(got, ref, dtype, 2, f"up {up} part {part}")


def test_decode_reports_bad_blocks_and_lengths():
    kc, vc, tables = q4.filled([40, 40], 2, 16, 64, F16, 3)
    q = rows((2, 4, 64), F16, 1)
    bad = tables.clone()
    bad[1, 1] = 1 << 20
    for part in (0, 32, pk.PARTITION_BALANCED):
        decode(q, kc, vc, bad, [40, 40], 0.1, part)
        assert pk.device_errors() == 2                       # BLOCK_ID
        out = decode(q, kc, vc, tables, [1000, -3], 0.1, part)
        assert pk.device_errors() & 4                        # CONTEXT_LEN
        assert bool((out[1] == 0).all())


def test_decode_nan_in_a_context_is_nan_and_past_it_is_nothing():
    n = 21
    tables, nb = q4.tables_for([n, n], 16, 3)
    kc, vc = q4.new_pool(nb, 2, 16, 64, 1), q4.new_pool(nb, 2, 16, 64, 2)
    for s in range(2):
        for pool in (kc, vc):
            x = rows((n, 2, 64), F16, 5 + s)
            if s == 0:
                x[4, 1, 3] = float("inf")
            q4.write_fast(pool, q4.sequence_slots(tables, s, n, 16), x)
    out = decode(rows((2, 4, 64), F16, 1), kc, vc, tables, [n, n], 0.125, 0)
    assert bool(out[0, 2:].isnan().all()) and bool(torch.isfinite(out[0, :2]).all()) and bool(torch.isfinite(out[1]).all())


# ------------------------------------------------------------------ prefill
def check_prefill(dtype, cached, chunk, heads, group, dim, block, seed=0, extra=0, most=None, **kw):
    lens = [c + n for c, n in zip(cached, chunk)]
    kc, vc, tables = q4.filled(lens, heads, block, dim, dtype, seed + 20, pad=seed % 2)
    starts = torch.tensor([0] + chunk).cumsum(0).to(torch.int32)
    total = int(starts[-1])
    q = rows((total + extra, heads * group, dim), dtype, seed + 3)
    out = torch.full_like(q, 5.0).cuda()
    pk.paged_attention_prefill_q4(q.cuda(), kc.cuda(), vc.cuda(), tables.cuda(), starts.cuda(),
                                  torch.tensor(lens, dtype=torch.int32).cuda(), dim ** -0.5, out, most, **kw)
    assert pk.device_errors() == 0
    assert bool((out[total:] == 5).all())
    ref = q4.attention(q[:total], (kc, vc), tables, starts, lens, dim ** -0.5, dim, dtype)
    # the output, the probabilities, and K and V as the tensor cores take them
    q4.assert_near(out[:total], ref, dtype, 4, f"{dtype} cached {cached} chunk {chunk}")


@pytest.mark.parametrize("parts", [1, 0, 2, 32])
@pytest.mark.parametrize("dtype,heads,group,dim,block", [
    (F16, 8, 4, 128, 16), (BF16, 2, 8, 128, 32), (F16, 1, 1, 64, 8), (BF16, 4, 3, 64, 16), (F16, 2, 6, 128, 8),
    (BF16, 1, 16, 64, 32), (F16, 1, 64, 128, 16), (BF16, 3, 7, 128, 16)])
def test_prefill(dtype, heads, group, dim, block, parts):
    check_prefill(dtype, [0, 5, 300, 64, 0], [1, 40, 17, 0, 130], heads, group, dim, block, seed=heads, extra=3,
                  key_parts=parts)


@pytest.mark.parametrize("parts", [1, 0])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_prefill_long_context(dtype, parts):
    check_prefill(dtype, [5000, 0], [70, 600], 2, 4, 128, 16, seed=3, key_parts=parts)


def test_prefill_single_tokens_equal_decode():
    lens = [1, 50, 700]
    kc, vc, tables = q4.filled(lens, 4, 16, 128, BF16, 8)
    q = rows((3, 16, 128), BF16, 9)
    a = decode(q, kc, vc, tables, lens, 0.09, 0)
    b = torch.zeros_like(a)
    pk.paged_attention_prefill_q4(q.cuda(), kc.cuda(), vc.cuda(), tables.cuda(), torch.arange(4, dtype=torch.int32).cuda(),
                                  torch.tensor(lens, dtype=torch.int32).cuda(), 0.09, b)
    ref = q4.attention(q, (kc, vc), tables, range(4), lens, 0.09, 128, BF16)
    for got in (a, b):
        q4.assert_near(got, ref, BF16, 4)


def test_prefill_reports_bad_sequences_and_leaves_their_rows():
    lens = [40, 40, 40]
    kc, vc, tables = q4.filled(lens, 2, 16, 64, F16, 3)
    q = rows((30, 4, 64), F16, 1).cuda()
    starts = torch.tensor([0, 10, 20, 30], dtype=torch.int32).cuda()

    def run(lens, most=10, tab=tables):
        out = torch.full_like(q, 5.0)
        pk.paged_attention_prefill_q4(q, kc.cuda(), vc.cuda(), tab.cuda(), starts,
                                      torch.tensor(lens, dtype=torch.int32).cuda(), 0.1, out, most)
        return out, pk.device_errors()

    out, err = run([40, 3, 40])                  # shorter than its chunk
    assert err == 4 and bool((out[10:20] == 5).all()) and not bool((out[:10] == 5).any())
    out, err = run([40, 40, 4000])               # past its table
    assert err == 4 and bool((out[20:] == 5).all())
    bad = tables.clone()
    bad[0, 0] = -7
    assert run(lens, tab=bad)[1] == 2            # BLOCK_ID


# ---------------------------------------------------- blocks, streams, graphs
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_blocks_copy_and_swap(dtype):
    kc, vc, _ = q4.filled([64], 3, 8, 64, dtype, 1)
    a, b = kc.cuda(), vc.cuda()
    pk.paged_kv_copy_blocks(a, b, torch.tensor([[0, 9], [3, 8]], dtype=torch.int32).cuda())
    kc[9], vc[9], kc[8], vc[8] = kc[0], vc[0], kc[3], vc[3]
    assert torch.equal(a.cpu(), kc) and torch.equal(b.cpu(), vc)
    hk, hv = torch.zeros_like(kc[:2]).pin_memory(), torch.zeros_like(vc[:2]).pin_memory()
    pk.paged_kv_swap_blocks(a, b, hk, hv, torch.tensor([[5, 1]], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert torch.equal(hk[1], kc[5]) and torch.equal(hv[1], vc[5])
    pk.paged_kv_swap_blocks(hk, hv, a, b, torch.tensor([[1, 2]], dtype=torch.int32).cuda())
    assert torch.equal(a[2].cpu(), kc[5])
    assert pk.device_errors() == 0


def step_state(dtype=BF16, heads=4, group=2, dim=128, block=16, steps=6):
    """Requests of a serving loop: lengths, tables, free stack, pools."""
    lens = [0, 15, 16, 100, 31]
    tables, nb = q4.tables_for(lens, block, 5, spare=24, pad=4)
    used = set(tables[tables >= 0].tolist())
    free = torch.tensor([i for i in range(nb) if i not in used], dtype=torch.int32)
    return lens, tables, nb, free


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_serving_loop(dtype, graph):
    """build_tables, append, decode and prefill together, step after step, on a
    side stream and captured: each step adds tokens, and its attention is that
    of a cache written and read by the definition."""
    heads, group, dim, block = 4, 2, 128, 16
    lens, tables, nb, free = step_state()
    S, steps, most = len(lens), 5, 4
    kc, vc = q4.new_pool(nb, heads, block, dim, 1), q4.new_pool(nb, heads, block, dim, 2)
    for s, n in enumerate(lens):
        for i, pool in enumerate((kc, vc)):
            q4.write_fast(pool, q4.sequence_slots(tables, s, n, block), rows((n, heads, dim), dtype, 10 * s + i))
    dev = dict(device="cuda", dtype=torch.int32)
    gk, gv, gt, gfree = kc.cuda(), vc.cuda(), tables.cuda(), free.cuda()
    ctx, count = torch.tensor(lens, **dev), torch.tensor([len(free)], **dev)
    new, T = torch.zeros(S, **dev), S * most
    starts, seq, pos = torch.zeros(S + 1, **dev), torch.zeros(T, **dev), torch.zeros(T, **dev)
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")
    k, v = torch.zeros(T, heads, dim, dtype=dtype, device="cuda"), torch.zeros(T, heads, dim, dtype=dtype, device="cuda")
    q = torch.zeros(T, heads * group, dim, dtype=dtype, device="cuda")
    qd = torch.zeros(S, heads * group, dim, dtype=dtype, device="cuda")
    out, outd = torch.zeros_like(q), torch.zeros_like(qd)
    ws = pk.new_workspace(qd, gt, block, pk.PARTITION_BALANCED)
    wp = pk.prefill_workspace(q)

    def step():
        pk.paged_kv_build_tables(new, ctx, gt, gfree, count, block, nb, starts, seq, pos, slots)
        pk.paged_kv_append_q4(k, v, slots, gk, gv)
        pk.paged_attention_prefill_q4(q, gk, gv, gt, starts, ctx, dim ** -0.5, out, most, workspace=wp, key_parts=0)
        pk.paged_attention_decode_q4(qd, gk, gv, gt, ctx, dim ** -0.5, outd, pk.PARTITION_BALANCED, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = None
    if graph:
        # a first pass with nothing to add leaves the state as it is
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
    now = list(lens)
    for i in range(steps):
        add = [(s + i) % (most + 1) for s in range(S)]
        x = [rows((T, heads, dim), dtype, 100 + 3 * i + j) for j in range(2)]
        y, z = rows(q.shape, dtype, 300 + i), rows(qd.shape, dtype, 400 + i)
        torch.cuda.synchronize()
        new.copy_(torch.tensor(add, dtype=torch.int32))
        k.copy_(x[0]), v.copy_(x[1]), q.copy_(y), qd.copy_(z)
        torch.cuda.synchronize()
        if graph:
            g.replay()
        else:
            with torch.cuda.stream(side):
                step()
        torch.cuda.synchronize()
        assert pk.device_errors() == 0
        st = [0]
        for s in range(S):
            n = add[s]
            now[s] += n
            st.append(st[-1] + n)
        assert ctx.tolist() == now and starts.tolist() == st
        t = gt.cpu()
        for s in range(S):
            at = q4.sequence_slots(t, s, now[s], block)[now[s] - add[s]:]
            assert torch.equal(slots[st[s]:st[s + 1]].cpu(), at)
            for pool, rowsx in ((kc, x[0]), (vc, x[1])):
                q4.write(pool, at, rowsx[st[s]:st[s + 1]])
        ref = q4.attention(y[:st[-1]], (kc, vc), t, st, now, dim ** -0.5, dim, dtype)
        q4.assert_near(out[:st[-1]], ref, dtype, 4, f"prefill step {i}")
        ref = q4.attention(z, (kc, vc), t, range(S + 1), now, dim ** -0.5, dim, dtype)
        q4.assert_near(outd, ref, dtype, 2, f"decode step {i}")
    held = t[t >= 0].tolist()
    assert len(set(held)) == len(held)
    assert int(count) == nb - len(held)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gather_into_a_16_bit_pool(dtype):
    """A 4-bit sequence moved into 16-bit pools: paged_kv_append_tokens right behind
    the gather that makes its rows, many times over."""
    n, heads, dim, block = 3000, 8, 128, 16
    kc, vc, tables = q4.filled([n], heads, block, dim, dtype, 5)
    slots = q4.sequence_slots(tables, 0, n, block).cuda()
    gk, gv, gt = kc.cuda(), vc.cuda(), tables.cuda()
    seq, pos = torch.zeros(n, dtype=torch.int32).cuda(), torch.arange(n, dtype=torch.int32).cuda()
    want = [q4.read(p, slots.cpu(), dim, dtype) for p in (kc, vc)]
    for i in range(5):
        k, v = (torch.full((n, heads, dim), float(i), dtype=dtype, device="cuda") for _ in range(2))
        k16, v16 = (torch.zeros(kc.shape[0], block, heads, dim, dtype=dtype, device="cuda") for _ in range(2))
        torch.cuda.synchronize()
        pk.paged_kv_gather_q4(gk, gv, slots, k, v)
        pk.paged_kv_append_tokens(k, v, gt, seq, pos, k16, v16)
        torch.cuda.synchronize()
        for pool, ref in ((k16, want[0]), (v16, want[1])):
            err = (pool.flatten(0, 1)[slots].cpu().double() - ref).abs()
            assert bool((err <= ref.abs() * (q4.HALF_STEP[dtype] + 2.0 ** -24) + q4.TINY[dtype]).all())


def test_pools_past_4_gib():
    """Blocks whose bytes lie past 2^32 in their pool."""
    heads, dim, block, dtype = 8, 128, 32, BF16
    head_bytes = block * dim * 5 // 8
    nb = (1 << 32) // (heads * head_bytes) + 40
    pools = [pk.new_q4_pool(nb, heads, block, dim) for _ in range(2)]
    lens = [300, 70]
    tables = torch.tensor([[nb - 1 - 2 * j for j in range(10)], [nb - 2 - 2 * j if j < 3 else -1 for j in range(10)]],
                          dtype=torch.int32)
    small = [q4.new_pool(40, heads, block, dim, i) for i in range(2)]      # the pools' last 40 blocks
    near = torch.where(tables >= 0, tables - (nb - 40), tables)
    slots = torch.cat([q4.sequence_slots(tables, s, n, block) for s, n in enumerate(lens)])
    near_slots = torch.cat([q4.sequence_slots(near, s, n, block) for s, n in enumerate(lens)])
    k, v = rows((370, heads, dim), dtype, 1), rows((370, heads, dim), dtype, 2)
    for pool, x in zip(small, (k, v)):
        q4.write_fast(pool, near_slots, x)
    for pool in pools:
        pool[nb - 40:] = 255
    pk.paged_kv_append_q4(k.cuda(), v.cuda(), slots.cuda(), *pools)
    back = [torch.zeros(370, heads, dim, dtype=dtype, device="cuda") for _ in range(2)]
    pk.paged_kv_gather_q4(*pools, slots.cuda(), *back)
    for got, pool in zip(back, small):
        ref = q4.read(pool, near_slots, dim, dtype)
        assert bool(((got.cpu().double() - ref).abs() <= ref.abs() * 2.0 ** -8 * 1.01).all())
    q = rows((2, heads * 4, dim), dtype, 3)
    ref = q4.attention(q, small, near, range(3), lens, 0.09, dim, dtype)
    for part in (0, pk.PARTITION_BALANCED):
        q4.assert_near(decode(q, pools[0], pools[1], tables, lens, 0.09, part), ref, dtype, 2)
    qp = rows((370, heads * 4, dim), dtype, 4)
    starts = torch.tensor([0, 300, 370], dtype=torch.int32)
    out = torch.zeros_like(qp).cuda()
    pk.paged_attention_prefill_q4(qp.cuda(), *pools, tables.cuda(), starts.cuda(),
                                  torch.tensor(lens, dtype=torch.int32).cuda(), 0.09, out, 300)
    q4.assert_near(out, q4.attention(qp, small, near, starts, lens, 0.09, dim, dtype), dtype, 4)
    assert pk.device_errors() == 0


def test_decode_4096_sequences():
    rng = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 40, (4096,), generator=rng).tolist()
    for heads, group, dim in ((4, 2, 128), (1, 1, 64)):
        kc, vc, tables = q4.filled(lens, heads, 8, dim, BF16, 6)
        q = rows((4096, heads * group, dim), BF16, 7)
        ref = q4.attention(q, (kc, vc), tables, range(4097), lens, dim ** -0.5, dim, BF16)
        for part in (0, 32, pk.PARTITION_BALANCED):
            q4.assert_near(decode(q, kc, vc, tables, lens, dim ** -0.5, part), ref, BF16, 2)
        assert pk.device_errors() == 0


def test_two_streams_with_a_workspace_each():
    lens, heads, dim, block = [2000, 700, 31], 4, 128, 16
    kc, vc, tables = q4.filled(lens, heads, block, dim, BF16, 4)
    gk, gv, gt = kc.cuda(), vc.cuda(), tables.cuda()
    L = torch.tensor(lens, dtype=torch.int32).cuda()
    qs = [rows((3, heads * 2, dim), BF16, 20 + i).cuda() for i in range(2)]
    outs = [torch.zeros_like(q) for q in qs]
    ws = [pk.new_workspace(q, gt, block, pk.PARTITION_BALANCED) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(40):
        s = i % 2
        pk.paged_attention_decode_q4(qs[s], gk, gv, gt, L, 0.09, outs[s], pk.PARTITION_BALANCED, ws[s], stream=streams[s])
    torch.cuda.synchronize()
    for q, out in zip(qs, outs):
        q4.assert_near(out, q4.attention(q.cpu(), (kc, vc), tables, range(4), lens, 0.09, dim, BF16), BF16, 2)


def test_refusals_on_the_gpu():
    kc, vc, tables = (t.cuda() for t in q4.filled([20], 2, 16, 64, F16, 1))
    q, L = torch.zeros(1, 4, 64, dtype=F16, device="cuda"), torch.tensor([20], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    with pytest.raises(pk.PagedKVError, match="contiguous"):
        pk.paged_attention_decode_q4(q.transpose(1, 2).contiguous().transpose(1, 2), kc, vc, tables, L, 0.1, out)
    with pytest.raises(pk.PagedKVError, match="out must be"):
        pk.paged_attention_decode_q4(q, kc, vc, tables, L, 0.1, out.bfloat16())
    with pytest.raises(pk.PagedKVError, match="current device"):
        pk.paged_attention_decode_q4(q, kc, vc, tables.cpu(), L, 0.1, out)
    with pytest.raises(pk.PagedKVError, match="block_tables must be"):
        pk.paged_attention_decode_q4(q, kc, vc, tables.long(), L, 0.1, out)
    with pytest.raises(pk.PagedKVError, match="unsupported"):
        pk.paged_attention_decode_q4(q.float(), kc, vc, tables, L, 0.1, out.float())
    with pytest.raises(pk.PagedKVError, match="workspace"):
        pk.paged_attention_decode_q4(q, kc, vc, tables, L, 0.1, out, 32)
    with pytest.raises(TypeError):
        pk.paged_attention_decode_q4(q, kc, vc, tables, [20], 0.1, out)
    pk.paged_attention_decode_q4(q[:0], kc, vc, tables[:0], L[:0], 0.1, out[:0])
    with pytest.raises(pk.PagedKVError, match="workspace"):
        pk.paged_attention_prefill_q4(q, kc, vc, tables, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), L, 0.1,
                                      out, 1, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"), key_parts=4)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_decode_shared_prefixes_in_a_call_past_l2(dtype):
    """Sequences that hold the same blocks, in their order or another, in a call that
    reads more than the L2 holds."""
    heads, dim, block, n, S = 8, 128, 16, 30000, 4
    kc, vc, tables = q4.filled([n], heads, block, dim, dtype, 9)
    tables = tables.repeat(S, 1)
    tables[3] = tables[3].flip(0)
    q = rows((S, heads, dim), dtype, 2)
    lens = [n, n - 7, 12345, n]
    ref = q4.attention(q, (kc, vc), tables, range(S + 1), lens, dim ** -0.5, dim, dtype)
    for part in (0, 2048, pk.PARTITION_BALANCED):
        q4.assert_near(decode(q, kc, vc, tables, lens, dim ** -0.5, part), ref, dtype, 2, f"part {part}")
    assert pk.device_errors() == 0


@pytest.mark.parametrize("heads, dim, block", [(32, 64, 8), (2, 128, 32), (3, 64, 16)])
def test_decode_short_sequences_beside_long_ones(heads, dim, block):
    """A balanced split over sequences of one or two tiles, empty ones and a few long
    ones, in an order that ends shares inside, before and behind each of them."""
    lens = [(5000, 0, 1, 32, 33, 64, 700, 31)[(3 * i + i // 8) % 8] for i in range(150)]
    kc, vc, tables = q4.filled(lens, heads, block, dim, F16, 4)
    q = rows((len(lens), heads, dim), F16, 6)
    ref = q4.attention(q, (kc, vc), tables, range(len(lens) + 1), lens, dim ** -0.5, dim, F16)
    q4.assert_near(decode(q, kc, vc, tables, lens, dim ** -0.5, pk.PARTITION_BALANCED), ref, F16, 2, "short and long")
    assert pk.device_errors() == 0
