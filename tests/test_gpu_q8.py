"""The 8-bit cache on the GPU against its definition in 64 bits."""
import math

import pytest
import torch

import paged_kv_cache_233_gb300 as pk
import q8_support as q8

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


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def append(k, v, tables, starts, lens, kc, vc):
    a, b = kc.cuda(), vc.cuda()
    pk.paged_kv_append_q8(k.cuda(), v.cuda(), tables.cuda(), i32(starts), i32(lens), a, b)
    return a, b


def same_pool(got, want, dim):
    """Codes, scales and marks of every block; the bytes behind them are nobody's."""
    return all(torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
               for a, b in zip(q8.views(got.cpu(), dim), q8.views(want, dim)))


# ------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("cached,chunk,heads,dim,block", [
    ([0], [1], 1, 64, 8), ([5, 0, 7, 8, 9], [3, 9, 1, 8, 0], 3, 128, 8), ([0, 33, 15], [70, 0, 2], 8, 128, 16),
    ([3, 31, 32, 64], [30, 1, 1, 33], 5, 64, 32), ([100] * 9, [1] * 9, 2, 64, 16), ([16, 1], [17, 200], 32, 128, 32),
    ([2], [600], 4, 64, 8)])
def test_append_bytes(dtype, cached, chunk, heads, dim, block):
    lens = [c + n for c, n in zip(cached, chunk)]
    tables, nb = q8.tables_for(lens, block, 7, pad=2)
    starts = torch.tensor([0] + chunk).cumsum(0)
    T = int(starts[-1])
    kc, vc = q8.new_pool(nb, heads, block, dim, 5), q8.new_pool(nb, heads, block, dim, 6)
    for pool, spread in ((kc, 0.7), (vc, 20.0)):
        for s, n in enumerate(cached):
            q8.fill(pool, tables[s], rows((n, heads, dim), dtype, 10 * s + 1, spread))
    # padding behind the last sequence's rows; rows of very different sizes
    size = torch.exp2(torch.arange(T + 3) % 7 - 3.0)[:, None, None]
    k, v = (rows((T + 3, heads, dim), torch.float32, 2 + i) * size for i in range(2))
    k, v = k.to(dtype), (30 * v).to(dtype)
    gk, gv = append(k, v, tables, starts, lens, kc, vc)
    assert pk.device_errors() == 0
    q8.append(kc, k, tables, starts, lens)
    q8.append(vc, v, tables, starts, lens)
    assert same_pool(gk, kc, dim) and same_pool(gv, vc, dim)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_append_one_by_one_and_growing(dtype):
    """A token at a time, each larger than the one before, then small ones, then zeros."""
    n, heads, dim, block = 40, 2, 64, 16
    tables, nb = q8.tables_for([n], block, 3)
    kc, vc = q8.new_pool(nb, heads, block, dim, 1), q8.new_pool(nb, heads, block, dim, 2)
    gk, gv = kc.cuda(), vc.cuda()
    size = torch.exp2(torch.tensor([-12.0 + i % 20 for i in range(n)]))
    size[25:30] = 0
    x = (rows((n, heads, dim), torch.float32, 4) * size[:, None, None]).to(dtype)
    for t in range(n):
        pk.paged_kv_append_q8(x[t:t + 1].cuda(), -x[t:t + 1].cuda(), tables.cuda(), i32([0, 1]), i32([t + 1]), gk, gv)
        q8.append(kc, x[t:t + 1], tables, [0, 1], [t + 1])
        q8.append(vc, -x[t:t + 1], tables, [0, 1], [t + 1])
        assert same_pool(gk, kc, dim) and same_pool(gv, vc, dim), t
    assert pk.device_errors() == 0


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_append_borders_and_odd_rows(dtype):
    """Ties between codes, zeros, signed zeros, tiny and huge values, largest values
    at the border of a power of two, NaN and infinities."""
    top, tiny = torch.finfo(dtype).max, torch.finfo(dtype).tiny
    base = torch.arange(64).float()
    odd = [base * 0, -base * 0, base * top / 63, -base * top / 63, base * tiny, base * tiny / 64, 448 - base, base + 385,
           448.0 + 2 * base, (base - 32) / 64, (base % 32 + 16.5) / 8, base * 2.0 ** -9, (base + 0.5) * 2.0 ** -9,
           (base - 20) * 1e-3, base % 2 * 57344.0, torch.full((64,), top)]
    nan, inf = base.clone(), base.clone()
    nan[9], inf[30] = math.nan, math.inf
    odd += [nan, -nan, inf, -inf, torch.full((64,), math.nan), torch.full((64,), math.inf)]
    x = torch.stack(odd).to(dtype)[:, None]                        # one row each
    block, S = 8, len(odd)
    tables, nb = q8.tables_for([1] * S, block, 3)
    kc = q8.new_pool(nb, 1, block, 64, 1)
    gk, _ = append(x, x, tables, torch.arange(S + 1), [1] * S, kc, kc)
    q8.append(kc, x, tables, torch.arange(S + 1), [1] * S)
    assert same_pool(gk, kc, 64)
    # the same rows in shared blocks
    tables, nb = q8.tables_for([S], 32, 3)
    kc = q8.new_pool(nb, 1, 32, 64, 1)
    gk, _ = append(x, x, tables, [0, S], [S], kc, kc)
    q8.append(kc, x, tables, [0, S], [S])
    assert same_pool(gk, kc, 64)
    assert pk.device_errors() == 0


def test_append_reports_bad_sequences_and_leaves_their_blocks():
    block, heads, dim = 16, 2, 64
    tables, nb = q8.tables_for([40, 40, 40], block, 3)
    x = rows((30, heads, dim), F16, 1)
    kc = q8.new_pool(nb, heads, block, dim, 1)
    q8.views(kc, dim)[1].fill_(2.0 ** -9)

    def run(starts, lens, tab=tables, skip=()):
        want, starts = kc.clone(), torch.tensor(starts)
        gk, _ = append(x, x, tab, starts, lens, kc, kc)
        err = pk.device_errors()
        for s in range(3):
            if s not in skip:
                one = torch.tensor([0, int(starts[s + 1] - starts[s])])
                q8.append(want, x[int(starts[s]):int(starts[s + 1])], tables[s:s + 1], one, [lens[s]])
        assert same_pool(gk, want, dim)
        return err

    assert run([0, 10, 20, 30], [40, 40, 40]) == 0
    assert run([0, 10, 20, 30], [40, 3, 40], skip=[1]) == 4          # CONTEXT_LEN: shorter than its chunk
    assert run([0, 10, 20, 30], [40, 40, 4000], skip=[2]) == 4       # past its table
    assert run([0, 10, 20, 31], [40, 40, 40], skip=[2]) == 8         # POSITION: rows past the call's
    bad = tables.clone()
    bad[1] = -7
    assert run([0, 10, 20, 30], [40, 40, 40], bad, skip=[1]) == 2    # BLOCK_ID


def test_append_many_sequences():
    """4096 sequences, most of them without rows."""
    S, block = 4096, 8
    n = [(s * 7 + 3) % 11 % 3 if s % 5 == 0 else 0 for s in range(S)]
    old = [s % 9 for s in range(S)]
    lens = [a + b for a, b in zip(n, old)]
    tables, nb = q8.tables_for(lens, block, 3)
    starts = torch.tensor([0] + n).cumsum(0)
    kc = torch.zeros(nb, 1, block, 64 + q8.tail(block), dtype=torch.uint8)
    q8.views(kc, 64)[1].fill_(2.0 ** -9)
    x = rows((int(starts[-1]), 1, 64), BF16, 1)
    gk, _ = append(x, x, tables, starts, lens, kc, kc)
    q8.append(kc, x, tables, starts, lens)
    assert same_pool(gk, kc, 64) and pk.device_errors() == 0


# ------------------------------------------------------------------- gather
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("tokens,heads,dim,block", [(1, 1, 64, 8), (65, 3, 128, 16), (40, 8, 64, 32)])
def test_gather_rows(dtype, tokens, heads, dim, block):
    kc, vc, tables = q8.filled([tokens], heads, block, dim, dtype, 3)
    slots = q8.sequence_slots(tables, 0, tokens, block)
    slots = torch.cat([slots, slots[:1], torch.tensor([-1]), slots[-1:], torch.tensor([1 << 35])])
    k = torch.full((len(slots), heads, dim), 7.0, dtype=dtype, device="cuda")
    v = torch.full_like(k, -3.0)
    pk.paged_kv_gather_q8(kc.cuda(), vc.cuda(), slots.cuda(), k, v)
    assert pk.device_errors() == 1
    live = (slots >= 0) & (slots < kc.shape[0] * block)
    assert bool((k[~live.cuda()] == 7).all()) and bool((v[~live.cuda()] == -3).all())
    for got, pool in ((k, kc), (v, vc)):
        # four significant bits: nothing is rounded
        assert torch.equal(got.cpu()[live].double(), q8.read(pool, slots[live], dim))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gather_of_the_largest_values_is_finite(dtype):
    top = torch.finfo(dtype).max
    x = torch.full((1, 1, 64), top).to(dtype)
    x[0, 0, 1], x[0, 0, 2], x[0, 0, 3] = -top, math.nan, 0
    tables, nb = q8.tables_for([1], 8, 1)
    gk, gv = append(x, x, tables, [0, 1], [1], *(q8.new_pool(nb, 1, 8, 64),) * 2)
    k, v = torch.zeros_like(x).cuda(), torch.zeros_like(x).cuda()
    pk.paged_kv_gather_q8(gk, gv, torch.tensor([int(tables[0, 0]) * 8]).cuda(), k, v)
    for got in (k.cpu()[0, 0], v.cpu()[0, 0]):
        assert float(got[0]) == top and float(got[1]) == -top and bool(got[2].isnan()) and float(got[3]) == 0


# ------------------------------------------------------------------- decode
def decode(q, kc, vc, tables, lens, scale, part, out=None):
    out = torch.full_like(q, float("nan")).cuda() if out is None else out
    q, tables = q.cuda(), tables.cuda()
    ws = pk.new_workspace(q, tables, kc.shape[2], part)
    if ws is not None:
        ws.fill_(255)                          # NaN
    pk.paged_attention_decode_q8(q, kc.cuda(), vc.cuda(), tables, i32(lens), scale, out, part, ws)
    return out


def check_decode(dtype, lens, heads, group, dim, block, part, seed=0, spread=1.0, scale=None):
    kc, vc, tables = q8.filled(lens, heads, block, dim, dtype, seed + 10, spread, pad=seed % 3)
    q = rows((len(lens), heads * group, dim), dtype, seed + 1)
    scale = dim ** -0.5 if scale is None else scale
    got = decode(q, kc, vc, tables, lens, scale, part)
    assert pk.device_errors() == 0
    ref = q8.attention(q, (kc, vc), tables, range(len(lens) + 1), lens, scale, dim)
    empty = [s for s, n in enumerate(lens) if n == 0]
    assert bool((got[empty] == 0).all())
    # the output is rounded, and the probabilities (to fp16, the finer of the types)
    q8.assert_near(got, ref, dtype, 2, f"{dtype} lens {lens} part {part}")


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


@pytest.mark.parametrize("dtype,spread", [(F16, 1e-3), (F16, 300.0), (BF16, 1e-6), (BF16, 1e-17), (BF16, 1e5), (BF16, 1e19)])
def test_decode_small_and_large_values(dtype, spread):
    """V of any size (K's size goes into the scale)."""
    check_decode(dtype, [40, 700], 4, 2, 128, 16, pk.PARTITION_BALANCED, spread=spread, scale=128 ** -0.5 / spread)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_decode_values_that_grow_along_the_context(dtype):
    """Scales and scores far larger late than early, and the other way round."""
    for up in (False, True):
        n, heads, dim, block = 600, 2, 128, 16
        tables, nb = q8.tables_for([n], block, 4)
        kc, vc = q8.new_pool(nb, heads, block, dim, 1), q8.new_pool(nb, heads, block, dim, 2)
        ramp = torch.logspace(-3, 3, n) if up else torch.logspace(3, -3, n)
        q8.fill(kc, tables[0], (rows((n, heads, dim), torch.float32, 5) * ramp.sqrt()[:, None, None] * 0.3).to(dtype))
        q8.fill(vc, tables[0], (rows((n, heads, dim), torch.float32, 6) * ramp[:, None, None]).to(dtype))
        q = rows((1, heads * 4, dim), dtype, 7)
        for part in (0, 64, pk.PARTITION_BALANCED):
            got = decode(q, kc, vc, tables, [n], dim ** -0.5, part)
            ref = q8.attention(q, (kc, vc), tables, [0, 1], [n], dim ** -0.5, dim)
            q8.assert_near(got, ref, dtype, 2, f"up {up} part {part}")


def test_decode_reports_bad_blocks_and_lengths():
    kc, vc, tables = q8.filled([40, 40], 2, 16, 64, F16, 3)
    q = rows((2, 4, 64), F16, 1)
    bad = tables.clone()
    bad[1, 1] = 1 << 20
    for part in (0, 32, pk.PARTITION_BALANCED):
        decode(q, kc, vc, bad, [40, 40], 0.1, part)
        assert pk.device_errors() == 2                       # BLOCK_ID
        out = decode(q, kc, vc, tables, [1000, -3], 0.1, part)
        assert pk.device_errors() & 4                        # CONTEXT_LEN
        assert bool((out[1] == 0).all())


@pytest.mark.parametrize("operand", ["q", "k", "v"])
def test_decode_nan_in_a_context_is_nan_and_past_it_is_nothing(operand):
    n, heads, dim, block = 21, 2, 64, 16
    tables, nb = q8.tables_for([n, n], block, 3)
    kc, vc = (torch.full((nb, heads, block, dim + 1), 0xFF, dtype=torch.uint8) for _ in range(2))   # NaN codes and scales
    for s in range(2):
        for name, pool in (("k", kc), ("v", vc)):
            x = rows((n, heads, dim), F16, 5 + s)
            if s == 0 and name == operand:
                x[4, 1, 3] = float("inf")
            q8.fill(pool, tables[s], x.nan_to_num(posinf=0.0))
            if s == 0 and name == operand:
                q8.views(pool, dim)[0][int(tables[0, 0]), 1, 0, 4, 3] = q8.NAN
    q = rows((2, 4, dim), F16, 1)
    if operand == "q":
        q[0, 2:, 5] = float("inf")
    for part in (0, 32, pk.PARTITION_BALANCED):
        out = decode(q, kc, vc, tables, [n, n], 0.125, part)
        hit = out[0, 2:, 3:4] if operand == "v" else out[0, 2:]
        assert bool(hit.isnan().all()) and bool(torch.isfinite(out[0, :2]).all()) and bool(torch.isfinite(out[1]).all())
        if operand == "v":
            assert bool(torch.isfinite(out[0, 2:, 4:]).all()) and bool(torch.isfinite(out[0, 2:, :3]).all())


# ------------------------------------------------------------------ prefill
def prefill(q, kc, vc, tables, starts, lens, scale, out=None, most=None, **kw):
    out = torch.full_like(q, 5.0).cuda() if out is None else out
    pk.paged_attention_prefill_q8(q.cuda(), kc.cuda(), vc.cuda(), tables.cuda(), i32(starts), i32(lens), scale, out, most, **kw)
    return out


def check_prefill(dtype, cached, chunk, heads, group, dim, block, seed=0, extra=0, most=None, spread=1.0, scale=None, **kw):
    lens = [c + n for c, n in zip(cached, chunk)]
    kc, vc, tables = q8.filled(lens, heads, block, dim, dtype, seed + 20, spread, pad=seed % 2)
    starts = torch.tensor([0] + chunk).cumsum(0)
    total = int(starts[-1])
    q = rows((total + extra, heads * group, dim), dtype, seed + 3)
    scale = dim ** -0.5 if scale is None else scale
    out = prefill(q, kc, vc, tables, starts, lens, scale, None, most, **kw)
    assert pk.device_errors() == 0
    assert bool((out[total:] == 5).all())
    ref = q8.attention(q[:total], (kc, vc), tables, starts, lens, scale, dim)
    # the output and the probabilities (to fp16, the finer of the types)
    q8.assert_near(out[:total], ref, dtype, 2, f"{dtype} cached {cached} chunk {chunk}")


@pytest.mark.parametrize("parts", [1, 0, 2, 32])
@pytest.mark.parametrize("dtype,heads,group,dim,block", [
    (F16, 8, 4, 128, 16), (BF16, 2, 8, 128, 32), (F16, 1, 1, 64, 8), (BF16, 4, 3, 64, 16), (F16, 2, 6, 128, 8),
    (BF16, 1, 16, 64, 32), (F16, 1, 64, 128, 16), (BF16, 3, 7, 128, 16), (BF16, 2, 4, 128, 8), (F16, 2, 2, 64, 32)])
def test_prefill(dtype, heads, group, dim, block, parts):
    check_prefill(dtype, [0, 5, 300, 64, 0], [1, 40, 17, 0, 130], heads, group, dim, block, seed=heads, extra=3,
                  key_parts=parts)


@pytest.mark.parametrize("parts", [1, 0])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_prefill_long_context(dtype, parts):
    check_prefill(dtype, [5000, 0], [70, 600], 2, 4, 128, 16, seed=3, key_parts=parts)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_prefill_scales(dtype, scale):
    check_prefill(dtype, [50, 129], [33, 70], 2, 4, 64, 16, scale=scale)


@pytest.mark.parametrize("dtype,spread", [(F16, 1e-3), (F16, 300.0), (BF16, 1e-17), (BF16, 1e5), (BF16, 1e19)])
def test_prefill_small_and_large_values(dtype, spread):
    """V of any size (K's size goes into the scale)."""
    check_prefill(dtype, [40, 700], [20, 100], 4, 2, 128, 16, spread=spread, scale=128 ** -0.5 / spread, key_parts=0)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_prefill_values_that_grow_along_the_context(dtype):
    for up in (False, True):
        n, heads, dim, block = 600, 2, 128, 16
        tables, nb = q8.tables_for([n], block, 4)
        kc, vc = q8.new_pool(nb, heads, block, dim, 1), q8.new_pool(nb, heads, block, dim, 2)
        ramp = torch.logspace(-3, 3, n) if up else torch.logspace(3, -3, n)
        q8.fill(kc, tables[0], (rows((n, heads, dim), torch.float32, 5) * ramp.sqrt()[:, None, None] * 0.3).to(dtype))
        q8.fill(vc, tables[0], (rows((n, heads, dim), torch.float32, 6) * ramp[:, None, None]).to(dtype))
        q = rows((90, heads * 4, dim), dtype, 7)
        for parts in (1, 32):
            got = prefill(q, kc, vc, tables, [0, 90], [n], dim ** -0.5, key_parts=parts)
            ref = q8.attention(q, (kc, vc), tables, [0, 90], [n], dim ** -0.5, dim)
            # each row on its own: their outputs differ by orders of magnitude
            for r in range(0, 90, 7):
                q8.assert_near(got[r], ref[r], dtype, 2, f"up {up} parts {parts} row {r}")


def test_prefill_single_tokens_equal_decode():
    lens = [1, 50, 700]
    kc, vc, tables = q8.filled(lens, 4, 16, 128, BF16, 8)
    q = rows((3, 16, 128), BF16, 9)
    a = decode(q, kc, vc, tables, lens, 0.09, 0)
    b = prefill(q, kc, vc, tables, range(4), lens, 0.09)
    ref = q8.attention(q, (kc, vc), tables, range(4), lens, 0.09, 128)
    for got in (a, b):
        q8.assert_near(got, ref, BF16, 2)


def test_prefill_reports_bad_sequences_and_leaves_their_rows():
    lens = [40, 40, 40]
    kc, vc, tables = q8.filled(lens, 2, 16, 64, F16, 3)
    q = rows((30, 4, 64), F16, 1)

    def run(lens, most=10, tab=tables):
        return prefill(q, kc, vc, tab, [0, 10, 20, 30], lens, 0.1, None, most), pk.device_errors()

    out, err = run([40, 3, 40])                  # shorter than its chunk
    assert err == 4 and bool((out[10:20] == 5).all()) and not bool((out[:10] == 5).any())
    out, err = run([40, 40, 4000])               # past its table
    assert err == 4 and bool((out[20:] == 5).all())
    bad = tables.clone()
    bad[0, 0] = -7
    assert run(lens, tab=bad)[1] == 2            # BLOCK_ID


@pytest.mark.parametrize("dtype,dim,block", [(F16, 64, 16), (BF16, 128, 8)])
@pytest.mark.parametrize("operand", ["q", "k", "v"])
def test_prefill_nan_reaches_the_rows_that_attend_to_it(operand, dtype, dim, block):
    """A NaN at a chunk's token: rows before it, other heads and sequences stay finite."""
    n, chunk, heads, at = 83, 40, 2, 60
    tables, nb = q8.tables_for([n, n], block, 3)
    kc, vc = (torch.full((nb, heads, block, dim + q8.tail(block)), 0xFF, dtype=torch.uint8) for _ in range(2))
    for s in range(2):
        for pool in (kc, vc):
            q8.fill(pool, tables[s], rows((n, heads, dim), dtype, 5 + s))
    q = rows((2 * chunk, 4, dim), dtype, 1)
    first = at - (n - chunk)                     # the chunk's row at that token
    if operand == "q":
        q[first, 2:, 5] = float("inf")
    else:
        pool = kc if operand == "k" else vc
        codes, _, mark = q8.views(pool, dim)
        codes[int(tables[0, at // block]), 1, 1, at % block, 3] = q8.NAN
        mark[int(tables[0, at // block]), 1] = 1 << at % block
    for parts in (1, 32):
        out = prefill(q, kc, vc, tables, [0, chunk, 2 * chunk], [n, n], 0.125, key_parts=parts).cpu()
        assert bool(torch.isfinite(out[:, :2]).all()) and bool(torch.isfinite(out[chunk:]).all())
        assert bool(torch.isfinite(out[:first]).all())
        assert bool(out[first, 2:].isnan().all())
        after = out[first + 1:chunk, 2:]
        assert bool(torch.isfinite(after).all()) if operand == "q" else bool(after.isnan().all())


# ---------------------------------------------------- blocks, streams, graphs
@pytest.mark.parametrize("dtype,block", [(F16, 8), (BF16, 16), (F16, 32)])
def test_blocks_copy_and_swap(dtype, block):
    kc, vc, _ = q8.filled([10 * block], 3, block, 64, dtype, 1)
    a, b = kc.cuda(), vc.cuda()
    pk.paged_kv_copy_blocks(a, b, i32([[0, 9], [3, 8]]))
    kc[9], vc[9], kc[8], vc[8] = kc[0], vc[0], kc[3], vc[3]
    assert torch.equal(a.cpu(), kc) and torch.equal(b.cpu(), vc)
    hk, hv = torch.zeros_like(kc[:2]).pin_memory(), torch.zeros_like(vc[:2]).pin_memory()
    pk.paged_kv_swap_blocks(a, b, hk, hv, i32([[5, 1]]))
    torch.cuda.synchronize()
    assert torch.equal(hk[1], kc[5]) and torch.equal(hv[1], vc[5])
    pk.paged_kv_swap_blocks(hk, hv, a, b, i32([[1, 2]]))
    assert torch.equal(a[2].cpu(), kc[5])
    assert pk.device_errors() == 0
