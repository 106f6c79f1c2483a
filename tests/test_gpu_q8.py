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


@pytest.mark.parametrize("far", [0, 4, 20])
@pytest.mark.parametrize("dtype,dim,block", [(F16, 64, 8), (BF16, 128, 16), (BF16, 64, 32), (BF16, 128, 8)])
def test_every_code(dtype, dim, block, far):
    """Codes drawn from all that are numbers, those below 2^-6 among them, and K's scales
    up to 2^far apart within 64 tokens."""
    heads, lens, chunk = 2, [230, 64, 77], [70, 64, 1]
    kc, vc, tables = q8.filled(lens, heads, block, dim, dtype, 8)
    g = torch.Generator().manual_seed(9)
    for pool, most in ((kc, far), (vc, 3)):
        codes, scale, mark = q8.views(pool, dim)
        codes[:] = torch.randint(0, 256, codes.shape, generator=g, dtype=torch.int32).to(torch.uint8)
        codes[(codes & 0x7f) == 0x7f] = 3
        scale[:] = torch.exp2(-torch.randint(0, most + 1, scale.shape, generator=g).float())
        mark[:] = 0
    starts = torch.tensor([0] + chunk).cumsum(0)
    q = (torch.randn(int(starts[-1]), 2 * heads, dim, generator=g) * 0.1).to(dtype)
    out = prefill(q, kc, vc, tables, starts, lens, 0.125)
    q8.assert_near(out, q8.attention(q, (kc, vc), tables, starts, lens, 0.125, dim), dtype, 2, "prefill")
    one = torch.arange(4)
    out = decode(q[:3], kc, vc, tables, lens, 0.125, 0)
    q8.assert_near(out, q8.attention(q[:3], (kc, vc), tables, one, lens, 0.125, dim), dtype, 2, "decode")
    assert pk.device_errors() == 0


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


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("dtype,dim,block", [(F16, 128, 16), (BF16, 64, 8)])
def test_serving_loop(dtype, dim, block, graph):
    """Forks with their blocks' copies, tables, append, prefill, decode and release
    together, step after step, on a side stream and captured: each step's attention is
    that of caches kept by the definition, and no block is lost or held twice."""
    from test_gpu_pages import ALL, Cache
    heads, group, steps, most = 2, 3, 6, 5
    start = [0, block - 1, 2 * block, 100, 3, 0, 0, 0]
    c = Cache(start, block, 20, 60, 7)
    S, nb = len(start), c.blocks
    T = S * most
    kc, vc = q8.new_pool(nb, heads, block, dim, 1), q8.new_pool(nb, heads, block, dim, 2)
    for s, n in enumerate(start):
        for i, pool in enumerate((kc, vc)):
            q8.fill(pool, c.tables[s], rows((n, heads, dim), dtype, 10 * s + i))
    d = c.device()
    gk, gv, lens, count = kc.cuda(), vc.cuda(), d["lens"], d["count"]
    dev = dict(device="cuda", dtype=torch.int32)
    parents, keep, new = torch.full((S,), -1, **dev), torch.full((S,), ALL, **dev), torch.zeros(S, **dev)
    pairs, starts = torch.zeros(S, 2, **dev), torch.zeros(S + 1, **dev)
    seq, pos = torch.zeros(T, **dev), torch.zeros(T, **dev)
    k, v = (torch.zeros(T, heads, dim, dtype=dtype, device="cuda") for _ in range(2))
    q, qd = (torch.zeros(n, heads * group, dim, dtype=dtype, device="cuda") for n in (T, S))
    out, outd = torch.zeros_like(q), torch.zeros_like(qd)
    ws, wp = pk.new_workspace(qd, d["tables"], block, pk.PARTITION_BALANCED), pk.prefill_workspace(q)

    def step():
        pk.paged_kv_fork(parents, lens, d["tables"], d["shared"], d["free"], count, pairs, block)
        pk.paged_kv_copy_blocks(gk, gv, pairs)
        pk.paged_kv_build_tables(new, lens, d["tables"], d["free"], count, block, nb, starts, seq, pos)
        pk.paged_kv_append_q8(k, v, d["tables"], starts, lens, gk, gv)
        pk.paged_attention_prefill_q8(q, gk, gv, d["tables"], starts, lens, dim ** -0.5, out, most, workspace=wp, key_parts=0)
        pk.paged_attention_decode_q8(qd, gk, gv, d["tables"], lens, dim ** -0.5, outd, pk.PARTITION_BALANCED, ws)
        pk.paged_kv_release(keep, lens, d["tables"], d["shared"], d["free"], count, block)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    if graph:
        with torch.cuda.stream(side):
            step()                      # with nothing to do: it leaves the state as it is
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
    for i in range(steps):
        fork_of = [-1] * S
        if i % 2 == 0:
            empty, full = ([s for s in range(S) if (c.lens[s] == 0) == e and s > 0] for e in (True, False))
            for e, s in zip(empty[:2], full):
                fork_of[e] = s
        want_pairs = c.fork(fork_of)
        for a, b in want_pairs:
            for pool in (kc, vc):
                pool[b] = pool[a].clone()
        add = [(s + i) % (most + 1) if c.lens[s] else 0 for s in range(S)]
        x, y, z = [rows(k.shape, dtype, 100 + 3 * i + j) for j in range(2)], rows(q.shape, dtype, 300 + i), rows(qd.shape, dtype, 400 + i)
        before = list(c.lens)
        st = [0]
        for s in range(S):
            for j in range(-(-before[s] // block), -(-(before[s] + add[s]) // block)):
                c.tables[s, j] = c.stack.pop()
            c.lens[s] += add[s]
            st.append(st[-1] + add[s])
        now = list(c.lens)
        drop = [0 if (s + i) % 5 == 4 else max(0, now[s] - 2) if (s + i) % 4 == 1 and now[s] - 2 >= before[s] else ALL
                for s in range(S)]
        torch.cuda.synchronize()
        for t, value in ((parents, fork_of), (new, add), (keep, drop)):
            t.copy_(torch.tensor(value, dtype=torch.int32))
        k.copy_(x[0]), v.copy_(x[1]), q.copy_(y), qd.copy_(z)
        torch.cuda.synchronize()
        if graph:
            g.replay()
        else:
            with torch.cuda.stream(side):
                step()
        torch.cuda.synchronize()
        assert pk.device_errors() == 0
        assert pairs.tolist() == want_pairs and starts.tolist() == st
        t = torch.from_numpy(c.tables)
        for pool, r in ((kc, x[0]), (vc, x[1])):
            q8.append(pool, r, t, st, now)
        ref = q8.attention(y[:st[-1]], (kc, vc), t, st, now, dim ** -0.5, dim)
        q8.assert_near(out[:st[-1]], ref, dtype, 2, f"prefill step {i}")
        ref = q8.attention(z, (kc, vc), t, range(S + 1), now, dim ** -0.5, dim)
        q8.assert_near(outd, ref, dtype, 2, f"decode step {i}")
        c.release(drop)
        c.check(d, lens, count)


def test_calls_repeat_bit_for_bit():
    lens, heads, dim, block = [3000, 17, 1, 640], 4, 128, 16
    kc, vc, tables = q8.filled(lens, heads, block, dim, BF16, 4)
    q, qp = rows((4, heads * 4, dim), BF16, 5), rows((80, heads * 4, dim), BF16, 6)
    first = [decode(q, kc, vc, tables, lens, 0.09, part) for part in (0, 256, pk.PARTITION_BALANCED)]
    chunk = [0, 60, 70, 71, 80]
    first += [prefill(qp, kc, vc, tables, chunk, lens, 0.09, key_parts=parts) for parts in (1, 0, 32)]
    for _ in range(10):
        again = [decode(q, kc, vc, tables, lens, 0.09, part) for part in (0, 256, pk.PARTITION_BALANCED)]
        again += [prefill(qp, kc, vc, tables, chunk, lens, 0.09, key_parts=parts) for parts in (1, 0, 32)]
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    assert pk.device_errors() == 0


def test_prefill_many_items_per_block():
    """More items than SMs, of one to many key tiles, whole and split: the rings and
    their phases run on across items."""
    lens = [(1, 40, 64, 65, 300, 900)[(5 * i + i // 6) % 6] for i in range(90)]
    chunk = [min(n, (1, 7, 40, 130)[i % 4]) for i, n in enumerate(lens)]
    for dtype, dim, block in ((BF16, 128, 8), (F16, 64, 16)):
        kc, vc, tables = q8.filled(lens, 4, block, dim, dtype, 4)
        starts = torch.tensor([0] + chunk).cumsum(0)
        q = rows((int(starts[-1]), 8, dim), dtype, 6)
        ref = q8.attention(q, (kc, vc), tables, starts, lens, dim ** -0.5, dim)
        for parts in (1, 32):
            out = prefill(q, kc, vc, tables, starts, lens, dim ** -0.5, key_parts=parts)
            q8.assert_near(out, ref, dtype, 2, f"parts {parts}")
    assert pk.device_errors() == 0


@pytest.mark.parametrize("seqs", [7, 256, 257, 300])
def test_prefill_of_many_sequences_some_without_rows(seqs):
    """Up to 256 sequences are taken longest first, more in their own order; those
    without rows in this call come between the others."""
    lens = [(0, 33, 90, 16, 200)[(3 * i + i // 7) % 5] for i in range(seqs)]
    chunk = [min(n, (0, 9, 70, 0, 1)[i % 5]) for i, n in enumerate(lens)]
    kc, vc, tables = q8.filled(lens, 2, 16, 64, F16, 11)
    starts = torch.tensor([0] + chunk).cumsum(0)
    q = rows((int(starts[-1]) + 2, 6, 64), F16, 12)
    ref = q8.attention(q[:-2], (kc, vc), tables, starts, lens, 0.125, 64)
    for parts in (1, 2, 0):
        out = prefill(q, kc, vc, tables, starts, lens, 0.125, most=max(chunk), key_parts=parts)
        assert bool((out[-2:] == 5).all())
        q8.assert_near(out[:-2], ref, F16, 2, f"parts {parts}")
    assert pk.device_errors() == 0


def test_two_graphs_take_turns_with_one_workspace():
    """Two captured steps share their workspaces; each replay gives what the eager call did."""
    steps = []
    for i, (lens, chunk) in enumerate((([700, 40, 64], [20, 1, 9]), ([25, 900, 33], [5, 20, 5]))):
        kc, vc, tables = q8.filled(lens, 4, 16, 128, BF16, 13 + i)
        tables = torch.cat([tables, torch.full((3, 60 - tables.shape[1]), -1, dtype=torch.int32)], 1)
        one, many = rows((3, 16, 128), BF16, 14 + i), rows((30, 16, 128), BF16, 15 + i)
        steps.append([t.cuda() for t in (one, many, kc, vc, tables)] + [i32([0] + torch.tensor(chunk).cumsum(0).tolist()), i32(lens)])
    ws = pk.new_workspace(steps[0][0], steps[0][4], 16, pk.PARTITION_BALANCED)
    split = pk.prefill_workspace(steps[0][1])

    def step(x, out):
        one, many, kc, vc, tables, starts, lens = x
        pk.paged_attention_decode_q8(one, kc, vc, tables, lens, 0.1, out[0], pk.PARTITION_BALANCED, ws)
        pk.paged_attention_prefill_q8(many, kc, vc, tables, starts, lens, 0.1, out[1], 20, workspace=split, key_parts=32)

    outs = [[torch.zeros_like(t) for t in x[:2]] for x in steps]
    want, graphs = [], []
    for x, out in zip(steps, outs):
        step(x, out)
        want.append([t.clone() for t in out])
    torch.cuda.synchronize()
    for x, out in zip(steps, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step(x, out)
    for i in (0, 1, 1, 0, 1):
        for t in outs[i]:
            t.zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))
    assert pk.device_errors() == 0


def test_pools_past_4_gib():
    """Blocks whose bytes lie past 2^32 in their pool."""
    heads, dim, block, dtype = 8, 128, 32, BF16
    nb = (1 << 32) // (heads * block * (dim + 1)) + 40
    pools = [pk.new_q8_pool(nb, heads, block, dim) for _ in range(2)]
    lens = [300, 70]
    tables = torch.tensor([[nb - 1 - 2 * j for j in range(10)], [nb - 2 - 2 * j if j < 3 else -1 for j in range(10)]],
                          dtype=torch.int32)
    small = [q8.new_pool(40, heads, block, dim, i) for i in range(2)]      # the pools' last 40 blocks
    near = torch.where(tables >= 0, tables - (nb - 40), tables)
    slots = torch.cat([q8.sequence_slots(tables, s, n, block) for s, n in enumerate(lens)])
    near_slots = torch.cat([q8.sequence_slots(near, s, n, block) for s, n in enumerate(lens)])
    k, v = rows((370, heads, dim), dtype, 1), rows((370, heads, dim), dtype, 2)
    starts = [0, 300, 370]
    for pool, x in zip(small, (k, v)):
        q8.append(pool, x, near, starts, lens)
    for pool in pools:
        pool[nb - 40:] = 255
    pk.paged_kv_append_q8(k.cuda(), v.cuda(), tables.cuda(), i32(starts), i32(lens), *pools)
    back = [torch.zeros(370, heads, dim, dtype=dtype, device="cuda") for _ in range(2)]
    pk.paged_kv_gather_q8(*pools, slots.cuda(), *back)
    for got, pool in zip(back, small):
        assert torch.equal(got.cpu().double(), q8.read(pool, near_slots, dim))
    q = rows((2, heads * 4, dim), dtype, 3)
    ref = q8.attention(q, small, near, range(3), lens, 0.09, dim)
    for part in (0, pk.PARTITION_BALANCED):
        q8.assert_near(decode(q, pools[0], pools[1], tables, lens, 0.09, part), ref, dtype, 2)
    qp = rows((370, heads * 4, dim), dtype, 4)
    out = prefill(qp, *pools, tables, starts, lens, 0.09, torch.zeros_like(qp).cuda(), 300)
    q8.assert_near(out, q8.attention(qp, small, near, starts, lens, 0.09, dim), dtype, 2)
    assert pk.device_errors() == 0


def test_decode_4096_sequences():
    rng = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 40, (4096,), generator=rng).tolist()
    for heads, group, dim in ((4, 2, 128), (1, 1, 64)):
        kc, vc, tables = q8.filled(lens, heads, 8, dim, BF16, 6)
        q = rows((4096, heads * group, dim), BF16, 7)
        ref = q8.attention(q, (kc, vc), tables, range(4097), lens, dim ** -0.5, dim)
        for part in (0, 32, pk.PARTITION_BALANCED):
            q8.assert_near(decode(q, kc, vc, tables, lens, dim ** -0.5, part), ref, BF16, 2)
        assert pk.device_errors() == 0


@pytest.mark.parametrize("heads, dim, block", [(32, 64, 8), (2, 128, 32), (3, 64, 16)])
def test_decode_short_sequences_beside_long_ones(heads, dim, block):
    """A balanced split over sequences of one or two tiles, empty ones and a few long
    ones, in an order that ends shares inside, before and behind each of them."""
    lens = [(5000, 0, 1, 32, 33, 64, 700, 31)[(3 * i + i // 8) % 8] for i in range(150)]
    kc, vc, tables = q8.filled(lens, heads, block, dim, F16, 4)
    q = rows((len(lens), heads, dim), F16, 6)
    ref = q8.attention(q, (kc, vc), tables, range(len(lens) + 1), lens, dim ** -0.5, dim)
    q8.assert_near(decode(q, kc, vc, tables, lens, dim ** -0.5, pk.PARTITION_BALANCED), ref, F16, 2, "short and long")
    assert pk.device_errors() == 0


def test_two_streams_with_a_workspace_each():
    lens, heads, dim, block = [2000, 700, 31], 4, 128, 16
    kc, vc, tables = q8.filled(lens, heads, block, dim, BF16, 4)
    gk, gv, gt, L = kc.cuda(), vc.cuda(), tables.cuda(), i32(lens)
    qs = [rows((3, heads * 2, dim), BF16, 20 + i).cuda() for i in range(2)]
    outs = [torch.zeros_like(q) for q in qs]
    ws = [pk.new_workspace(q, gt, block, pk.PARTITION_BALANCED) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(40):
        s = i % 2
        pk.paged_attention_decode_q8(qs[s], gk, gv, gt, L, 0.09, outs[s], pk.PARTITION_BALANCED, ws[s], stream=streams[s])
    torch.cuda.synchronize()
    for q, out in zip(qs, outs):
        q8.assert_near(out, q8.attention(q.cpu(), (kc, vc), tables, range(4), lens, 0.09, dim), BF16, 2)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gather_into_a_16_bit_pool(dtype):
    """An 8-bit sequence moved into 16-bit pools: paged_kv_append_tokens right behind
    the gather that makes its rows, many times over."""
    n, heads, dim, block = 3000, 8, 128, 16
    kc, vc, tables = q8.filled([n], heads, block, dim, dtype, 5)
    slots = q8.sequence_slots(tables, 0, n, block).cuda()
    gk, gv, gt = kc.cuda(), vc.cuda(), tables.cuda()
    seq, pos = torch.zeros(n, dtype=torch.int32).cuda(), torch.arange(n, dtype=torch.int32).cuda()
    want = [q8.read(p, slots.cpu(), dim) for p in (kc, vc)]
    for i in range(5):
        k, v = (torch.full((n, heads, dim), float(i), dtype=dtype, device="cuda") for _ in range(2))
        k16, v16 = (torch.zeros(kc.shape[0], block, heads, dim, dtype=dtype, device="cuda") for _ in range(2))
        torch.cuda.synchronize()
        pk.paged_kv_gather_q8(gk, gv, slots, k, v)
        pk.paged_kv_append_tokens(k, v, gt, seq, pos, k16, v16)
        torch.cuda.synchronize()
        for pool, ref in ((k16, want[0]), (v16, want[1])):
            assert torch.equal(pool.flatten(0, 1)[slots].cpu().double(), ref)


def test_refusals_on_the_gpu():
    kc, vc, tables = (t.cuda() for t in q8.filled([20], 2, 16, 64, F16, 1))
    q, L, out = torch.zeros(1, 4, 64, dtype=F16, device="cuda"), i32([20]), torch.zeros(1, 4, 64, dtype=F16, device="cuda")
    with pytest.raises(pk.PagedKVError, match="contiguous"):
        pk.paged_attention_decode_q8(q.transpose(1, 2).contiguous().transpose(1, 2), kc, vc, tables, L, 0.1, out)
    with pytest.raises(pk.PagedKVError, match="out must be"):
        pk.paged_attention_decode_q8(q, kc, vc, tables, L, 0.1, out.bfloat16())
    with pytest.raises(pk.PagedKVError, match="current device"):
        pk.paged_attention_decode_q8(q, kc, vc, tables.cpu(), L, 0.1, out)
    with pytest.raises(pk.PagedKVError, match="unsupported"):
        pk.paged_attention_decode_q8(q.float(), kc, vc, tables, L, 0.1, out.float())
    with pytest.raises(pk.PagedKVError, match="8-bit pools"):
        pk.paged_attention_decode_q8(q, *(pk.new_q4_pool(4, 2, 16, 64) for _ in range(2)), tables, L, 0.1, out)
    with pytest.raises(pk.PagedKVError, match="4-bit pools"):
        pk.paged_attention_decode_q4(q, kc, vc, tables, L, 0.1, out)
    with pytest.raises(pk.PagedKVError, match="workspace"):
        pk.paged_attention_decode_q8(q, kc, vc, tables, L, 0.1, out, 32)
    with pytest.raises(pk.PagedKVError, match="workspace"):
        pk.paged_attention_prefill_q8(q, kc, vc, tables, i32([0, 1]), L, 0.1, out, 1,
                                      workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"), key_parts=4)
    k = torch.zeros(3, 2, 64, dtype=F16, device="cuda")
    with pytest.raises(pk.PagedKVError, match="kv heads"):
        pk.paged_kv_append_q8(k[:, :1].contiguous(), k[:, :1].contiguous(), tables, i32([0, 3]), L, kc, vc)
    with pytest.raises(pk.PagedKVError, match="query_start must"):
        pk.paged_kv_append_q8(k, k, tables, i32([0, 3, 3]), L, kc, vc)
    with pytest.raises(pk.PagedKVError, match="v must be"):
        pk.paged_kv_append_q8(k, k.bfloat16(), tables, i32([0, 3]), L, kc, vc)
    pk.paged_attention_decode_q8(q[:0], kc, vc, tables[:0], L[:0], 0.1, out[:0])
    pk.paged_kv_append_q8(k[:0], k[:0], tables, i32([0, 0]), L, kc, vc)
    assert pk.device_errors() == 0
