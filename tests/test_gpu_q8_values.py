"""Attention over the 8-bit cache at the ends of its types: infinite queries, scales far
apart, values at the documented limits. Against the definition in 64 bits."""
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


def decode(q, kc, vc, tables, lens, scale, part):
    q, tables = q.cuda(), tables.cuda()
    out, ws = torch.full_like(q, 5.0), pk.new_workspace(q, tables, kc.shape[2], part)
    pk.paged_attention_decode_q8(q, kc.cuda(), vc.cuda(), tables, i32(lens), scale, out, part, ws)
    return out


def prefill(q, kc, vc, tables, starts, lens, scale, **kw):
    out = torch.full_like(q, 5.0).cuda()
    pk.paged_attention_prefill_q8(q.cuda(), kc.cuda(), vc.cuda(), tables.cuda(), i32(starts), i32(lens), scale, out, **kw)
    return out


def pools(k, v, block):
    """Pools whose one sequence holds the rows k, v [n][Hkv][D], and its table."""
    tables, nb = q8.tables_for([len(k)], block, 4)
    kc, vc = (q8.new_pool(nb, k.shape[1], block, k.shape[2], i) for i in (1, 2))
    q8.fill(kc, tables[0], k)
    q8.fill(vc, tables[0], v)
    return kc, vc, tables


# ---------------------------------------------------------- infinite queries
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("n,chunk", [(1, 1), (70, 70), (900, 40), (6000, 33)])
@pytest.mark.parametrize("dtype,dim,block", [(F16, 64, 16), (F16, 128, 8), (BF16, 64, 32), (BF16, 128, 16)])
def test_an_infinite_query_is_nan(dtype, dim, block, n, chunk, sign):
    """Every key has the same sign in the channel where a query is infinite, so that all
    of its scores are +inf, or all of them -inf: no softmax, whole or split over the keys."""
    heads, group = 2, 2
    k, v = rows((n, heads, dim), dtype, 1), rows((n, heads, dim), dtype, 2)
    k[..., 5] = (1 + k[..., 5].abs()).to(dtype)
    kc, vc, tables = pools(k, v, block)
    q = rows((chunk, heads * group, dim), dtype, 3)
    bad = torch.zeros(chunk, heads * group, dtype=torch.bool)
    bad[::3, 1] = bad[0, 2] = bad[-1, 3] = True
    q[bad, 5] = sign * math.inf
    ref = q8.attention(q, (kc, vc), tables, [0, chunk], [n], 0.125, dim)
    assert bool(ref[bad].isnan().all()) and bool(torch.isfinite(ref[~bad]).all())
    for parts in (1, 8, 32):
        out = prefill(q, kc, vc, tables, [0, chunk], [n], 0.125, key_parts=parts).cpu()
        assert bool(out[bad].isnan().all()), f"parts {parts}"
        q8.assert_near(out[~bad], ref[~bad], dtype, 2, f"parts {parts}")
    one = q8.attention(q[-1:], (kc, vc), tables, [0, 1], [n], 0.125, dim)
    for part in (0, 64, pk.PARTITION_BALANCED):
        out = decode(q[-1:], kc, vc, tables, [n], 0.125, part).cpu()
        assert bool(out[bad[-1:]].isnan().all()), f"part {part}"
        q8.assert_near(out[~bad[-1:]], one[~bad[-1:]], dtype, 2, f"part {part}")
    assert pk.device_errors() == 0


# --------------------------------------------------- scales far apart in a key tile
def spread_pool(n, heads, dim, block, tables, nb, far, seed, least):
    """A pool of random codes whose blocks' scales are 2^least and 2^(least - far) in turn."""
    pool = q8.new_pool(nb, heads, block, dim, seed)
    codes, scale, mark = q8.views(pool, dim)
    g = torch.Generator().manual_seed(seed)
    codes[:] = torch.randint(0, 256, codes.shape, generator=g, dtype=torch.int32).to(torch.uint8)
    codes[(codes & 0x7f) == 0x7f] = 3
    scale[:], mark[:] = 2.0 ** least, 0
    scale[tables[0, 1::2].long()] = 2.0 ** (least - far)
    return pool


def as_staged(x, block, least, far):
    """Rows [n][Hkv][D] of such a pool as a prefill documents them: multiples of 2^-30 of the
    largest scale of 64 neighbouring tokens, those of scales more than 2^30 below it zeros."""
    small = (torch.arange(len(x)) // block % 2 == 1)[:, None, None]
    step = 2.0 ** (least - 30)
    return torch.where(small, torch.round(x / step) * step if far <= 30 else torch.zeros_like(x), x)


def softmax_rows(q, k, v, scale):
    """fp64 causal attention of the chunk q [r][Hq][D] at the end of k, v [n][Hkv][D]."""
    r, n, heads = len(q), len(k), k.shape[1]
    z = torch.einsum("rhgd,khd->rhgk", q.double().unflatten(1, (heads, -1)), k.double()) * scale
    seen = torch.arange(n)[None] <= torch.arange(n - r, n)[:, None]
    w = torch.softmax(z.masked_fill(~seen[:, None, None], -math.inf), -1)
    return torch.einsum("rhgk,khd->rhgd", w, v.double()).flatten(1, 2)


@pytest.mark.parametrize("far", [20, 25, 30, 31, 40, 60])
@pytest.mark.parametrize("dtype,dim,block", [(F16, 64, 8), (F16, 128, 32), (BF16, 128, 16), (BF16, 64, 8)])
def test_scales_of_v_far_apart(dtype, dim, block, far):
    """Rows that attend to the blocks of small values all but alone, and rows that attend to
    all of them; each row on its own, since their outputs differ by orders of magnitude."""
    n, chunk, heads, group = 150, 60, 2, 2
    tables, nb = q8.tables_for([n], block, 4)
    kc, vc = q8.new_pool(nb, heads, block, dim, 1), spread_pool(n, heads, dim, block, tables, nb, far, 2, 6)
    k = rows((n, heads, dim), dtype, 3)
    k[..., 0] = (torch.arange(n) // block % 2)[:, None].to(dtype)          # 1 in the blocks of small values
    q8.fill(kc, tables[0], k)
    q = rows((chunk, heads * group, dim), dtype, 5)
    q[..., 0] = 0
    q[::2, :, 0] = 2000.0
    slots = q8.sequence_slots(tables, 0, n, block)
    kx, vx = q8.read(kc, slots, dim), q8.read(vc, slots, dim)
    ref = softmax_rows(q, kx, as_staged(vx, block, 6, far), dim ** -0.5)
    for parts in (1, 32):
        out = prefill(q, kc, vc, tables, [0, chunk], [n], dim ** -0.5, key_parts=parts)
        for r in range(chunk):
            q8.assert_near(out[r], ref[r], dtype, 2, f"parts {parts} row {r}")
    assert pk.device_errors() == 0


@pytest.mark.parametrize("far", [20, 25, 31, 40, 60])
@pytest.mark.parametrize("dtype,dim,block", [(F16, 64, 8), (F16, 128, 32), (BF16, 128, 16), (BF16, 64, 8)])
def test_scales_of_k_far_apart(dtype, dim, block, far):
    """Keys of small blocks count as documented in fp16, and as they are in bf16."""
    n, chunk, heads, group, least = 150, 60, 2, 2, 7
    tables, nb = q8.tables_for([n], block, 4)
    kc, vc = spread_pool(n, heads, dim, block, tables, nb, far, 2, least), q8.new_pool(nb, heads, block, dim, 1)
    codes = q8.views(kc, dim)[0]
    codes[tables[0, ::2].long(), :, 0, :, 8:] = 0         # the large blocks' keys: channels 0 to 7 alone
    codes[tables[0, ::2].long(), :, 1:] = 0
    q8.fill(vc, tables[0], rows((n, heads, dim), dtype, 3))
    # queries that see the small keys alone, as large as a type of 16 bits lets them be
    size = min(2.0 ** (far - least - 4), 2.0 ** 14) if dtype == F16 else 2.0 ** (far - least - 4)
    q = (rows((chunk, heads * group, dim), torch.float32, 5) * size / 4).to(dtype)
    q[..., :8] = 0
    slots = q8.sequence_slots(tables, 0, n, block)
    kx, vx = q8.read(kc, slots, dim), q8.read(vc, slots, dim)
    ref = softmax_rows(q, as_staged(kx, block, least, far) if dtype == F16 else kx, vx, dim ** -0.5)
    for parts in (1, 32):
        out = prefill(q, kc, vc, tables, [0, chunk], [n], dim ** -0.5, key_parts=parts)
        q8.assert_near(out, ref, dtype, 2, f"parts {parts}")
    assert pk.device_errors() == 0


# ------------------------------------------------------- the ends of bf16's range
@pytest.mark.parametrize("size", [2.0 ** 90, 2.0 ** 108, 2.0 ** 113, 2.0 ** 118, 2.0 ** 124])
@pytest.mark.parametrize("dim,block", [(64, 16), (128, 8)])
def test_large_queries(dim, block, size):
    """Queries of any size, and a scale that brings their scores back to ordinary ones."""
    n, heads, group = 300, 2, 4
    k, v = rows((n, heads, dim), BF16, 1, 2.0 ** -10), rows((n, heads, dim), BF16, 2)
    kc, vc, tables = pools(k, v, block)
    q = (rows((70, heads * group, dim), torch.float32, 3) * size).to(BF16)
    scale = dim ** -0.5 * 2.0 ** 10 / size
    ref = q8.attention(q, (kc, vc), tables, [0, 70], [n], scale, dim)
    for parts in (1, 32):
        q8.assert_near(prefill(q, kc, vc, tables, [0, 70], [n], scale, key_parts=parts), ref, BF16, 2, f"parts {parts}")
    for part in (0, 64, pk.PARTITION_BALANCED):
        q8.assert_near(decode(q[-1:], kc, vc, tables, [n], scale, part), ref[-1:], BF16, 2, f"part {part}")
    assert pk.device_errors() == 0


@pytest.mark.parametrize("size", [2.0 ** 45, 2.0 ** 111])
@pytest.mark.parametrize("dim,block", [(64, 16), (128, 8)])
def test_large_keys(dim, block, size):
    """Keys of any size, small ones beside them."""
    n, heads, group = 300, 2, 4
    k, v = rows((n, heads, dim), torch.float32, 1), rows((n, heads, dim), BF16, 2)
    k[:200] *= size
    kc, vc, tables = pools(k.to(BF16), v, block)
    q = (rows((70, heads * group, dim), torch.float32, 3) / size).to(BF16)
    scale = dim ** -0.5
    ref = q8.attention(q, (kc, vc), tables, [0, 70], [n], scale, dim)
    for parts in (1, 32):
        q8.assert_near(prefill(q, kc, vc, tables, [0, 70], [n], scale, key_parts=parts), ref, BF16, 2, f"parts {parts}")
    for part in (0, 64, pk.PARTITION_BALANCED):
        q8.assert_near(decode(q[-1:], kc, vc, tables, [n], scale, part), ref[-1:], BF16, 2, f"part {part}")


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("dtype,log2_size", [(F16, 14), (BF16, 14), (BF16, 40)])
def test_blocks_of_zeros_beside_the_largest_values(dtype, log2_size, first):
    """Tokens whose values are zeros keep their part of the softmax's sum, although their
    scale is the least there is: 4000 of them at 2^-8 of the others' weight each."""
    heads, group, dim, block, few = 2, 2, 64, 16, 64
    n = 4000 + few
    large = torch.zeros(n, dtype=torch.bool)
    large[:few if first else n] = True
    if not first:
        large[:n - few] = False
    k, v = torch.zeros(n, heads, dim), rows((n, heads, dim), torch.float32, 2, 0.25).clamp(-1, 1) * 2.0 ** log2_size
    k[large, :, 0] = 8 * math.log(2.0)
    v[~large] = 0
    kc, vc, tables = pools(k.to(dtype), v.to(dtype), block)
    q = torch.zeros(few // 2, heads * group, dim, dtype=dtype)
    q[..., 0] = 1
    ref = q8.attention(q, (kc, vc), tables, [0, len(q)], [n], 1.0, dim)
    for parts in (1, 32):
        out = prefill(q, kc, vc, tables, [0, len(q)], [n], 1.0, key_parts=parts)
        q8.assert_near(out, ref, dtype, 2, f"parts {parts}")
    for part in (0, 256, pk.PARTITION_BALANCED):
        out = decode(q[-1:], kc, vc, tables, [n], 1.0, part)
        q8.assert_near(out, ref[-1:], dtype, 2, f"part {part}")
    assert pk.device_errors() == 0


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -126])
@pytest.mark.parametrize("dim,block", [(64, 16), (128, 8)])
def test_a_scale_of_none_with_large_queries(dim, block, scale):
    """Every token the same weight."""
    n, heads, group = 300, 2, 4
    kc, vc, tables = pools(rows((n, heads, dim), BF16, 1, 2.0 ** -30), rows((n, heads, dim), BF16, 2), block)
    q = (rows((70, heads * group, dim), torch.float32, 3) * 2.0 ** 124).to(BF16)
    ref = q8.attention(q, (kc, vc), tables, [0, 70], [n], scale, dim)
    for parts in (1, 32):
        q8.assert_near(prefill(q, kc, vc, tables, [0, 70], [n], scale, key_parts=parts), ref, BF16, 2, f"parts {parts}")
    for part in (0, 64, pk.PARTITION_BALANCED):
        q8.assert_near(decode(q[-1:], kc, vc, tables, [n], scale, part), ref[-1:], BF16, 2, f"part {part}")


# ------------------------------------------------- tables wider than the contexts
@pytest.mark.parametrize("wider", [4, 32])
@pytest.mark.parametrize("cached,chunk", [([6001], [33]), ([900, 0, 40, 500], [64] * 4), ([100] * 20, [64] * 20), ([8192], [600])])
@pytest.mark.parametrize("dtype,dim", [(BF16, 128), (F16, 64)])
def test_a_split_chosen_by_the_tables_width(dtype, dim, cached, chunk, wider):
    """key_parts 0 goes by a width that says little about the contexts: the results are the
    same, whole or split."""
    heads, group, block = 8, 4, 16
    lens = [c + n for c, n in zip(cached, chunk)]
    kc, vc, tables = q8.filled(lens, heads, block, dim, dtype, 5)
    wide = torch.full((len(lens), wider * tables.shape[1]), -1, dtype=torch.int32)
    wide[:, :tables.shape[1]] = tables
    starts = torch.tensor([0] + chunk).cumsum(0)
    q = rows((int(starts[-1]), heads * group, dim), dtype, 6)
    ref = q8.attention(q, (kc, vc), tables, starts, lens, dim ** -0.5, dim)
    for t in (tables, wide):
        out = prefill(q, kc, vc, t, starts, lens, dim ** -0.5, key_parts=0)
        q8.assert_near(out, ref, dtype, 2, f"width {t.shape[1]}")
    assert pk.device_errors() == 0


@pytest.mark.parametrize("parts", [1, 0, 32])
@pytest.mark.parametrize("cached,chunk", [([6001], [33]), ([40, 0, 500], [1, 300, 64])])
def test_any_bound_of_the_chunks_will_do(cached, chunk, parts):
    """max_query_len far above every chunk, up to the largest int: the same as the exact one."""
    heads, group, dim, block = 4, 4, 128, 16
    lens = [c + n for c, n in zip(cached, chunk)]
    kc, vc, tables = q8.filled(lens, heads, block, dim, BF16, 5)
    starts = torch.tensor([0] + chunk).cumsum(0)
    q = rows((int(starts[-1]), heads * group, dim), BF16, 6)
    ref = q8.attention(q, (kc, vc), tables, starts, lens, 0.09, dim)
    for most in (max(chunk), 4096, (1 << 31) - 1):
        out = prefill(q, kc, vc, tables, starts, lens, 0.09, max_query_len=most, key_parts=parts)
        q8.assert_near(out, ref, BF16, 2, f"most {most}")
    assert pk.device_errors() == 0


@pytest.mark.parametrize("dtype,dim,block", [(F16, 64, 8), (BF16, 128, 16), (BF16, 64, 32)])
def test_nan_tokens_taken_back_and_kept_through_growth(dtype, dim, block):
    """A token with a NaN stays one when later rows make its block's scale grow, and leaves
    nothing behind when it is taken back, before the next token takes its place or after."""
    heads, group, n = 2, 2, block + 3
    tables, nb = q8.tables_for([2 * block], block, 3)
    kc, vc = (q8.new_pool(nb, heads, block, dim, i).cuda() for i in (1, 2))
    gt = tables.cuda()
    k, v = rows((n, heads, dim), dtype, 4), rows((n, heads, dim), dtype, 5)
    bad = k.clone()
    bad[block, 1, 7] = math.nan
    big = rows((1, heads, dim), dtype, 6, 300.0)
    q = rows((2, heads * group, dim), dtype, 7)

    def append(x, y, L):
        pk.paged_kv_append_q8(x.cuda(), y.cuda(), gt, i32([0, len(x)]), i32([L]), kc, vc)

    def check(L, what, nan):
        host = kc.cpu(), vc.cpu()
        ref = q8.attention(q[:1], host, tables, [0, 1], [L], 0.1, dim)
        assert bool(ref.isnan().any()) == nan, what
        for out in (decode(q[:1], kc, vc, gt, [L], 0.1, 0), prefill(q[:1], kc, vc, gt, [0, 1], [L], 0.1),
                    prefill(q[:1], kc, vc, gt, [0, 1], [L], 0.1, key_parts=32)):
            out = out.cpu()
            if nan:
                assert bool(out[0, group:].isnan().all()) and bool(torch.isfinite(out[0, :group]).all()), what
                q8.assert_near(out[:, :group], ref[:, :group], dtype, 2, what)
            else:
                q8.assert_near(out, ref, dtype, 2, what)

    append(bad[:block + 1], v[:block + 1], block + 1)
    check(block + 1, "appended", True)
    check(block, "taken back", False)
    append(bad[block:block + 1], v[block:block + 1], block + 1)
    append(big, big, block + 2)                              # its block's scales grow
    check(block + 2, "kept through growth", True)
    assert int(q8.views(kc.cpu(), dim)[2][int(tables[0, 1]), 1, 0]) & 3 == 1
    append(k[block:block + 2], v[block:block + 2], block + 2)    # both taken back, others in their place
    check(block + 2, "replaced", False)
    append(k[block + 1:block + 2], v[block + 1:block + 2], block + 2)
    check(block + 1, "part of it taken back", False)
    assert pk.device_errors() == 0


@pytest.mark.parametrize("dtype,small", [(F16, 2.0 ** -12), (BF16, 2.0 ** -90)])
@pytest.mark.parametrize("dim,block", [(64, 16), (128, 8)])
def test_small_queries_under_a_large_scale(dtype, small, dim, block):
    """Queries and keys as small as they come, and a scale that brings their scores back."""
    n, heads, group = 300, 2, 4
    least = 2.0 ** -10 if dtype == F16 else 2.0 ** -30
    kc, vc, tables = pools(rows((n, heads, dim), dtype, 1, least), rows((n, heads, dim), dtype, 2), block)
    q = (rows((70, heads * group, dim), torch.float32, 3) * small).to(dtype)
    scale = dim ** -0.5 / small / least
    ref = q8.attention(q, (kc, vc), tables, [0, 70], [n], scale, dim)
    for parts in (1, 32):
        q8.assert_near(prefill(q, kc, vc, tables, [0, 70], [n], scale, key_parts=parts), ref, dtype, 2, f"parts {parts}")
    for part in (0, 64, pk.PARTITION_BALANCED):
        q8.assert_near(decode(q[-1:], kc, vc, tables, [n], scale, part), ref[-1:], dtype, 2, f"part {part}")
    assert pk.device_errors() == 0
