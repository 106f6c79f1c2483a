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
