"""The 4-bit decode on values at the ends of what its arithmetic takes."""
import pytest
import torch

import paged_kv_cache_233_gb300 as pk
import q4_support as q4

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
SPLITS = [0, 32, 64, pk.PARTITION_BALANCED]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pk.load()
    torch.cuda.set_device(0)
    pk.device_errors()


def rows(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def pools(k, v, block, seed=1):
    """One sequence's K and V [n][Hkv][D] in 4-bit pools of stale bytes, and its table."""
    n, heads, dim = k.shape
    tables, nb = q4.tables_for([n], block, seed)
    out = []
    for i, x in enumerate((k, v)):
        pool = q4.new_pool(nb, heads, block, dim, seed + i)
        q4.write_fast(pool, q4.sequence_slots(tables, 0, n, block), x)
        out.append(pool)
    return out[0], out[1], tables


def decode(q, kc, vc, tables, lens, scale, part):
    out = torch.full_like(q, 7.0).cuda()
    q, tables = q.cuda(), tables.cuda()
    ws = pk.new_workspace(q, tables, kc.shape[2], part)
    if ws is not None:
        ws.fill_(255)                          # NaN
    pk.paged_attention_decode_q4(q, kc.cuda(), vc.cuda(), tables, torch.tensor(lens, dtype=torch.int32).cuda(), scale, out,
                                 part, ws)
    return out.cpu()


def check(q, k, v, block, scale, what):
    dtype, dim = q.dtype, q.shape[2]
    kc, vc, tables = pools(k, v, block)
    n = k.shape[0]
    ref = q4.attention(q, (kc, vc), tables, [0, 1], [n], scale, dim, dtype)
    for part in SPLITS:
        got = decode(q, kc, vc, tables, [n], scale, part)
        # the output is rounded, and so are the probabilities (times a scale)
        q4.assert_near(got, ref, dtype, 2, f"{what} part {part}")
    assert pk.device_errors() == 0


# ------------------------------------------- scales of the values, small and none
@pytest.mark.parametrize("heads,dim,block", [(4, 128, 16), (2, 64, 8), (1, 128, 32)])
@pytest.mark.parametrize("flat", [0.0, 0.5, 1e-4])
def test_fp16_flat_values_before_small_ones(flat, heads, dim, block):
    """Tiles whose groups have no spread (scale 0), then tiles of size 1e-4."""
    n = 200
    v = (rows((n, heads, dim), 3) * 1e-4).to(F16)
    v[:64] = flat
    v[130:140] = flat
    check(rows((1, heads * 2, dim), 1).to(F16), rows((n, heads, dim), 2).to(F16), v, block, dim ** -0.5, f"flat {flat}")


@pytest.mark.parametrize("heads,dim,block", [(4, 128, 16), (2, 64, 8), (1, 128, 32)])
@pytest.mark.parametrize("rise", [20.0, -20.0])
def test_fp16_scales_from_the_smallest_with_moving_scores(rise, heads, dim, block):
    """Values from 15 steps of 2^-24 to a spread of 15 * 2^-13, over tiles of 32 tokens,
    while the scores rise or fall by `rise` in all."""
    n = 32 * 8
    step = 2.0 ** (-24 + (torch.arange(n) // 32 * 1.5).round())           # 2^-24 .. 2^-14 (or -13)
    code = torch.randint(0, 16, (n, heads, dim), generator=torch.Generator().manual_seed(4))
    v = (code * step[:, None, None]).to(F16)
    k = rows((n, heads, dim), 2) * 0.3
    k[..., 0] += torch.linspace(0, rise / 8, n)[:, None]
    q = rows((1, heads * 2, dim), 1) * 0.5
    q[..., 0] = 8.0
    check(q.to(F16), k.to(F16), v, block, 1.0, f"rise {rise}")


# --------------------------------------------------------------- NaN goes through
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads", [1, 2, 3, 4])
@pytest.mark.parametrize("what", ["query", "key", "key tile", "first key tile", "value", "value tile", "all keys"])
def test_nan_reaches_the_outputs(what, heads, dtype):
    """A NaN in a query, in one key or value, or in a whole tile of them beside clean
    ones makes the rows that attend to it NaN (a value's: its group's channels; the
    rest of that head may be), and no others."""
    n, dim, block, group = 160, 64, 16, 3
    k, v = rows((n, heads, dim), 2).to(dtype), rows((n, heads, dim), 3).to(dtype)
    q = rows((1, heads * group, dim), 1).to(dtype)
    h = heads - 1
    bad = torch.zeros(heads * group, dtype=torch.bool)
    bad[h * group:] = True
    sure = bad
    if what == "query":
        q[0, -1, 5] = float("nan")
        bad[:-1] = False
    else:
        x = v if what.startswith("value") else k
        at = {"tile": slice(64, 96), "keys": slice(0, n)}.get(what.split()[-1], slice(70, 71))
        if what.startswith("first"):
            at = slice(0, 32)
        x[at, h, 40] = float("nan")
        if what.startswith("value"):
            sure = bad[:, None] & (torch.arange(dim) >= 32)
    kc, vc, tables = pools(k, v, block)
    for part in SPLITS:
        got = decode(q, kc, vc, tables, [n], dim ** -0.5, part)[0]
        assert bool(got[sure].isnan().all()), f"part {part}"
        assert bool(torch.isfinite(got[~bad]).all()), f"part {part}"
    assert pk.device_errors() == 0


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("what", ["query", "key", "keys"])
@pytest.mark.parametrize("parts", [1, 8])
def test_nan_reaches_the_outputs_of_a_prefill(what, parts, bits):
    """The rows that attend to a NaN are NaN, split over the keys or not, and the
    other rows are what they are without it, whatever the workspace held."""
    n, rows_n, heads, group, dim, block = 6000, 40, 2, 2, 64, 16
    k, v = rows((n, heads, dim), 2).to(F16), rows((n, heads, dim), 3).to(F16)
    q = rows((rows_n, heads * group, dim), 1).to(F16)
    clean = torch.ones(rows_n, heads * group, dtype=torch.bool)
    starts, lens = torch.tensor([0, rows_n], dtype=torch.int32).cuda(), torch.tensor([n], dtype=torch.int32).cuda()

    def run(fill):
        if bits == 4:
            kc, vc, tables = pools(k, v, block)
            f = pk.paged_attention_prefill_q4
        else:
            tables, nb = q4.tables_for([n], block, 1)
            at = q4.sequence_slots(tables, 0, n, block)
            kc, vc = (torch.zeros(nb * block, heads, dim, dtype=F16).index_copy_(0, at, x).view(nb, block, heads, dim)
                      for x in (k, v))
            f = pk.paged_attention_prefill
        out = torch.full_like(q, 7.0).cuda()
        ws = pk.prefill_workspace(q.cuda())
        ws.fill_(fill)
        f(q.cuda(), kc.cuda(), vc.cuda(), tables.cuda(), starts, lens, 0.125, out, rows_n, workspace=ws, key_parts=parts)
        return out.cpu()

    want = run(0)
    if what == "query":
        q[7, 3, 5] = float("nan")
        clean[7, 3] = False
    else:
        at = slice(n - 20, n - 19) if what == "key" else slice(1500, 3500)     # (3500: several whole pieces)
        k[at, 1, 40] = float("nan")
        clean[20 if what == "key" else 0:, group:] = False
    for fill in (0, 255):
        got = run(fill)
        assert bool(got[~clean].isnan().all())
        assert torch.equal(got[clean], want[clean])
    assert pk.device_errors() == 0


# ------------------------------------------------- values far larger than others
@pytest.mark.parametrize("heads,dim,block", [(4, 128, 16), (2, 64, 8)])
@pytest.mark.parametrize("dtype,size", [(F16, 6e4), (F16, -1.0), (BF16, 1e10), (BF16, -1e15), (BF16, 1e19), (BF16, 1e-10)])
def test_flat_values_of_any_size(dtype, size, heads, dim, block):
    """Groups without spread, whose middles are all there is, alone and before and
    after tiles of other sizes."""
    q, k = rows((1, heads * 2, dim), 1).to(dtype), rows((150, heads, dim), 2).to(dtype)
    v = torch.full((150, heads, dim), size)
    check(q, k, v.to(dtype), block, dim ** -0.5, "flat")
    v[40:80] = rows((40, heads, dim), 3) * abs(size) * 0.25
    check(q, k, v.to(dtype), block, dim ** -0.5, "some flat")
    v[:40], v[120:] = 0, size / 1000
    check(q, k, v.to(dtype), block, dim ** -0.5, "some zero")


@pytest.mark.parametrize("heads,dim,block", [(4, 128, 16), (2, 64, 8)])
@pytest.mark.parametrize("dtype,factor,base", [(F16, 1e4, 1.0), (F16, 1e6, 1e-2), (BF16, 1e4, 1.0), (BF16, 1e7, 1.0),
                                               (BF16, 1e10, 1.0)])
@pytest.mark.parametrize("at", [5, 70, 299])
def test_a_token_of_large_values_and_no_weight(dtype, factor, base, at, heads, dim, block):
    """One token whose values are `factor` times the others', with a weight of about e^-60."""
    n, scale = 300, 0.5
    q = rows((1, heads * 2, dim), 1)
    q[:, 1::2] = q[:, ::2]
    k = rows((n, heads, dim), 2) * 0.3
    k[at] = -q[0, ::2] * 60 / scale / (q[0, ::2] ** 2).sum(-1, keepdim=True)
    v = rows((n, heads, dim), 3) * base
    v[at] *= factor
    check(q.to(dtype), k.to(dtype), v.to(dtype), block, scale, "outlier")


# ------------------------------------------------------------ far middles, repeats
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads,dim,block", [(4, 128, 16), (2, 64, 8)])
@pytest.mark.parametrize("middle,mean", [(20.0, 1.0), (-100.0, 1.0), (20.0, -6.0)])
def test_keys_far_off_zero_under_queries_of_one_sign(middle, mean, heads, dim, block, dtype):
    """A score's part in the groups' middles is far larger than the scores' spread. A
    group's sum of q is held in two parts of the type: off by half a step of the
    second, h^2 of the sum, times 72 s + |m|; its products and sums are fp32 ones."""
    n, group = 400, 3
    q = (rows((1, heads * group, dim), 1) + mean).to(dtype)
    k = (rows((n, heads, dim), 2) + middle * torch.sign(rows((heads, dim // 32), 4)).repeat_interleave(32, 1)).to(dtype)
    v = rows((n, heads, dim), 3).to(dtype)
    kc, vc, tables = pools(k, v, block)
    scale = dim ** -0.5
    ref = q4.attention(q, (kc, vc), tables, [0, 1], [n], scale, dim, dtype)
    _, s, m, _ = q4.quantise(k)
    far = (72 * s.double() + m.double().abs()).amax(0)[..., 0]                       # [heads][groups]
    sums = q[0].double().unflatten(1, (-1, 32)).sum(-1).abs().unflatten(0, (heads, group))
    wide = q[0].double().unflatten(1, (-1, 32)).abs().sum(-1).unflatten(0, (heads, group))
    off = (q4.HALF_STEP[dtype] ** 2 * sums + 8 * 2.0 ** -24 * wide) * far[:, None]
    worst = scale * float(off.sum(-1).max())
    for part in SPLITS:
        got = decode(q, kc, vc, tables, [n], scale, part).double()
        # scores off by `worst` change a weight by a factor of up to e^(2 worst); beside the roundings
        rel = float((got - ref).norm() / ref.norm())
        assert rel <= 2 * q4.HALF_STEP[dtype] + 2.2 * worst, f"part {part}: {rel:.2e}, scores {worst:.2e}"
    assert worst < 0.25 and pk.device_errors() == 0


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_every_call_repeats_bit_for_bit(dtype):
    heads, group, dim, block = 8, 4, 128, 16
    lens = [3000, 17, 900, 64, 2500, 1]
    kc, vc, tables = (x.cuda() for x in q4.filled(lens, heads, block, dim, dtype, 6))
    L = torch.tensor(lens, dtype=torch.int32).cuda()
    q = rows((len(lens), heads * group, dim), 1).to(dtype).cuda()
    chunk = [min(n, 70) for n in lens]
    starts = torch.tensor([0] + chunk).cumsum(0).to(torch.int32).cuda()
    qp = rows((sum(chunk), heads * group, dim), 2).to(dtype).cuda()
    x = rows((500, heads, dim), 3).to(dtype).cuda()
    slots = torch.randperm(kc.shape[0] * block, generator=torch.Generator().manual_seed(1))[:500].cuda()

    def run():
        out = []
        for part in SPLITS:
            y = torch.empty_like(q)
            pk.paged_attention_decode_q4(q, kc, vc, tables, L, 0.09, y, part, pk.new_workspace(q, tables, block, part))
            out.append(y)
        for parts in (1, 0, 7):
            y = torch.empty_like(qp)
            pk.paged_attention_prefill_q4(qp, kc, vc, tables, starts, L, 0.09, y, 70, key_parts=parts)
            out.append(y)
        a, b = kc.clone(), vc.clone()
        pk.paged_kv_append_q4(x, x, slots, a, b)
        return [*out, a, b]

    first = run()
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(first, run()))
    assert pk.device_errors() == 0
