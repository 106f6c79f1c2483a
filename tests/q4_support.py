"""The 4-bit cache's definition in 64 bits, and pools built from it, for the tests.

Written from the definition alone: groups of 32 channels, a scale s and a
middle m of the cache's 16-bit type, codes c of 0 .. 15 that stand for
s * (c - 8) + m; a pool holds [num_blocks][n_kv_heads] runs of codes
[D / 32][B][16 bytes] followed by (s, m) pairs [B][D / 32].
"""
import numpy as np
import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}   # finfo.eps / 2
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}      # half the smallest step


def toward_zero(x, dtype):
    """fp32 values >= 0 rounded down to a 16-bit type."""
    y = x.to(dtype)
    over = y.float() > x
    y[over] = (y.view(torch.int16)[over] - 1).view(dtype)
    return y


def quantise(x):
    """CPU tensor [..., D] of a 16-bit type -> (codes 0..15 [..., G, 32], s, m
    [..., G, 1] of that type, the quotients the codes are rounded from)."""
    y = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32).float()
    lo, hi = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
    s = toward_zero((hi - lo) / 15, x.dtype)
    m = ((0.5 * lo + 0.5 * hi) + 0.5 * s.float()).to(x.dtype)
    t = (y - m.float()).double() / s.double()
    c = torch.where((s > 0) & torch.isfinite(s), t.round().clamp(-8, 7) + 8, torch.full_like(t, 8))
    return c.to(torch.uint8), s, m, t


def stands_for(c, s, m):
    return (s.double() * (c.double() - 8) + m.double()).flatten(-2)


def new_pool(num_blocks, heads, block, dim, seed=0):
    """A pool of random bytes: stale contents, NaN scales among them."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, 256, (num_blocks, heads, block, dim * 5 // 8), generator=g, dtype=torch.int32).to(torch.uint8)


def views(pool, dim, dtype):
    nb, heads, block, _ = pool.shape
    flat, groups = pool.view(nb, heads, -1), dim // 32
    codes = flat[..., :block * dim // 2].unflatten(-1, (groups, block, 16))
    pairs = flat[..., block * dim // 2:].view(dtype).unflatten(-1, (block, groups, 2))
    return codes, pairs


def write(pool, slots, x):
    """Quantise rows [T][Hkv][D] into a CPU pool at slots >= 0."""
    block = pool.shape[2]
    codes, pairs = views(pool, x.shape[-1], x.dtype)
    c, s, m, _ = quantise(x)
    for t, slot in enumerate(slots.tolist()):
        if slot < 0:
            continue
        b, o = divmod(slot, block)
        codes[b, :, :, o] = c[t][..., 0::2] | (c[t][..., 1::2] << 4)
        pairs[b, :, o] = torch.cat([s[t], m[t]], -1)


def read(pool, slots, dim, dtype):
    """fp64 rows [T][Hkv][D] of a CPU pool."""
    block = pool.shape[2]
    codes, pairs = views(pool, dim, dtype)
    b, o = slots // block, slots % block
    raw = codes[b, :, :, o]                                     # [T][Hkv][G][16]
    c = torch.stack([raw % 16, raw // 16], -1).flatten(-2)
    p = pairs[b, :, o]
    return stands_for(c, p[..., 0:1], p[..., 1:2])


def tables_for(lens, block, seed, spare=2, pad=0):
    """Shuffled block tables [S][width + pad] (-1 past a sequence's blocks) and the pool's block count."""
    rng = np.random.default_rng(seed)
    need = [-(-int(n) // block) for n in lens]
    ids = rng.permutation(sum(need) + spare)
    tables = np.full((len(lens), max([1] + need) + pad), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = ids[at:at + n]
        at += n
    return torch.from_numpy(tables), len(ids)


def sequence_slots(tables, s, n, block):
    i = torch.arange(n)
    return tables[s].long()[i // block] * block + i % block


def filled(lens, heads, block, dim, dtype, seed, spread=1.0, pad=0):
    """Pools whose sequences hold N(0, spread) rows, stale bytes elsewhere."""
    tables, nb = tables_for(lens, block, seed, pad=pad)
    g = torch.Generator().manual_seed(seed + 1)
    pools = [new_pool(nb, heads, block, dim, seed + 2 + i) for i in range(2)]
    for s, n in enumerate(lens):
        for pool in pools:
            x = (torch.randn(int(n), heads, dim, generator=g) * spread).to(dtype)
            write_fast(pool, sequence_slots(tables, s, int(n), block), x)
    return pools[0], pools[1], tables


def write_fast(pool, slots, x):
    """write() for slots that are all valid and distinct, without a loop."""
    block = pool.shape[2]
    codes, pairs = views(pool, x.shape[-1], x.dtype)
    c, s, m, _ = quantise(x)
    b, o = slots // block, slots % block
    codes[b, :, :, o] = c[..., 0::2] | (c[..., 1::2] << 4)
    pairs[b, :, o] = torch.cat([s, m], -1)


def attention(q, pools, tables, starts, lens, scale, dim, dtype):
    """fp64 causal attention of rows starts[s] .. starts[s + 1] over sequence s's
    first lens[s] tokens (the chunk its last ones); zero rows without keys."""
    out = torch.zeros(q.shape, dtype=torch.float64)
    heads = pools[0].shape[1]
    group, block = q.shape[1] // heads, pools[0].shape[2]
    for s, n in enumerate(lens):
        a, b = int(starts[s]), int(starts[s + 1])
        n = int(n)
        if n == 0 or a == b:
            continue
        k, v = (read(p, sequence_slots(tables, s, n, block), dim, dtype) for p in pools)
        x = q[a:b].double().unflatten(1, (heads, group))
        z = torch.einsum("rhgd,khd->rhgk", x, k) * scale
        seen = torch.arange(n)[None] <= torch.arange(n - (b - a), n)[:, None]
        w = torch.softmax(z.masked_fill(~seen[:, None, None], float("-inf")), -1)
        out[a:b] = torch.einsum("rhgk,khd->rhgd", w, v).flatten(1, 2)
    return out


def assert_near(got, ref, dtype, roundings, what=""):
    """Error of 16-bit outputs against fp64 ones. `roundings` counts the values
    on the way that are rounded to the 16-bit type, each off by at most half a
    step h and independent of the others: their relative 2-norm is below
    roundings * h (uniform errors have a root mean square of h / sqrt(3), and
    independent ones add in squares, so this leaves a factor of at least 1.7).
    A single output is allowed six times that of the outputs' root mean square
    beside its own rounding."""
    g, h = got.detach().cpu().double(), HALF_STEP[dtype]
    assert torch.isfinite(g).all(), f"{what}: non-finite outputs"
    if not g.numel():
        return
    norm = float(ref.norm())
    rel = float((g - ref).norm()) / max(norm, 1e-300)
    assert rel <= roundings * h or float((g - ref).abs().max()) <= 4 * TINY[dtype], f"{what}: relative error {rel:.3e}"
    rms = norm / ref.numel() ** 0.5
    worst = float(((g - ref).abs() - (roundings + 1) * h * ref.abs()).max())
    assert worst <= 6 * roundings * h * rms + 4 * TINY[dtype], f"{what}: an output is {worst:.3e} off, rms {rms:.3e}"
