"""The 8-bit cache's definition in 64 bits, and pools built from it, for the tests.

Written from the definition alone: the tokens of a block and kv head share a scale
2^e, a channel is an e4m3 code c that stands for c * 2^e; a pool holds
[num_blocks][n_kv_heads] runs of codes [D / 16][B][16] followed by the scale in
fp32, 32 marks of tokens whose rows hold a NaN, and padding up to 16 bytes (32 in
blocks of 32).
"""
import math

import torch

from q4_support import HALF_STEP, TINY, assert_near, sequence_slots, tables_for  # noqa: F401  (for the tests)

NAN = 0x7F


def _table():
    """What the codes 0 .. 127 stand for: 3 bits of mantissa under 4 of exponent, bias 7."""
    v = [m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)]
    v[NAN] = math.nan
    return torch.tensor(v, dtype=torch.float64)


VALUES = _table()


def value(codes):
    c = codes.long()
    return torch.where(c >= 128, -VALUES[c % 128], VALUES[c % 128])


def code(x):
    """fp64 values to the nearest code, ties to the even one; NaN and infinities to NaN."""
    a = x.abs().nan_to_num(0.0, 0.0, 0.0)
    e = (torch.frexp(a.clamp(min=2.0 ** -7))[1] - 1).clamp(min=-6)   # the binade, smaller ones in that of 2^-6
    r = torch.round(torch.ldexp(a, 3 - e))                     # eighths of it: 8 .. 16, less below 2^-6
    c = ((e + 6) * 8 + r.int()).clamp(max=NAN - 1)             # (16 eighths are the next binade's 8)
    c = c + torch.where(torch.signbit(x), 128, 0)
    return torch.where(torch.isfinite(x), c, torch.full_like(c, NAN)).to(torch.uint8)   # (a NaN has no sign)


def exponent(x):
    """The smallest e >= -64 with |x| <= 448 * 2^e for every finite element (a Python int)."""
    a = x[torch.isfinite(x)].abs()
    top = float(a.max()) if a.numel() else 0.0
    e = -64
    while top > 448 * 2.0 ** e:
        e += 1
    return e


def tail(block):
    return max(16, block) // block


def new_pool(num_blocks, heads, block, dim, seed=0):
    """A pool of random bytes: stale contents, NaN codes and odd scales among them."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, 256, (num_blocks, heads, block, dim + tail(block)), generator=g, dtype=torch.int32).to(torch.uint8)


def views(pool, dim):
    """Codes [NB][Hkv][D / 16][B][16], scales [NB][Hkv][1] and marks [NB][Hkv][1] (int32)."""
    nb, heads, block, _ = pool.shape
    flat, at = pool.view(nb, heads, -1), block * dim
    return (flat[..., :at].unflatten(-1, (dim // 16, block, 16)), flat[..., at:at + 4].view(torch.float32),
            flat[..., at + 4:at + 8].view(torch.int32))


def marks(rows):
    """The marks of rows [n][D] as the first tokens of a block (a Python int)."""
    return sum(1 << t for t in range(len(rows)) if not bool(torch.isfinite(rows[t]).all()))


def signed(x):
    return x - (1 << 32) if x >= 1 << 31 else x


def append(pool, x, tables, starts, lens):
    """Rows [T][Hkv][D] (a CPU tensor of a 16-bit type) into a CPU pool behind each sequence's older tokens."""
    block, dim = pool.shape[2], x.shape[-1]
    codes, scale, mark = views(pool, dim)
    x = x.double()
    for s, L in enumerate(int(n) for n in lens):
        a, b = int(starts[s]), int(starts[s + 1])
        old = L - (b - a)
        if a == b:
            continue
        for j in range(old // block, -(-L // block)):
            bid = int(tables[s, j])
            first, end = max(old, j * block), min(L, (j + 1) * block)
            held = first - j * block                       # older tokens in front of them, if any
            new = x[a + first - old:a + end - old]         # [n][Hkv][D]
            for h in range(x.shape[1]):
                e = exponent(new[:, h])
                if held:
                    before = int(math.log2(float(scale[bid, h, 0])))
                    if before > e:
                        e = before
                    elif before < e:
                        was = codes[bid, h, :, :held]
                        codes[bid, h, :, :held] = code(value(was) * 2.0 ** (before - e))
                c = code(new[:, h] * 2.0 ** -e)            # [n][D]
                codes[bid, h, :, held:held + len(new)] = c.unflatten(-1, (-1, 16)).transpose(0, 1)
                scale[bid, h, 0] = 2.0 ** e
                old_marks = int(mark[bid, h, 0]) & ((1 << held) - 1)
                mark[bid, h, 0] = signed(old_marks | marks(new[:, h]) << held)


def read(pool, slots, dim):
    """fp64 rows [T][Hkv][D] of a CPU pool."""
    block = pool.shape[2]
    codes, scale, _ = views(pool, dim)
    b, o = slots // block, slots % block
    return value(codes[b, :, :, o]).flatten(-2) * scale[b].double()


def filled(lens, heads, block, dim, dtype, seed, spread=1.0, pad=0):
    """Pools whose sequences hold N(0, spread) rows (each block's scale its own: every
    third one is larger than it has to be), stale bytes elsewhere."""
    tables, nb = tables_for(lens, block, seed, pad=pad)
    g = torch.Generator().manual_seed(seed + 1)
    pools = [new_pool(nb, heads, block, dim, seed + 2 + i) for i in range(2)]
    for s, n in enumerate(int(n) for n in lens):
        for pool in pools:
            fill(pool, tables[s], (torch.randn(n, heads, dim, generator=g) * spread).to(dtype))
    return pools[0], pools[1], tables


def fill(pool, table, x):
    """A sequence's rows x [n][Hkv][D] into its blocks, all at once (whole blocks: what
    lies behind the last row becomes zeros and NaN)."""
    block, dim, n = pool.shape[2], x.shape[-1], len(x)
    blocks = -(-n // block)
    if n == 0:
        return
    codes, scale, mark = views(pool, dim)
    rows = torch.zeros(blocks * block, *x.shape[1:], dtype=torch.float64)
    rows[:n] = x.double()
    rows = rows.unflatten(0, (blocks, block))                  # [blocks][B][Hkv][D]
    top = rows.abs().amax((1, 3)).clamp(min=448 * 2.0 ** -64)
    e = torch.ceil(torch.log2(top / 448)) + (torch.arange(blocks) % 3 == 2)[:, None]
    c = code(rows * torch.exp2(-e)[:, None, :, None])
    if n % block:
        c[-1, n % block:, :, ::3] = NAN
    ids = torch.as_tensor(table)[:blocks].long()
    codes[ids] = c.unflatten(-1, (-1, 16)).permute(0, 2, 3, 1, 4)
    scale[ids, :, 0] = torch.exp2(e).float()
    mark[ids] = 0


def attention(q, pools, tables, starts, lens, scale, dim):
    """fp64 causal attention of rows starts[s] .. starts[s + 1] over sequence s's
    first lens[s] tokens (the chunk its last ones); zero rows without keys."""
    out = torch.zeros(q.shape, dtype=torch.float64)
    heads = pools[0].shape[1]
    group, block = q.shape[1] // heads, pools[0].shape[2]
    for s, n in enumerate(int(n) for n in lens):
        a, b = int(starts[s]), int(starts[s + 1])
        if n == 0 or a == b:
            continue
        k, v = (read(p, sequence_slots(tables, s, n, block), dim) for p in pools)
        x = q[a:b].double().unflatten(1, (heads, group))
        z = torch.einsum("rhgd,khd->rhgk", x, k) * scale
        seen = torch.arange(n)[None] <= torch.arange(n - (b - a), n)[:, None]
        w = torch.softmax(z.masked_fill(~seen[:, None, None], float("-inf")), -1)
        out[a:b] = torch.einsum("rhgk,khd->rhgd", w, v).flatten(1, 2)
    return out
