"""The 4-bit cache's entry points and paged_kv_build_tables: what the host refuses
(nothing here reaches a GPU), and the definition the GPU tests compare with."""
import ctypes

import pytest
import torch

import paged_kv_cache_233_gb300 as pk
import q4_support as q4
from paged_kv_cache_233_gb300 import build as pk_build

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -5
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    pk_build.build()
    return pk.load()


@pytest.mark.parametrize("name", ["paged_kv_append_q4", "paged_kv_gather_q4"])
def test_row_calls_refuse_bad_arguments(lib, name):
    def call(**kw):
        a = dict(p=[16] * 5, T=4, NB=8, B=16, H=2, D=64, dtype=1)
        a.update(kw)
        return getattr(lib, name)(*(vp(x) for x in a["p"]), a["T"], a["NB"], a["B"], a["H"], a["D"], a["dtype"], None)

    assert call(T=-1) == INVALID
    assert call(NB=0) == INVALID
    assert call(H=0) == INVALID
    assert call(dtype=7) == INVALID
    assert call(dtype=0) == UNSUPPORTED              # fp32
    assert call(D=96) == UNSUPPORTED
    assert call(B=12) == UNSUPPORTED
    assert call(B=64) == UNSUPPORTED
    for i in range(5):
        assert call(p=[0 if j == i else 16 for j in range(5)]) == INVALID
        assert call(p=[20 if j == i else 16 for j in range(5)]) == INVALID   # misaligned
    assert call(T=0, p=[0] * 5) == 0


def test_decode_refuses_bad_arguments(lib):
    def call(**kw):
        a = dict(p=[1 << 12] * 5, scale=0.1, out=1 << 12, S=4, Hq=4, Hkv=2, D=64, NB=32, B=16, MB=5, P=0, ws=0,
                 n=0, dtype=1)
        a.update(kw)
        return lib.paged_attention_decode_q4(*(vp(x) for x in a["p"]), a["scale"], vp(a["out"]), a["S"], a["Hq"],
                                             a["Hkv"], a["D"], a["NB"], a["B"], a["MB"], a["P"], vp(a["ws"]), a["n"],
                                             a["dtype"], None)

    assert call(S=-1) == INVALID
    assert call(Hq=3) == INVALID
    assert call(MB=0) == INVALID
    assert call(scale=float("inf")) == INVALID
    assert call(P=-2) == INVALID
    assert call(P=48) == INVALID                      # not a multiple of 32
    assert call(dtype=0) == UNSUPPORTED
    assert call(D=32) == UNSUPPORTED
    assert call(B=4) == UNSUPPORTED
    assert call(Hq=18) == UNSUPPORTED                 # group of 9
    assert call(S=4097) == UNSUPPORTED
    assert call(P=32) == WORKSPACE
    assert call(P=32, ws=1 << 12, n=64) == WORKSPACE
    assert call(P=-1) == WORKSPACE
    assert call(out=0) == INVALID
    assert call(out=8) == INVALID
    assert call(S=0, out=0) == 0


def test_prefill_refuses_bad_arguments(lib):
    def call(**kw):
        a = dict(p=[1 << 12] * 6, scale=0.1, out=1 << 12, S=2, T=9, n=5, Hq=4, Hkv=2, D=64, NB=32, B=16, MB=5, dtype=2,
                 parts=1)
        a.update(kw)
        return lib.paged_attention_prefill_q4(*(vp(x) for x in a["p"]), a["scale"], vp(a["out"]), a["S"], a["T"], a["n"],
                                              a["Hq"], a["Hkv"], a["D"], a["NB"], a["B"], a["MB"], a["dtype"],
                                              a["parts"], None, 0, None)

    assert call(T=-1) == INVALID
    assert call(n=-1) == INVALID
    assert call(parts=33) == INVALID
    assert call(parts=-1) == INVALID
    assert call(Hq=5) == INVALID
    assert call(scale=float("nan")) == INVALID
    assert call(dtype=0) == UNSUPPORTED
    assert call(D=256) == UNSUPPORTED
    assert call(Hq=130) == UNSUPPORTED                # group of 65
    assert call(out=0) == INVALID
    assert call(T=0, out=0) == 0
    assert call(S=0, out=0) == 0


def test_build_tables_refuses_bad_arguments(lib):
    def call(**kw):
        a = dict(p=[16] * 11, S=4, MB=5, F=9, T=6, B=16, NB=32)
        a.update(kw)
        return lib.paged_kv_build_tables(*(vp(x) for x in a["p"]), a["S"], a["MB"], a["F"], a["T"], a["B"], a["NB"], None)

    assert call(S=-1) == INVALID
    assert call(MB=0) == INVALID
    assert call(F=-1) == INVALID
    assert call(T=-1) == INVALID
    assert call(B=0) == INVALID
    assert call(NB=0) == INVALID
    assert call(S=4097) == UNSUPPORTED
    assert call(T=1 << 30) == UNSUPPORTED
    assert call(F=1 << 30) == UNSUPPORTED
    assert call(MB=1 << 28) == UNSUPPORTED
    for i in range(11):
        if i != 8:                                    # the slots are optional
            assert call(p=[0 if j == i else 16 for j in range(11)]) == INVALID
        assert call(p=[18 if j == i else 16 for j in range(11)]) == INVALID


def test_binding_refuses_cpu_tensors_and_shapes(lib):
    k = torch.zeros(3, 2, 64, dtype=torch.float16)
    slots, pool = torch.zeros(3, dtype=torch.int64), torch.zeros(4, 2, 16, 40, dtype=torch.uint8)
    with pytest.raises(pk.PagedKVError, match="CUDA"):
        pk.paged_kv_append_q4(k, k, slots, pool, pool)
    with pytest.raises(pk.PagedKVError, match="4-bit pools"):
        pk.paged_kv_append_q4(k, k, slots, pool[..., :32], pool[..., :32])
    with pytest.raises(pk.PagedKVError, match="kv heads"):
        pk.paged_kv_gather_q4(pool, pool, slots, k[:, :1], k[:, :1])
    with pytest.raises(pk.PagedKVError, match="slot"):
        pk.paged_kv_append_q4(k, k, slots[:2], pool, pool)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(pk.PagedKVError, match="requests"):
        pk.paged_kv_build_tables(i, i, torch.zeros(3, 4, dtype=torch.int32), i, i[:1], 16, 9, i, i, i)
    with pytest.raises(pk.PagedKVError, match="length"):
        pk.paged_kv_build_tables(i, i, torch.zeros(3, 4, dtype=torch.int32), i, i[:1], 16, 9,
                                 torch.zeros(4, dtype=torch.int32), i, i[:2])
    with pytest.raises(pk.PagedKVError):
        pk.new_q4_pool(4, 2, 16, 80, device="cpu")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_definition_stays_within_half_a_step(dtype):
    """What a code stands for is off by at most half a scale, and at a group's
    ends by what rounding s down and m to nearest leave out: 15 s is short of
    hi - lo by up to 15 steps of s, half on each side, beside half a step of m."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(50, 4, 128, generator=g).to(dtype)
    c, s, m, _ = q4.quantise(x)
    err = (q4.stands_for(c, s, m) - x.double()).abs().unflatten(-1, (-1, 32))
    h = q4.HALF_STEP[dtype]
    allowed = s.double() * (0.5 + 15 * h) + m.double().abs() * h
    assert bool((err <= allowed).all())
    assert int(c.min()) == 0 and int(c.max()) == 15


def test_definition_of_flat_and_broken_groups():
    x = torch.full((1, 1, 64), 3.25, dtype=torch.float16)
    x[0, 0, 40] = float("nan")
    c, s, m, _ = q4.quantise(x)
    y = q4.stands_for(c, s, m)
    assert float(s[0, 0, 0]) == 0 and bool((c[0, 0, 0] == 8).all()) and bool((y[0, 0, :32] == 3.25).all())
    assert bool(y[0, 0, 32:].isnan().all())


@pytest.mark.parametrize("shape", [(4, 16, 2, 64), (4, 2, 16, 41), (4, 2, 16, 20), (4, 2, 1, 40), (4, 2, 16, 160)])
def test_uint8_pools_that_are_no_4_bit_pools_are_refused(lib, shape):
    pool, pairs = torch.zeros(shape, dtype=torch.uint8), torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(pk.PagedKVError, match="4-bit"):
        pk.paged_kv_copy_blocks(pool, pool, pairs)
    with pytest.raises(pk.PagedKVError, match="4-bit"):
        pk.paged_kv_swap_blocks(pool, pool, pool, pool, pairs)
