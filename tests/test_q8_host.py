"""The 8-bit cache's entry points, forks and releases: what the host refuses
(nothing here reaches a GPU), and the definition the GPU tests compare with."""
import ctypes

import pytest
import torch

import paged_kv_cache_233_gb300 as pk
import q8_support as q8
from paged_kv_cache_233_gb300 import build as pk_build

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -5
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    pk_build.build()
    return pk.load()


def test_append_refuses_bad_arguments(lib):
    def call(**kw):
        a = dict(p=[16] * 7, S=3, T=4, MB=5, NB=8, B=16, H=2, D=64, dtype=1)
        a.update(kw)
        return lib.paged_kv_append_q8(*(vp(x) for x in a["p"]), a["S"], a["T"], a["MB"], a["NB"], a["B"], a["H"], a["D"],
                                      a["dtype"], None)

    for bad in (dict(S=-1), dict(T=-1), dict(MB=0), dict(NB=0), dict(H=0), dict(dtype=7)):
        assert call(**bad) == INVALID
    for bad in (dict(dtype=0), dict(D=96), dict(D=256), dict(B=12), dict(B=64), dict(S=4097), dict(T=1 << 30), dict(MB=1 << 28)):
        assert call(**bad) == UNSUPPORTED
    for i in range(7):
        assert call(p=[0 if j == i else 16 for j in range(7)]) == INVALID
        assert call(p=[18 if j == i else 16 for j in range(7)]) == INVALID   # misaligned
    assert call(T=0, p=[0] * 7) == 0
    assert call(S=0, p=[0] * 7) == 0


def test_gather_refuses_bad_arguments(lib):
    def call(**kw):
        a = dict(p=[16] * 5, T=4, NB=8, B=16, H=2, D=64, dtype=1)
        a.update(kw)
        return lib.paged_kv_gather_q8(*(vp(x) for x in a["p"]), a["T"], a["NB"], a["B"], a["H"], a["D"], a["dtype"], None)

    for bad in (dict(T=-1), dict(NB=0), dict(H=0), dict(dtype=7)):
        assert call(**bad) == INVALID
    for bad in (dict(dtype=0), dict(D=96), dict(B=12), dict(H=70000)):
        assert call(**bad) == UNSUPPORTED
    for i in range(5):
        assert call(p=[0 if j == i else 16 for j in range(5)]) == INVALID
        assert call(p=[20 if j == i else 16 for j in range(5)]) == INVALID
    assert call(T=0, p=[0] * 5) == 0


def test_decode_refuses_bad_arguments(lib):
    def call(**kw):
        a = dict(p=[1 << 12] * 5, scale=0.1, out=1 << 12, S=4, Hq=4, Hkv=2, D=64, NB=32, B=16, MB=5, P=0, ws=0,
                 n=0, dtype=1)
        a.update(kw)
        return lib.paged_attention_decode_q8(*(vp(x) for x in a["p"]), a["scale"], vp(a["out"]), a["S"], a["Hq"],
                                             a["Hkv"], a["D"], a["NB"], a["B"], a["MB"], a["P"], vp(a["ws"]), a["n"],
                                             a["dtype"], None)

    for bad in (dict(S=-1), dict(Hq=3), dict(MB=0), dict(scale=float("inf")), dict(scale=float("nan")), dict(P=-2), dict(P=48),
                dict(out=0), dict(out=8)):
        assert call(**bad) == INVALID
    for bad in (dict(dtype=0), dict(D=32), dict(B=4), dict(Hq=18), dict(S=4097)):
        assert call(**bad) == UNSUPPORTED
    for bad in (dict(P=32), dict(P=32, ws=1 << 12, n=64), dict(P=-1)):
        assert call(**bad) == WORKSPACE
    assert call(S=0, out=0) == 0


def test_prefill_refuses_bad_arguments(lib):
    def call(**kw):
        a = dict(p=[1 << 12] * 6, scale=0.1, out=1 << 12, S=2, T=9, n=5, Hq=4, Hkv=2, D=64, NB=32, B=16, MB=5, dtype=2,
                 parts=1)
        a.update(kw)
        return lib.paged_attention_prefill_q8(*(vp(x) for x in a["p"]), a["scale"], vp(a["out"]), a["S"], a["T"], a["n"],
                                              a["Hq"], a["Hkv"], a["D"], a["NB"], a["B"], a["MB"], a["dtype"],
                                              a["parts"], None, 0, None)

    for bad in (dict(T=-1), dict(n=-1), dict(parts=33), dict(parts=-1), dict(Hq=5), dict(scale=float("nan")), dict(out=0)):
        assert call(**bad) == INVALID
    for bad in (dict(dtype=0), dict(D=256), dict(Hq=130)):
        assert call(**bad) == UNSUPPORTED
    assert call(T=0, out=0) == 0
    assert call(S=0, out=0) == 0


@pytest.mark.parametrize("name", ["paged_kv_fork", "paged_kv_release"])
def test_page_calls_refuse_bad_arguments(lib, name):
    n = 9 if name == "paged_kv_fork" else 8

    def call(**kw):
        a = dict(p=[16] * n, S=4, MB=5, F=9, B=16, NB=32)
        a.update(kw)
        return getattr(lib, name)(*(vp(x) for x in a["p"]), a["S"], a["MB"], a["F"], a["B"], a["NB"], None)

    for bad in (dict(S=-1), dict(MB=0), dict(F=-1), dict(B=0), dict(NB=0)):
        assert call(**bad) == INVALID
    for bad in (dict(S=4097), dict(F=1 << 30), dict(NB=(1 << 24) + 1), dict(MB=1 << 28)):
        assert call(**bad) == UNSUPPORTED
    for i in range(n):
        assert call(p=[0 if j == i else 16 for j in range(n)]) == INVALID
        assert call(p=[18 if j == i else 16 for j in range(n)]) == INVALID
    assert call(S=0) == 0                            # in place: nothing to do


def test_binding_refuses_cpu_tensors_and_shapes(lib):
    k = torch.zeros(3, 2, 64, dtype=torch.float16)
    pool, i = pk.new_q8_pool(4, 2, 16, 64, device="cpu"), torch.zeros(3, dtype=torch.int32)
    assert pool.shape == (4, 2, 16, 65) and pk.new_q8_pool(4, 2, 8, 64, device="cpu").shape == (4, 2, 8, 66)
    tables = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(pk.PagedKVError, match="CUDA"):
        pk.paged_kv_append_q8(k, k, tables, i, i[:2], pool, pool)
    with pytest.raises(pk.PagedKVError, match="8-bit pools"):
        pk.paged_kv_append_q8(k, k, tables, i, i[:2], pool[..., :40], pool[..., :40])
    with pytest.raises(pk.PagedKVError, match="kv heads"):
        pk.paged_kv_gather_q8(pool, pool, i.long(), k[:, :1], k[:, :1])
    with pytest.raises(pk.PagedKVError, match="slot"):
        pk.paged_kv_gather_q8(pool, pool, i[:2].long(), k, k)
    with pytest.raises(pk.PagedKVError, match="query_start"):
        pk.paged_kv_append_q8(k, k, tables, i[:2], i[:2], pool, pool)
    with pytest.raises(pk.PagedKVError, match="sequences"):
        pk.paged_kv_fork(i, i[:2], tables, i, i, i[:1], torch.zeros(3, 2, dtype=torch.int32), 16)
    with pytest.raises(pk.PagedKVError, match="sequences"):
        pk.paged_kv_release(i, i, tables, i, i, i[:1], 16)
    with pytest.raises(pk.PagedKVError, match="one number"):
        pk.paged_kv_release(i[:2], i[:2], tables, i, i, i, 16)
    with pytest.raises(TypeError):
        pk.paged_kv_release(i[:2], i[:2], tables, None, i, i[:1], 16)
    with pytest.raises(pk.PagedKVError, match="block_size"):
        pk.new_q8_pool(4, 2, 12, 64, device="cpu")


def test_definition_of_the_codes():
    every = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    v = q8.value(every)
    assert torch.equal(v.nan_to_num(0.0), every.view(torch.float8_e4m3fn).double().nan_to_num(0.0))
    assert bool(v[[0x7F, 0xFF]].isnan().all()) and float(v[0x7E]) == 448
    real = every[~v.isnan()]
    assert torch.equal(q8.code(q8.value(real)), real)
    # half a step at most: 2^-4 of the value, 2^-10 below 2^-6
    x = torch.randn(4000, generator=torch.Generator().manual_seed(1)).double() * torch.exp2(torch.arange(4000) % 18 - 9.0)
    x = x.clamp(-448, 448)
    err = (q8.value(q8.code(x)) - x).abs()
    assert bool((err <= (x.abs() * 2.0 ** -4).clamp(min=2.0 ** -10)).all())


@pytest.mark.parametrize("top,e", [(0.0, -64), (448.0, 0), (448.5, 1), (224.0, -1), (1.0, -8), (65504.0, 8), (3.3e38, 120)])
def test_definition_of_the_scale(top, e):
    x = torch.tensor([top, -top / 2, float("nan"), float("-inf")], dtype=torch.float64)
    assert q8.exponent(x) == e
