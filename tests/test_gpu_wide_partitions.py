"""Partitions wider than any context: the decode as a whole, whatever the number."""
import pytest
import torch

import paged_kv_cache_233_gb300 as pk
import q4_support as q4
import q8_support as q8

pytestmark = pytest.mark.gpu
F16 = torch.float16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pk.load()
    torch.cuda.set_device(0)
    pk.device_errors()


@pytest.mark.parametrize("part", [1 << 20, 1 << 30, (1 << 31) - 32])
@pytest.mark.parametrize("bits", [4, 8, 16])
def test_partitions_wider_than_the_contexts(bits, part):
    lens, heads, dim, block = [0, 1, 33, 34, 300], 4, 64, 16
    if bits == 16:
        tables, nb = q4.tables_for(lens, block, 3)
        g = torch.Generator().manual_seed(1)
        kc, vc = (torch.randn(nb, block, heads, dim, generator=g).to(F16) for _ in range(2))
        decode = pk.paged_attention_decode
    else:
        kc, vc, tables = (q4 if bits == 4 else q8).filled(lens, heads, block, dim, F16, 3)
        decode = pk.paged_attention_decode_q4 if bits == 4 else pk.paged_attention_decode_q8
    q = torch.randn(len(lens), heads * 2, dim, generator=torch.Generator().manual_seed(2)).to(F16).cuda()
    kc, vc, tables, n = kc.cuda(), vc.cuda(), tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    outs = [torch.full_like(q, 7.0) for _ in range(2)]
    decode(q, kc, vc, tables, n, 0.125, outs[0])
    decode(q, kc, vc, tables, n, 0.125, outs[1], part, ws)
    assert torch.equal(outs[0], outs[1]) and not bool((outs[0] == 7).all(-1).any())
    assert pk.device_errors() == 0
