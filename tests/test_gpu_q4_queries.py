"""The 4-bit decode with queries at the end of bfloat16's range."""
import pytest
import torch

from test_gpu_q4_values import BF16, check, gpu, rows  # noqa: F401  (gpu: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [2.0 ** 90, 2.0 ** 113, 2.0 ** 118, 2.0 ** 124])
@pytest.mark.parametrize("heads,dim,block", [(4, 64, 16), (1, 128, 8), (2, 128, 32)])
def test_large_queries(heads, dim, block, size):
    """Queries of any size, and a scale that brings their scores back to ordinary ones."""
    n = 300
    k, v = (rows((n, heads, dim), 1) * 2.0 ** -10).to(BF16), rows((n, heads, dim), 2).to(BF16)
    q = (rows((1, heads * 4, dim), 3) * size).to(BF16)
    check(q, k, v, block, dim ** -0.5 * 2.0 ** 10 / size, f"queries of {size:.0e}")
