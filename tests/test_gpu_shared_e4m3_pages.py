"""Shared-prefix attention over e4m3 caches whose pages are no multiple of 8
tokens: the warp-level kernels of heads up to 128."""
import pytest

from tests._share_model import SharedCase
from tests.test_gpu_shared import _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_softmax_gb300 as m
    m.build()
    return m


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [48, 64, 112, 128])
@pytest.mark.parametrize("page", [1, 5, 100])
@pytest.mark.parametrize("gamma,packed", [(0, False), (9, True)])
def test_e4m3_pages(sv, dtype, dim, page, gamma, packed):
    """16 rows a KV head at most, and more."""
    pages = max(1, 230 // page)
    n = pages * page
    _run(sv, SharedCase(share=[([0, 2, 3], pages)], lens=[n, 99, n + 128, n + 1], ell=[gamma, gamma // 2, gamma, gamma],
                        gamma=gamma, page=page, heads=8, kv_heads=2, dim=dim, dtype=dtype, cache="e4m3", packed=packed,
                        seed=page + dim))
