"""Many keys whose weights are far below a few dominant ones': the products with
V are taken in fp16 over fp16 and e4m3 caches, and must not lose them."""
import math

import pytest
import torch

from tests._cache_model import TYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_softmax_gb300 as m
    m.build()
    return m


@pytest.mark.parametrize("dtype,cache", [("fp16", "fp16"), ("fp16", "e4m3"), ("bf16", "e4m3"), ("bf16", "bf16")])
@pytest.mark.parametrize("gamma,B", [(0, 320), (16, 80)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("high,low", [(18.0, 0.0), (22.0, -1.375), (26.0, -0.5)])
def test_a_long_rest_below_dominant_keys(sv, dtype, cache, gamma, B, dim, high, low):
    """Scores to base 2 of `high` at a few keys and of `low` at all others.  The
    dominant keys (one in each 16 of the first 256) have values of zero, so the
    output is the rest's alone.  All requests share one cache: enough units for
    each to be long in its block."""
    page, heads, H, keys, few = 64, 8, 2, 32768, 16
    n = keys - gamma - 1
    dt, ct = TYPES[dtype], TYPES[cache]
    k, v = torch.zeros(keys, H, dim), torch.zeros(keys, H, dim)
    k[:, :, 0] = low
    c = torch.tensor([256.0, 320.0, -384.0, 448.0]).repeat(dim // 4)
    v[:] = c
    k[:16 * few:16, :, 0], v[:16 * few:16] = high, 0.0
    K, V = (x.view(keys // page, page, H, dim).cuda().to(ct) for x in (k, v))
    assert torch.equal(K.float().cpu().view(k.shape), k) and torch.equal(V.float().cpu().view(v.shape), v)
    q = torch.zeros(B, gamma + 1, heads, dim, dtype=dt, device="cuda")
    q[..., 0] = 1.0
    table = torch.arange(keys // page, dtype=torch.int32, device="cuda").repeat(B, 1)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    lse = torch.zeros(q.shape[:-1], device="cuda")
    scale = math.log(2.0)
    out, ws = sv.attend(q, K, V, table, lens, scale=scale, out_lse=lse)
    assert sv.read_status(ws) == 0
    eps = torch.finfo(dt).eps
    weight = torch.finfo(torch.float16).eps if cache == "e4m3" else eps
    for j in range(gamma + 1):
        rest = (n + j + 1 - few) * 2.0 ** (low - high)   # weights relative to a dominant key's
        share = rest / (few + rest)
        # the output's rounding; each weight's; twice the score's fp32 error (D
        # products and sums); exp2 and a sum of n terms in fp32
        off = (dim + 8) * 2.0 ** -24 * high
        r = eps / 2 * 1.01 + weight / 2 + 2 * off + 2.0 ** -20 + (n + 64) * 2.0 ** -24
        if weight == torch.finfo(torch.float16).eps:
            # half the least fp16 step of each weight, dominant keys' being 2^11 or more
            r += 2.0 ** (-25 - 11) / 2.0 ** (low - high)
        want = c.double() * share
        d = (out[:, j].double().cpu() - want).abs() / want.abs()
        assert (d <= r).all(), (j, float(d.max()), r)
        want = math.log(few * 2.0 ** high + (n + j + 1 - few) * 2.0 ** low)
        assert ((lse[:, j].double().cpu() - want).abs() <= 2e-5 * (1 + want)).all()
