"""Scores so large that fp32 has steps of more than one: the weights of the keys
that share the largest score stay finite in fp16, and all others are zero.

An fp32 score s (base 2) is off by half a step, 2^-24 s, and by as much again where
the same product is rounded on another way (before or within the subtraction of the
maximum).  So two keys of one score may weigh 2^(2^-22 s) times one another, and the
output lies between their values whatever s is."""
import math
import random

import pytest
import torch

from tests._cache_model import TYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_softmax_gb300 as m
    m.build()
    return m


@pytest.mark.parametrize("dtype,cache", [("fp16", "fp16"), ("fp16", "e4m3"), ("bf16", "e4m3"), ("bf16", "bf16"),
                                         ("fp32", "fp32")])
@pytest.mark.parametrize("gamma", [0, 16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("sign", [1, -1])
def test_huge_scores(sv, dtype, cache, gamma, dim, sign):
    """Eight keys with the same largest score of 2^20 to 2^100 (base 2) among 600
    of half and a quarter of it (or of a quarter of the others' size, all negative): their values' mean, as far as fp32 holds
    the scores, and always between those values."""
    page, heads, H, keys = 16, 8, 2, 608
    n = keys - gamma - 1
    r = random.Random(dim + gamma)
    g = torch.Generator().manual_seed(dim)
    dt, ct = TYPES[dtype], TYPES[cache]
    top = torch.randperm(n, generator=g)[:8]           # seen by all rows
    level = torch.tensor([0.5 if t % 2 else 0.25 for t in range(keys)])
    level[top] = 1.0
    if sign < 0:
        level = 0.25 / level                           # 0.25 at the keys, 0.5 and 1 at the others
    v = torch.randn(keys, H, dim, generator=g).to(ct)
    value = v.double()[top]                            # [8, H, dim]
    mean, size = value.mean(0), value.abs().mean(0)
    least, most = value.amin(0), value.amax(0)
    eps, weight = torch.finfo(dt).eps, torch.finfo(torch.float16).eps if cache == "e4m3" else torch.finfo(dt).eps
    # the output's rounding, the weights', exp2 and sums in fp32
    tol = eps / 2 * 1.01 * mean.abs() + (weight / 2 + 2.0 ** -18) * size
    table = torch.arange(keys // page, dtype=torch.int32, device="cuda").view(1, -1)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    V = v.view(keys // page, page, H, dim).cuda()
    for i in range(120):
        bits = 20 + i % 30 if i < 90 else r.uniform(50, 100)
        k0 = float(torch.tensor(r.uniform(1, 2)).to(ct))
        q0 = float(torch.tensor(r.uniform(1, 2)).to(dt))
        k = torch.zeros(keys, H, dim)
        k[:, :, 0] = k0 * level[:, None]
        K = k.to(ct).view(keys // page, page, H, dim).cuda()
        q = torch.zeros(1, gamma + 1, heads, dim, dtype=dt, device="cuda")
        q[..., 0] = q0
        scale = math.log(2.0) * r.uniform(1, 2) * 2.0 ** bits / (k0 * q0)
        q *= sign
        lse = torch.zeros(q.shape[:-1], device="cuda")
        out, ws = sv.attend(q, K, V, table, lens, scale=scale, out_lse=lse)
        assert sv.read_status(ws) == 0
        got = out.double().cpu()[0].view(gamma + 1, H, heads // H, dim)
        uneven = 2.0 ** min(2.0 ** -22 * scale * q0 * k0 / math.log(2.0), 30.0) - 1.0
        off = torch.minimum(tol + uneven * size, tol + (most - least))[:, None]
        d = (got - mean[:, None]).abs()
        assert (d <= off).all(), (i, bits, float(d.max()))     # NaN fails too
        assert (got >= (least - tol)[:, None]).all() and (got <= (most + tol)[:, None]).all(), (i, bits)
        want = scale * q0 * k0 * (1.0 if sign > 0 else -0.25)
        assert ((lse.double().cpu() - want).abs() <= 2.0 ** -21 * abs(want) + 3).all(), (i, bits)
