"""Causal attention with factors of the scores that are 0 or next to it, and products near the end of
fp32's range.  Tolerances as in test_attn."""
import pytest
import torch

import rht_bit_block_amd as U
from test_attn import formulas, near, packed, rand


@pytest.mark.gpu
@pytest.mark.parametrize("empty", [0, 600])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -107, -(2.0 ** -107), 2.0 ** -126, 1e-42])
def test_large_products(scale, empty):
    """Products of up to 2^107 and more: a factor of 0 leaves every score 0, one of 2^-107 gives scores of
    ordinary size, smaller ones scores next to 0."""
    lens, heads, kv, D = [150, 70], 4, 2, 64
    T, up = sum(lens), 2.0 ** 52
    q, k = (rand(T, h, D, s) * up for h, s in ((heads, 1), (kv, 2)))
    v, do = rand(T, kv, D, 3), rand(T, heads, D, 4)
    scale = float(torch.tensor(scale, dtype=torch.float32))
    want = formulas(q, k, v, lens, scale, do)
    starts = packed(lens + [0] * empty).cuda()
    Q, K, V, dO = (x.cuda() for x in (q, k, v, do))
    o, lse = U.ufp4_attn_fwd(Q, K, V, starts, scale=scale)
    near("o", o, want["o"])
    near("lse", lse, want["lse"])
    for name, x in zip(("dq", "dk", "dv"), U.ufp4_attn_bwd(Q, K, V, starts, o, lse, dO, scale=scale)):
        near(name, x, want[name])
