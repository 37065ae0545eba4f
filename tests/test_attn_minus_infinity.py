"""Causal attention where a tile of keys gives a row nothing but scores of -inf: keys with -inf, or
with the type's lowest value, in a channel that the queries hold.  Such a key has weight 0, and what
the row's other keys say stands.  Tolerances as in test_attn."""
import math

import pytest
import torch

import rht_bit_block_amd as U
from test_attn import EPS, formulas, near, packed, rand

LOWEST = torch.finfo(torch.bfloat16).min   # times 8 past fp32's range, as each product is


def inputs(n, heads, kv, D, hidden, bad, seed):
    q, k, v, do = rand(n, heads, D, seed), rand(n, kv, D, seed + 1), rand(n, kv, D, seed + 2), rand(n, heads, D, seed + 3)
    q[..., 5] = 8.0
    k[..., 5] = 0.0
    far = k.double()
    far[hidden, :, 5] = -1e30   # a weight of exactly 0 in 64 bits
    open_k = k.clone()
    k[hidden, :, 5] = bad
    return q, k, v, do, far, open_k


# empty sequences make many workgroups of it; without, two sets of waves share a tile's keys
@pytest.mark.gpu
@pytest.mark.parametrize("empty", [0, 600])
@pytest.mark.parametrize("bad", [-math.inf, LOWEST])
@pytest.mark.parametrize("first", [1, 64, 128, 200])
def test_first_keys(first, bad, empty):
    """The first keys of a sequence: rows behind them are the rest's own attention, rows among them have
    no finite score, o = NaN and lse = -inf."""
    n, heads, kv, D = 330, 4, 2, 64
    q, k, v, _, _, _ = inputs(n, heads, kv, D, slice(0, first), bad, 5)
    want = formulas(q[first:], k[first:], v[first:], [n - first], D ** -0.5)
    o, lse = U.ufp4_attn_fwd(q.cuda(), k.cuda(), v.cuda(), packed([n] + [0] * empty).cuda())
    near("o", o[first:], want["o"])
    near("lse", lse[first:], want["lse"])
    assert bool(torch.isnan(o[:first]).all()) and bool((lse[:first] == -math.inf).all())
