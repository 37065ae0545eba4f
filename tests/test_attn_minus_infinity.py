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


@pytest.mark.gpu
@pytest.mark.parametrize("empty", [0, 600])
@pytest.mark.parametrize("bad", [-math.inf, LOWEST])
@pytest.mark.parametrize("a,b", [(1, 64), (64, 128), (1, 128), (32, 96), (64, 300)])
@pytest.mark.parametrize("D", [64, 128])
def test_keys_among_others(D, a, b, bad, empty):
    """Keys in the middle, forward and backward: whole tiles, halves of tiles, the second set of waves'
    first tile.  Their gradients are 0; dq's channel that meets -inf is 0 times it, and not looked at."""
    n, heads, kv, scale = 330, 4, 2, D ** -0.5
    q, k, v, do, far, open_k = inputs(n, heads, kv, D, slice(a, b), bad, 15)
    want = formulas(q, far, v, [n], scale, do)
    # errors of the scores that count; those of the keys that do not are as large as they are
    slack = formulas(q, open_k, v, [n], scale)["lse"][1]
    starts = packed([n] + [0] * empty).cuda()
    Q, K, V, dO = (x.cuda() for x in (q, k, v, do))
    o, lse = U.ufp4_attn_fwd(Q, K, V, starts)
    near("o", o, want["o"])
    near("lse", lse, (want["lse"][0], slack + 4 * EPS * want["lse"][0].abs()))
    dq, dk, dv = U.ufp4_attn_bwd(Q, K, V, starts, o, lse, dO)
    keep = [d for d in range(D) if d != 5]
    near("dq", dq[..., keep], tuple(x[..., keep] for x in want["dq"]))
    near("dk", dk, want["dk"])
    near("dv", dv, want["dv"])
    assert not bool(dk[a:b].any()) and not bool(dv[a:b].any())


@pytest.mark.gpu
@pytest.mark.parametrize("empty", [0, 600])
@pytest.mark.parametrize("first", [1, 64, 200])
def test_rows_without_a_score_have_no_gradient_of_others(first, empty):
    """Rows whose every key is hidden (filling before a sequence), gradients of 0 for them: keys and values
    behind them have the rest's own gradients, those among them 0."""
    n, heads, kv, D = 330, 4, 2, 64
    q, k, v, do, _, _ = inputs(n, heads, kv, D, slice(0, first), -math.inf, 25)
    do[:first] = 0
    want = formulas(q[first:], k[first:], v[first:], [n - first], D ** -0.5, do[first:])
    starts = packed([n] + [0] * empty).cuda()
    Q, K, V, dO = (x.cuda() for x in (q, k, v, do))
    o, lse = U.ufp4_attn_fwd(Q, K, V, starts)
    dq, dk, dv = U.ufp4_attn_bwd(Q, K, V, starts, o, lse, dO)
    keep = [d for d in range(D) if d != 5]
    near("dq", dq[first:][..., keep], tuple(x[..., keep] for x in want["dq"]))
    near("dk", dk[first:], want["dk"])
    near("dv", dv[first:], want["dv"])
    assert not bool(dk[:first].any()) and not bool(dv[:first].any())
