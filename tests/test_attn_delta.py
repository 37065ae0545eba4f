"""Gradients of attention whose delta starts from a rounded, or another, o.

dq and dk come from ds = p (do . v - delta), and the ds of a row add to 0: whatever error delta starts
with is taken off again.  Bounds on norms: with ds0 = p (do . v - delta0) from the o that the call is
given, each ds0 and p that enters a product is rounded to bf16, a random half step at most, 2^-8
relative and of variance 4^-8 / 3, and so is the result.  So the squared error of dq is expected below
4^-8 / 3 times the sum of ds0^2 |scale k|^2, of (sum of ds0 of the row)^2 p^2 |scale k|^2 and of dq^2, and
that of dk (whose delta is the exact one) below 4^-8 / 3 times that of ds^2 |scale q|^2 and of dk^2; a
quarter more in the norm for chance and for fp32."""
import math

import pytest
import torch

import rht_bit_block_amd as U
from test_attn import BF16, packed, rand


def expected(q, k, v, do, o, lens, scale):
    """dq, dk in 64 bits, the bounds of their errors' norms, and the errors that a delta of do . o without
    the correction would leave."""
    q, k, v, do, o = (x.double() for x in (q, k, v, do, o))
    heads, G = q.shape[1], q.shape[1] // k.shape[1]
    dq, dk, plain_q, plain_k = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(q), torch.zeros_like(k)
    var = [0.0, 0.0]
    at = 0
    for n in lens:
        rows = slice(at, at + n)
        at += n
        for h in range(heads):
            Q, K, V, dO, o_in = q[rows, h], k[rows, h // G], v[rows, h // G], do[rows, h], o[rows, h]
            z = scale * (Q @ K.t())
            z[torch.ones(n, n, dtype=torch.bool).triu(1)] = -math.inf
            p = torch.softmax(z, 1)
            dp = dO @ V.t()
            ds = p * (dp - (p * dp).sum(1, keepdim=True))
            ds0 = p * (dp - (dO * o_in).sum(1, keepdim=True))
            dq[rows, h] = scale * ds @ K
            dk[rows, h // G] += scale * ds.t() @ Q
            plain_q[rows, h] = scale * ds0 @ K
            plain_k[rows, h // G] += scale * ds0.t() @ Q
            kk, qq = (scale * K).square().sum(1), (scale * Q).square().sum(1)
            var[0] += float((ds0.square() @ kk).sum() + (ds0.sum(1).square() * (p.square() @ kk)).sum())
            var[1] += float((ds.square().t() @ qq).sum())
    bound = [1.25 * BF16 / math.sqrt(3.0) * math.sqrt(v + float(x.square().sum())) for v, x in zip(var, (dq, dk))]
    return (dq, dk), bound, [float((a - b).norm()) for a, b in ((plain_q, dq), (plain_k, dk))]


@pytest.mark.gpu
@pytest.mark.parametrize("empty", [0, 600])
@pytest.mark.parametrize("factor", [1.0, 1.02, 1.25, -1.0])
@pytest.mark.parametrize("lens,heads,kv,D", [([500], 2, 1, 64), ([300, 450], 2, 2, 96), ([700], 4, 1, 128), ([130, 257, 64], 4, 2, 128)])
def test_from_a_near_delta(lens, heads, kv, D, factor, empty):
    """The forward call's own o, one that is a fiftieth off, one a quarter off, and its negative."""
    T = sum(lens)
    q, k, v, do = (rand(T, h, D, s) for s, h in ((1, heads), (2, kv), (3, kv), (4, heads)))
    starts = packed(lens + [0] * empty).cuda()
    Q, K, V, dO = (x.cuda() for x in (q, k, v, do))
    o, lse = U.ufp4_attn_fwd(Q, K, V, starts)
    o = (o.float() * factor).to(torch.bfloat16)
    want, bound, without = expected(q, k, v, do, o.cpu(), lens, D ** -0.5)
    dq, dk, _ = U.ufp4_attn_bwd(Q, K, V, starts, o, lse, dO)
    for name, x, y, b, w in zip(("dq", "dk"), (dq, dk), want, bound, without):
        off = float((x.double().cpu() - y).norm())
        assert off <= b, (name, off, b, w)
        if factor != 1.0:   # nothing that leaves the correction out can pass
            assert w > 1.5 * b, (name, w, b)
