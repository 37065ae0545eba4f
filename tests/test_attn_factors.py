"""Causal attention with factors of the scores that are 0 or next to it, and products near the end of
fp32's range.  Tolerances as in test_attn."""
import ctypes

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


def test_largest_factors():
    """A factor of the scores is taken up to fp32's largest divided by log2(e), which the kernels multiply
    it by, and refused above, before any HIP call (pointers are numbers that nobody follows)."""
    L, A = U.lib_handle(), 1 << 20
    cfg = U.make_cfg(U.UFP4_INT4, U.UFP4_RTNE, U.UFP4_SCALE_F32, 1, 32, 32)
    cache = ctypes.byref(U.KVCacheC(A, A, A, A, 4, 16, 2, 64, cfg))
    for scale in (2.4e38, -2.4e38, 3.4e38):
        got = (L.ufp4_attn_fwd(A, 256, A, 128, A, 128, A, 2, 10, 4, 2, 64, scale, A, 256, A, None),
               L.ufp4_attn_bwd(A, 256, A, 128, A, 128, A, 2, 10, 4, 2, 64, scale, A, 256, A, A, 256, A, 256, A, 128, A, 128, A,
                               U.ufp4_attn_workspace_bytes(10, 4), None),
               L.ufp4_kv_attn(A, 256, A, 2, 3, 4, A, A, 5, 5, cache, scale, A, 256, A, U.ufp4_kv_attn_workspace_bytes(3, 2, 4, 2, 64), None))
        assert got == (U.UFP4_ERR_INVALID_ARG,) * 3, scale


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [2.3e38, -2.3e38])
def test_largest_factor_of_products_of_0(scale):
    """Keys of 0 score 0, whatever the factor is."""
    n, heads, kv, D = 70, 4, 2, 64
    q, k, v = rand(n, heads, D, 1), torch.zeros(n, kv, D, dtype=torch.bfloat16), rand(n, kv, D, 3)
    want = formulas(q, k, v, [n], scale)
    o, lse = U.ufp4_attn_fwd(q.cuda(), k.cuda(), v.cuda(), packed([n]).cuda(), scale=scale)
    near("o", o, want["o"])
    near("lse", lse, want["lse"])
