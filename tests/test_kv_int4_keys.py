"""Attention over a cache of INT4 keys: the error of a score goes by |K| |q'|, so a channel of q that
is loud where the keys' codes are 0 changes nothing.  Tolerances as in test_kv_cache."""
import pytest
import torch

import rht_bit_block_amd as U
from test_kv_cache import F32, Setup, check, filled, make, rand


@pytest.mark.gpu
@pytest.mark.parametrize("new,heads", [(1, 4), (5, 10)])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("D,block", [(64, 16), (64, 32), (128, 16), (128, 32), (80, 16)])
def test_loud_channel_over_zero_codes(D, block, page, new, heads):
    cfg, g = make(U.UFP4_INT4, F32, block, 1), torch.Generator().manual_seed(7)
    s = Setup([70, 130], [new] * 2, 2, D, page, cfg)
    filled(s)
    code = torch.randint(-2, 3, (*s.cache.k_codes.shape[:3], D), generator=g)
    loud = 37
    code[..., loud] = 0
    code = code.to(torch.uint8) & 15
    s.cache.k_codes.copy_(code[..., 0::2] | (code[..., 1::2] << 4))
    s.cache.k_scales.fill_(16.0)
    q = (rand(s.T, heads, D, 8).float() * 0.02).to(torch.bfloat16)
    q[..., loud] = 300.0
    check(s, q, scale=1.0)
