"""The least E8M0 scale, byte 0, is 2^-127 wherever a cache is read: attention over it sees what
ufp4_kv_read gives back."""
import numpy as np
import pytest
import torch

import oracle as O
import rht_bit_block_amd as U
from gpu_helpers import spec_of
from test_kv_cache import GRIDS, POW2, Setup, attended, make


@pytest.mark.gpu
@pytest.mark.parametrize("new,heads", [(1, 2), (3, 16)])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("grid", GRIDS)
def test_byte_0(grid, D, page, new, heads):
    """Values of k and v down to 2^-129, keys that meet queries of 2^126: z = 2^-1 level each.  A weight
    times 2^-127 is rounded to a multiple of 2^-133 at the least; the largest weight is 1 or more, so n tokens
    of levels up to `top` add top n 2^-134 to the other tolerances, and the result's own rounding 2^-134."""
    cfg, g = make(grid, POW2, 32, 1), torch.Generator().manual_seed(3)
    lens, kv = [9, 5], 2
    s = Setup(lens, [new] * 2, kv, D, page, cfg)
    for x in (s.cache.k_codes, s.cache.v_codes):
        code = torch.randint(0, 256, x.shape, generator=g, dtype=torch.uint8)
        if grid == U.UFP4_INT4:   # -8 is no level
            code = torch.where((code & 15) == 8, code & 0xF0, code)
            code = torch.where((code >> 4) == 8, code & 0x0F, code)
        x.copy_(code)
    s.cache.k_scales.fill_(0)
    s.cache.v_scales.fill_(0)
    q = torch.zeros(s.T, heads, D, dtype=torch.bfloat16)
    q[..., 3], q[..., 40] = 2.0 ** 126, -(2.0 ** 126)
    got = U.ufp4_kv_attn(q.cuda(), *s.dev(), s.cache, scale=1.0).double().cpu()
    want, tol = attended(s, q, 1.0)
    top = {U.UFP4_E1M2: 1.75, U.UFP4_INT4: 7.0, U.UFP4_E2M1: 6.0}[grid]
    tol = tol + (top * max(lens) + 1) * 2.0 ** -134
    assert bool((want.abs() > 4 * tol).any())
    assert bool(((got - want).abs() <= tol).all())
    # the same values by the other call, exactly
    starts = torch.tensor([0, 9, 14], dtype=torch.int32).cuda()
    for x, codes in zip(U.ufp4_kv_read(s.cache, starts, *s.dev()[1:], 14), (s.cache.k_codes, s.cache.v_codes)):
        val = O.dequant(codes.cpu().numpy().reshape(-1, D // 2), np.zeros((codes[..., 0].numel(), D // 32), dtype=np.uint8), spec_of(cfg),
                        codes[..., 0].numel(), D)[1]
        val = torch.from_numpy(np.asarray(val, dtype=np.float64)).view(*codes.shape[:3], D)
        where = [s.slot(b, t) for b, n in enumerate(lens) for t in range(n)]
        assert torch.equal(x.double().cpu(), torch.stack([val[p, :, at] for p, at in where]))
