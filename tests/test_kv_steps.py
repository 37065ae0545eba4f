"""Attention over the cache in lengths that give every wave many steps of 64 tokens, in batches of every
way of planning, and its calls captured together.  Tolerances as in test_kv_cache; besides, the whole
output's error: every weight is rounded once, at random by a half step at most, 2^-8 relative and of
variance 4^-8 / 3, and so is the result, sqrt(2 / 3) 2^-8 of the norm; a fifth more for the rest."""
import math

import pytest
import torch

import rht_bit_block_amd as U
from test_kv_cache import BF16, EPS, F32, POW2, Setup, make, rand, rotation, turn

GROUPS, STEP, ITEM, WAVES = 512, 64, 12, 4   # as the kernel divides its work


def most_steps(lens, new, kv, group, tile):
    """The most steps of one item (sequence, tile of rows, key head) that a workgroup takes."""
    items = [(max(1, -(-n // STEP)), -(-r * group // tile) * kv) for n, r in zip(lens, new)]
    quota = -(-sum((u + ITEM) * c for u, c in items) // GROUPS)
    if quota >= 4 * WAVES:
        quota = -(-quota // WAVES) * WAVES
    most, at = 0, 0
    for u, c in items:
        for _ in range(c):
            first = at + ITEM
            for w in range(first // quota, (first + u - 1) // quota + 1):
                most = max(most, min(first + u, (w + 1) * quota) - max(first, w * quota))
            at = first + u
    return most


LEVELS = {U.UFP4_E1M2: [0.25 * k for k in range(8)] + [-0.25 * k for k in range(8)],
          U.UFP4_INT4: list(range(8)) + list(range(-8, 0)),
          U.UFP4_E2M1: [0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6]}


def values(codes, scales, cfg):
    """What rows of codes stand for, 64 bits, in the basis of the rotation."""
    lv = torch.tensor(LEVELS[cfg.grid], dtype=torch.float64, device=codes.device)
    x = lv[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()]
    size = torch.exp2(scales.double() - 127) if cfg.scale_mode == POW2 else scales.double()
    return x * size.repeat_interleave(cfg.block_cols, -1)


def attended(s, q, scale):
    """o and its tolerance [T, heads, D] on the GPU, a sequence at a time."""
    cfg, dev = s.cfg, s.cache.k_codes.device
    R = rotation(cfg).to(dev)
    pages, kv, page, half = s.cache.k_codes.shape
    T, heads, D = q.shape
    G = heads // kv
    out, tol = (torch.zeros(T, heads, D, dtype=torch.float64, device=dev) for _ in range(2))
    x = q.to(dev).double()
    xr = turn(x, R)
    ex = 2.0 ** -16 * xr.abs() + 9 * EPS * turn(x.abs(), R.abs())
    table = s.table.to(dev).long()
    for b, (n, have) in enumerate(zip(s.new, s.lens_list)):
        if not n:
            continue
        rows = slice(int(s.starts[b]), int(s.starts[b]) + n)
        t = torch.arange(max(have, 0), device=dev)
        slot = t // page
        t = t[slot < table.shape[1]]
        t = t[(table[b, t // page] >= 0) & (table[b, t // page] < pages)]
        pg, at = table[b, t // page], t % page
        last = have - n + torch.arange(n, device=dev)
        seen = (t[None, :] <= last[:, None]).repeat_interleave(G, 0)
        # [key heads, tokens, D] and [key heads, rows of the group, D]
        K, V = (values(c[pg, :, at], z[pg, :, at], cfg).transpose(0, 1).contiguous()
                for c, z in ((s.cache.k_codes, s.cache.k_scales), (s.cache.v_codes, s.cache.v_scales)))
        Q, E = (y[rows].view(n, kv, G, D).transpose(0, 1).reshape(kv, n * G, D) for y in (xr, ex))
        Kt, Ka = K.transpose(1, 2).contiguous(), K.abs().transpose(1, 2).contiguous()
        z = scale * torch.matmul(Q, Kt)
        ez = abs(scale) * (torch.matmul(E, Ka) + (D + 16) * EPS * torch.matmul(Q.abs(), Ka)) + 3 * EPS * z.abs()
        z = z.masked_fill(~seen, -math.inf)
        p = torch.exp(z - z.amax(2, keepdim=True).clamp(min=-1e300)) if len(t) else z
        total = p.sum(2, keepdim=True)
        p = torch.where(total > 0, p / total.clamp(min=1e-300), torch.zeros_like(p))
        ep = ez + 2.0 ** -20
        ep = ep + (p * ep).sum(2, keepdim=True) + (len(t) + 64) * EPS
        e = torch.matmul(p * (BF16 + ep + (len(t) + 64) * EPS), V.abs())
        o = torch.matmul(p, V)
        val = turn(o, R.t().contiguous())
        err = turn(e, R.abs().t().contiguous()) + 12 * EPS * turn(o.abs(), R.abs().t().contiguous())
        back = lambda y: y.view(kv, n, G, D).transpose(0, 1).reshape(n, heads, D)  # noqa: E731
        out[rows], tol[rows] = back(val), back(err + BF16 * (val.abs() + err))
    return out, tol


def fill(s, seed):
    """Codes of every kind; scales that let a sequence's scores grow, shrink or neither from its
    first token to its last."""
    cache, cfg = s.cache, s.cfg
    g = torch.Generator(device=cache.k_codes.device).manual_seed(seed)
    dev = cache.k_codes.device
    for x in (cache.k_codes, cache.v_codes):
        x.copy_(torch.randint(0, 256, x.shape, generator=g, device=dev, dtype=torch.uint8))
        if cfg.grid == U.UFP4_INT4:   # -8 is no level
            x.sub_((x & 15).eq(8).to(torch.uint8)).sub_((x >> 4).eq(8).to(torch.uint8) * 16)
    size = torch.ones(cache.k_scales.shape[0], device=dev)
    for b in range(len(s.lens_list)):
        held = -(-s.lens_list[b] // s.page)
        if held > 1:
            along = torch.linspace(0.25, 1.75, held, device=dev)
            size[s.table[b, :held].long().to(dev)] = (along, along.flip(0), torch.ones_like(along))[b % 3]
    top = {U.UFP4_E1M2: 1.75, U.UFP4_INT4: 7.0, U.UFP4_E2M1: 6.0}[cfg.grid]
    for x, by in ((cache.k_scales, size), (cache.v_scales, torch.ones_like(size))):
        v = (0.5 + torch.rand(x.shape, generator=g, device=dev)) * by[:, None, None, None] * (2.0 / top)
        x.copy_((torch.log2(v).round() + 127) if cfg.scale_mode == POW2 else v)


def check(s, q, **kw):
    scale = q.shape[2] ** -0.5
    got = U.ufp4_kv_attn(q.cuda(), *s.dev(), s.cache, scale=scale, **kw)
    want, tol = attended(s, q, scale)
    off = (got.double() - want).abs()
    bad = ~(off <= tol + 1e-30)
    assert not bool(bad.any()), (int(bad.sum()), float((off / (tol + 1e-30)).max()), torch.nonzero(bad)[:3].tolist())
    assert float(off.norm()) <= 1.2 * math.sqrt(2 / 3) * BF16 * float(want.norm())
    assert torch.equal(got, U.ufp4_kv_attn(q.cuda(), *s.dev(), s.cache, scale=scale))
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("new,heads", [(1, 16), (3, 40)])
@pytest.mark.parametrize("D,page", [(128, 64), (128, 16), (64, 128), (96, 32)])
@pytest.mark.parametrize("mode,block,n", [(F32, 16, 16), (F32, 32, 1), (POW2, 32, 32)])
@pytest.mark.parametrize("grid", [U.UFP4_E1M2, U.UFP4_INT4, U.UFP4_E2M1])
def test_many_steps_of_a_wave(grid, mode, block, n, D, page, new, heads):
    """Sequences of a few hundred to 9000 tokens on eight key heads: whole items and parts of items of up to
    two dozen steps, several a wave, one and two tiles of rows, pages that do not exist among them."""
    lens = [301 + 31 * i for i in range(40)] + [5003, 7000, 9000, 6401, 8192, 5555]
    kv = 8
    assert most_steps(lens, [new] * len(lens), kv, heads // kv, 16 if new * heads // kv <= 16 else 32) >= 16
    s = Setup(lens, [new] * len(lens), kv, D, page, make(grid, mode, block, n))
    fill(s, 5)
    for b in (3, 17, 40, 43):
        s.table[b, s.table.shape[1] * lens[b] // max(lens) // 2] = -1
    check(s, rand(s.T, heads, D, 6, 2.0))


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [4, 24])
@pytest.mark.parametrize("B", [64, 65, 200, 256, 257])
def test_batches_of_every_plan(B, heads):
    """Up to 64 sequences a lane each, up to 256 a thread each, more of them block by block; empty ones first,
    last and between, one that many workgroups share."""
    lens = [(37 * i) % 400 for i in range(B)]
    new = [int(x > 0) for x in lens]
    lens[B // 2], new[B // 2] = 20000, 1
    lens[0], new[0], lens[-1], new[-1], lens[5], new[5] = 0, 0, 300, 0, 0, 0
    s = Setup(lens, new, 1, 64, 64, make(U.UFP4_E2M1, POW2, 32, 32))
    fill(s, 7)
    check(s, rand(s.T, heads, 64, 8, 2.0))


@pytest.mark.gpu
def test_captured_write():
    """The cache after a replayed step is, in every byte, the cache after the same calls made eagerly."""
    cfg, kv, heads, D, page, B = make(U.UFP4_INT4, F32, 16, 16), 2, 4, 64, 16, 3
    s = Setup([200] * B, [1] * B, kv, D, page, cfg)
    fill(s, 9)
    buffers = ("k_codes", "k_scales", "v_codes", "v_scales")
    q, k, v = (rand(B, h, D, 5).cuda() for h in (heads, kv, kv))
    starts, lens, table = s.dev()
    out = torch.zeros_like(q)
    ws = torch.empty(U.ufp4_kv_attn_workspace_bytes(B, B, heads, kv, D), dtype=torch.uint8, device="cuda")

    def step(cache, out, workspace=None):
        U.ufp4_kv_write(k, v, starts, lens, table, cache)
        return U.ufp4_kv_attn(q, starts, lens, table, cache, out=out, workspace=workspace)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(s.cache, out, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(s.cache, out, ws)
    for i, n in enumerate((1, 16, 17, 64, 130, 200)):
        for x, y in ((q, rand(B, heads, D, 50 + i)), (k, rand(B, kv, D, 60 + i)), (v, rand(B, kv, D, 70 + i))):
            x.copy_(y)
        lens.copy_(torch.tensor([n, max(1, n - 5), 201 - n]))
        twin = U.KVCache(*(getattr(s.cache, x).clone() for x in buffers), cfg)
        before = twin.k_codes.clone()
        torch.cuda.synchronize()
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        want = step(twin, torch.zeros_like(q))
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        for x in buffers:
            assert torch.equal(getattr(s.cache, x), getattr(twin, x)), x
        changed = (s.cache.k_codes != before).flatten(2).any(2).any(1).cpu()
        assert changed.nonzero().flatten().tolist() == sorted(s.slot(b, int(t) - 1)[0] for b, t in enumerate(lens.tolist()))
