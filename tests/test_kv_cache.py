"""The 4-bit cache: rows as they are written (bit for bit the oracle's quantization), read back,
and attended to, against the formulas in 64 bits.

Tolerances, elementwise.  Reading: a product, log2(n) sums and a product by c_n in fp32, 2^-24 of
the magnitudes each, and one rounding to bf16, 2^-8.  Attention: a rotated query carries 9 fp32
roundings of the magnitudes and is split into two bf16 pieces, half a step of half a step, 2^-16;
the second piece's own rounding is in that.  Scores: level products are exact, summed in fp32 over
D, (D + 16) 2^-24 of the magnitudes, with the scales.  Weights take 2^-20 for the exponential, and
2^-8 where they are rounded to bf16 together with a value's scale; sums over n tokens (n + 64) 2^-24.
An error of o in the rotation's basis is turned with it: it is bounded by its magnitudes through
|S H| / sqrt(n).  o is rounded once, 2^-8."""
import math

import numpy as np
import pytest
import torch

import oracle as O
import rht_bit_block_amd as U
from gpu_helpers import spec_of

BF16 = torch.finfo(torch.bfloat16).eps / 2
EPS = 2.0 ** -24
F32, POW2 = U.UFP4_SCALE_F32, U.UFP4_SCALE_POW2


def bits(x):
    return x.contiguous().view(torch.int16).numpy().view(np.uint16)


def make(grid, mode, block, n, seed=31):
    return U.make_cfg(grid, U.UFP4_RTNE, mode, 1, block, n, sign_seed=seed)


def rotation(cfg):
    """S H / sqrt(n), the signs from the oracle."""
    m = torch.ones(1, 1, dtype=torch.float64)
    while m.shape[0] < cfg.rht_n:
        m = torch.cat([torch.cat([m, m], 1), torch.cat([m, -m], 1)], 0)
    if cfg.rht_n == 1:
        return m
    s = torch.from_numpy(np.asarray(O.rht_signs(cfg.sign_seed, cfg.rht_n), dtype=np.float64).reshape(-1)[:cfg.rht_n])
    return s[:, None] * m / math.sqrt(cfg.rht_n)


def turn(x, R):
    return (x.reshape(-1, R.shape[0]) @ R).reshape(x.shape)


def rand(T, H, D, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=g) * spread
    x[torch.rand(T, H, D, generator=g) < 0.01] *= 20
    return x.to(torch.bfloat16)


class Setup:
    """A cache with scattered pages, and the packed rows of some sequences."""

    def __init__(self, lens, new, heads, D, page, cfg, seed=1, spare=2):
        g = torch.Generator().manual_seed(seed)
        self.lens_list, self.new, self.page, self.cfg = lens, new, page, cfg
        self.starts = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        held = [max(0, -(-x // page)) for x in lens]
        self.pages = sum(held) + spare
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), max(held + [1])), -1, dtype=torch.int32)
        at = 0
        for b, x in enumerate(held):
            self.table[b, :x] = order[at:at + x]
            at += x
        self.T = sum(new)
        self.cache = U.KVCache.empty(self.pages, heads, page, D, cfg)
        # what pages hold that nobody has written must not matter
        for x in (self.cache.k_codes, self.cache.v_codes):
            x.copy_(torch.randint(0, 256, x.shape, generator=g, dtype=torch.uint8))
        for x in (self.cache.k_scales, self.cache.v_scales):
            x.fill_(255 if x.dtype == torch.uint8 else math.nan)

    def dev(self):
        return self.starts.cuda(), self.lens.cuda(), self.table.cuda()

    def slot(self, b, t):
        return int(self.table[b, t // self.page]), t % self.page

    def tokens(self):
        """(packed row, sequence, token) of every packed row."""
        for b, n in enumerate(self.new):
            for i in range(n):
                yield int(self.starts[b]) + i, b, self.lens_list[b] - n + i


GRIDS = [U.UFP4_E1M2, U.UFP4_INT4, U.UFP4_E2M1]
SHAPES = [  # D, scale mode, block, n
    (128, F32, 16, 128), (128, F32, 32, 32), (128, POW2, 32, 64), (64, F32, 16, 16), (64, POW2, 32, 1), (64, F32, 32, 64),
    (96, F32, 32, 32), (96, POW2, 32, 8), (80, F32, 16, 16), (112, F32, 16, 2), (32, POW2, 32, 32), (32, F32, 32, 4), (16, F32, 16, 16),
    (48, F32, 16, 1), (128, F32, 16, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("grid", GRIDS)
@pytest.mark.parametrize("D,mode,block,n", SHAPES)
def test_write_and_read(D, mode, block, n, grid):
    cfg = make(grid, mode, block, n)
    heads = 3
    s = Setup([37, 0, 5, 100], [20, 0, 5, 1], heads, D, 16, cfg)
    k, v = rand(s.T, heads, D, 2), rand(s.T, heads, D, 3)
    old = [x.clone() for x in (s.cache.k_codes, s.cache.v_codes)]
    place = s.dev()
    U.ufp4_kv_write(k.cuda(), v.cuda(), *place, s.cache)
    got = U.ufp4_kv_read(s.cache, *place, s.T)
    torch.cuda.synchronize()
    R = rotation(cfg)
    for x, codes, scales, before, back in ((k, s.cache.k_codes, s.cache.k_scales, old[0], got[0]),
                                           (v, s.cache.v_codes, s.cache.v_scales, old[1], got[1])):
        ref = O.quantize(bits(x.reshape(-1, D)), 0, spec_of(cfg))
        want = torch.from_numpy(ref["codes"]).view(s.T, heads, D // 2)
        size = torch.from_numpy(np.ascontiguousarray(ref["scales"])).view(s.T, heads, D // block)
        codes, scales = codes.cpu(), scales.cpu()
        touched = torch.zeros(codes.shape[0], codes.shape[2], dtype=torch.bool)
        for row, b, t in s.tokens():
            page, at = s.slot(b, t)
            touched[page, at] = True
            assert torch.equal(codes[page, :, at], want[row]) and torch.equal(scales[page, :, at], size[row])
        left = ~touched[:, None, :, None].expand_as(codes)
        assert torch.equal(codes[left], before.cpu()[left])
        val = torch.from_numpy(np.asarray(O.dequant(ref["codes"], ref["scales"], spec_of(cfg), s.T * heads, D)[1], dtype=np.float64))
        x64 = turn(val, R.t()).view(s.T, heads, D)
        mag = turn(val.abs(), R.abs().t()).view(s.T, heads, D)
        tol = BF16 * x64.abs() + 12 * EPS * mag
        assert bool(((back.double().cpu() - x64).abs() <= tol).all())


@pytest.mark.gpu
def test_read_whole_sequences_and_missing_places():
    """Whole sequences through other starts; tokens before the first, past the table and in pages that do
    not exist read as zeros and are not written; rows of no sequence keep what they hold."""
    cfg, heads, D, page = make(U.UFP4_INT4, F32, 32, 32), 2, 64, 16
    s = Setup([40, 33], [40, 33], heads, D, page, cfg)
    k, v = rand(s.T, heads, D, 4), rand(s.T, heads, D, 5)
    place = s.dev()
    U.ufp4_kv_write(k.cuda(), v.cuda(), *place, s.cache)
    a = U.ufp4_kv_read(s.cache, *place, s.T)
    # the last 7 tokens of the first, 33 + 3 rows of the second (three before its first token), two rows of none
    starts = torch.tensor([1, 8, 44], dtype=torch.int32).cuda()
    out = tuple(torch.full((46, heads, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    U.ufp4_kv_read(s.cache, starts, place[1], place[2], 46, out=out)
    for x, y in zip(a, out):
        assert torch.equal(y[1:8], x[33:40]) and torch.equal(y[11:44], x[40:73])
        assert bool((y[8:11] == 0).all()) and bool((y[:1] == 9).all()) and bool((y[44:] == 9).all())
    # pages that do not exist
    codes = s.cache.k_codes.clone()
    table = place[2].clone()
    table[0, 1], table[1, 0] = s.pages, -5
    U.ufp4_kv_write(k.cuda() * 3, v.cuda() * 3, place[0], place[1], table, s.cache)
    b = U.ufp4_kv_read(s.cache, place[0], place[1], table, s.T)
    assert bool((b[0][16:32] == 0).all()) and bool((b[1][40:56] == 0).all()) and bool((b[0][:16] != 0).any())
    for p, slot in ((0, 1), (1, 0)):
        assert torch.equal(s.cache.k_codes[s.table[p, slot]], codes[s.table[p, slot]])
    # a table that is too narrow
    c = U.ufp4_kv_read(s.cache, place[0], place[1], place[2][:, :2], s.T)
    assert bool((c[0][32:40] == 0).all()) and bool((c[1][72:] == 0).all()) and bool((c[0][:32] != 0).any())


def attended(s, q, scale):
    """o and its tolerance [T, heads, D], from the codes and scales that the cache holds."""
    cfg, R = s.cfg, rotation(s.cfg)
    pages, kv, page, half = s.cache.k_codes.shape
    D, heads = 2 * half, q.shape[1]
    G = heads // kv
    val = []
    for c, z in ((s.cache.k_codes, s.cache.k_scales), (s.cache.v_codes, s.cache.v_scales)):
        c = c.cpu()
        if cfg.grid == U.UFP4_INT4:   # rows that nobody has written may hold -8, which is no level
            c = torch.where((c & 15) == 8, c & 0xF0, c)
            c = torch.where((c >> 4) == 8, c & 0x0F, c)
        _, x = O.dequant(c.numpy().reshape(-1, half), z.cpu().numpy().reshape(-1, D // cfg.block_cols), spec_of(cfg), pages * kv * page, D)
        val.append(torch.from_numpy(np.asarray(x, dtype=np.float64)).view(pages, kv, page, D))
    out, tol = torch.zeros(s.T, heads, D, dtype=torch.float64), torch.zeros(s.T, heads, D, dtype=torch.float64)
    for row, b, t in s.tokens():
        seen = [(int(s.table[b, j // page]), j % page) for j in range(t + 1)
                if j // page < s.table.shape[1] and 0 <= int(s.table[b, j // page]) < pages]
        if not seen:
            continue
        pg, at = (torch.tensor(x) for x in zip(*seen))
        n = len(seen)
        for h in range(heads):
            K, V = val[0][pg, h // G, at], val[1][pg, h // G, at]
            x = q[row, h].double()
            xr = turn(x, R)
            ex = 2.0 ** -16 * xr.abs() + 9 * EPS * turn(x.abs(), R.abs())
            z = scale * (K @ xr)
            ez = abs(scale) * (K.abs() @ ex + (D + 16) * EPS * (K.abs() @ xr.abs())) + 3 * EPS * z.abs()
            p = torch.softmax(z, 0)
            ep = ez + 2.0 ** -20
            ep = ep + (p * ep).sum() + (n + 64) * EPS
            e = (p * (BF16 + ep + (n + 64) * EPS)) @ V.abs()
            o = p @ V
            out[row, h] = turn(o, R.t())
            err = turn(e, R.abs().t()) + 12 * EPS * turn(o.abs(), R.abs().t())
            tol[row, h] = err + BF16 * (out[row, h].abs() + err)
    return out, tol


def filled(s, seed=11, spread=1.0):
    """All tokens of all sequences written, through their own starts."""
    pages, kv, page, half = s.cache.k_codes.shape
    starts = torch.tensor([0] + list(np.cumsum(s.lens_list)), dtype=torch.int32)
    k, v = rand(sum(s.lens_list), kv, 2 * half, seed, spread), rand(sum(s.lens_list), kv, 2 * half, seed + 1)
    U.ufp4_kv_write(k.cuda(), v.cuda(), starts.cuda(), s.lens.cuda(), s.table.cuda(), s.cache)
    return k, v


def check(s, q, scale=None, **kw):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    got = U.ufp4_kv_attn(q.cuda(), *s.dev(), s.cache, scale=scale, **kw)
    torch.cuda.synchronize()
    want, tol = attended(s, q, scale)
    off = (got.double().cpu() - want).abs()
    bad = ~(off <= tol + 1e-30)
    assert not bad.any(), (int(bad.sum()), float((off / (tol + 1e-30)).max()), torch.nonzero(bad)[:3].tolist())
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("grid", GRIDS)
@pytest.mark.parametrize("D,mode,block,n", SHAPES)
def test_attention_over_the_cache(D, mode, block, n, grid):
    s = Setup([1, 64, 65, 200], [1, 1, 1, 1], 2, D, 16, make(grid, mode, block, n))
    filled(s)
    check(s, rand(s.T, 8, D, 21))


@pytest.mark.gpu
@pytest.mark.parametrize("mode,block,n", [(F32, 16, 16), (F32, 32, 32), (POW2, 32, 32)])
@pytest.mark.parametrize("grid", GRIDS)
def test_several_rows_of_a_sequence(mode, block, n, grid):
    """Rows that see different tokens, tiles of 16 and of 32 rows, the last of them short."""
    for D, kv, heads, lens, new in ((128, 2, 10, [70, 300, 9], [5, 3, 9]), (64, 1, 1, [40, 130], [33, 1]), (64, 1, 4, [100], [1]),
                                    (128, 1, 16, [129], [2])):
        s = Setup(lens, new, kv, D, 32, make(grid, mode, block, n))
        filled(s)
        check(s, rand(s.T, heads, D, 22))


@pytest.mark.gpu
@pytest.mark.parametrize("new,heads", [(1, 10), (5, 10), (2, 40)])
@pytest.mark.parametrize("mode,block,n", [(F32, 16, 64), (F32, 32, 1), (POW2, 32, 32)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("grid", GRIDS)
def test_pages_of_whole_steps(grid, D, mode, block, n, new, heads):
    """Pages of 64 tokens and more, whose steps are copied as one run: lengths around the steps' and pages'
    ends, a page that does not exist, one and two tiles of rows."""
    s = Setup([new, 64, 129, 500], [new] * 4, 2, D, 128 if new == 5 else 64, make(grid, mode, block, n))
    filled(s)
    s.table[3, 1] = s.pages
    check(s, rand(s.T, heads, D, 41))


@pytest.mark.gpu
def test_more_sequences_than_are_kept_at_hand():
    lens = [1 + (7 * i) % 40 for i in range(1100)]
    cfg = make(U.UFP4_E2M1, POW2, 32, 32)
    s = Setup(lens, [1] * 1100, 1, 32, 16, cfg)
    k, _ = filled(s)
    first = [0] + list(np.cumsum(lens))
    starts = torch.tensor(first, dtype=torch.int32).cuda()
    all_rows = U.ufp4_kv_read(s.cache, starts, s.lens.cuda(), s.table.cuda(), sum(lens))
    ref = O.quantize(bits(k.view(-1, 32)), 0, spec_of(cfg))
    want = torch.from_numpy(ref["codes"]).view(-1, 1, 16)
    codes = s.cache.k_codes.cpu()
    for b in (0, 1, 63, 64, 500, 1023, 1024, 1025, 1099):   # each by itself
        n = lens[b]
        one = U.ufp4_kv_read(s.cache, torch.tensor([0, n], dtype=torch.int32).cuda(), s.lens[b:b + 1].cuda(),
                             s.table[b:b + 1].cuda(), n)
        for x, y in zip(one, all_rows):
            assert torch.equal(x, y[first[b]:first[b] + n])
        for t in range(n):
            page, at = s.slot(b, t)
            assert torch.equal(codes[page, :, at], want[first[b] + t])
    check(s, rand(s.T, 2, 32, 42))


@pytest.mark.gpu
@pytest.mark.parametrize("kv,lens", [(1, [5000]), (2, [1, 3000, 7, 64 * 17]), (8, [650, 2])])
def test_split_and_joined(kv, lens):
    """Long sequences cut among many workgroups, short ones beside them."""
    s = Setup(lens, [1] * len(lens), kv, 64, 64, make(U.UFP4_E2M1, POW2, 32, 32))
    filled(s, spread=3.0)
    a = check(s, rand(s.T, 2 * kv, 64, 23))
    assert torch.equal(a, U.ufp4_kv_attn(rand(s.T, 2 * kv, 64, 23).cuda(), *s.dev(), s.cache))


@pytest.mark.gpu
def test_many_sequences():
    """More sequences than a workgroup has threads."""
    lens = [(11 * i) % 70 for i in range(300)]
    s = Setup(lens, [int(x > 0) for x in lens], 1, 64, 16, make(U.UFP4_INT4, F32, 32, 32))
    filled(s)
    check(s, rand(s.T, 4, 64, 24))


@pytest.mark.gpu
@pytest.mark.parametrize("page", [1, 2, 64, 256])
def test_pages_of_any_size(page):
    s = Setup([3, 130, 75], [1, 2, 1], 2, 64, page, make(U.UFP4_E1M2, F32, 16, 16))
    filled(s)
    check(s, rand(s.T, 4, 64, 25))


@pytest.mark.gpu
@pytest.mark.parametrize("page,pages", [(64, 140000), (16, 560000)])
def test_pages_past_32_bits(page, pages):
    """Pages of a cache whose codes are more than 2^32 bytes hold what those of a small one do."""
    cfg, kv, heads, D, n = make(U.UFP4_E2M1, F32, 32, 32), 8, 8, 128, 150
    assert pages * kv * page * (D // 2) > 1 << 32
    starts, lens = torch.tensor([0, n], dtype=torch.int32).cuda(), torch.tensor([n], dtype=torch.int32).cuda()
    k, v, q = (rand(n, h, D, 80 + i).cuda() for i, h in enumerate((kv, kv, heads)))
    slots = -(-n // page)
    places = torch.arange(slots, dtype=torch.int32)
    got = []
    for cache, table in ((U.KVCache.empty(pages, kv, page, D, cfg), pages - 1 - 37 * places),
                         (U.KVCache.empty(slots, kv, page, D, cfg), places)):
        table = table[None].cuda()
        U.ufp4_kv_write(k, v, starts, lens, table, cache)
        got.append((*U.ufp4_kv_read(cache, starts, lens, table, n), U.ufp4_kv_attn(q, starts, lens, table, cache)))
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_two_streams_at_once():
    """Calls on two streams over one cache, each with a workspace of its own."""
    cfg, heads = make(U.UFP4_INT4, F32, 16, 64), 10
    s = Setup([3000, 700, 65], [1, 1, 1], 2, 128, 64, cfg)
    filled(s)
    place = s.dev()
    qs = [rand(s.T, heads, 128, 90 + i).cuda() for i in range(2)]
    want = [U.ufp4_kv_attn(q, *place, s.cache) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(3):
        got = []
        for st, q in zip(streams, qs):
            with torch.cuda.stream(st):
                got.append(U.ufp4_kv_attn(q, *place, s.cache))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.gpu
def test_rows_that_see_nothing():
    """No tokens, tokens without places, pages that do not exist in the middle of a sequence; rows behind
    the last sequence keep what they hold."""
    cfg = make(U.UFP4_INT4, F32, 32, 32)
    s = Setup([100, 0, 20, 90], [1, 2, 1, 3], 2, 64, 16, cfg)
    filled(s)
    s.table[0, 2] = -1          # tokens 32 .. 47
    s.table[2, :] = s.pages + 7  # all of them
    s.table[3, 0] = -2147483648
    q = rand(s.T, 4, 64, 26)
    got = check(s, q)
    assert bool((got[1:4] == 0).all())
    out = torch.full((s.T + 3, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    more = torch.cat([q, q[:3]]).cuda()
    U.ufp4_kv_attn(more, *s.dev(), s.cache, out=out)
    assert torch.equal(out[:s.T], got) and bool((out[s.T:] == 5).all())
    # a cache without pages
    none = U.KVCache.empty(0, 2, 16, 64, cfg)
    assert bool((U.ufp4_kv_attn(q.cuda(), *s.dev(), none) == 0).all())
    k = rand(s.T, 2, 64, 27).cuda()
    U.ufp4_kv_write(k, k, *s.dev(), none)
    assert bool((U.ufp4_kv_read(none, *s.dev(), s.T)[0] == 0).all())


@pytest.mark.gpu
def test_infinite_scales_of_tokens_not_seen():
    """A later token's scale that is infinite or NaN does not reach earlier rows."""
    s = Setup([80], [3], 1, 64, 16, make(U.UFP4_INT4, F32, 32, 32))
    filled(s)
    q = rand(3, 4, 64, 28)
    want = check(s, q)
    for t, bad in ((79, math.nan), (78, math.inf)):
        page, at = s.slot(0, t)
        s.cache.k_scales[page, 0, at] = bad
        s.cache.v_scales[page, 0, at] = bad
    got = U.ufp4_kv_attn(q.cuda(), *s.dev(), s.cache)
    assert torch.equal(got[0], want[0]) and not bool(torch.isfinite(got[2]).any())


@pytest.mark.gpu
def test_prompt_then_tokens():
    """The calls as a generation makes them: the prompt's attention on exact keys, its keys written, then token
    after token written and attended to; and the whole again over the cache at once."""
    cfg, kv, heads, D, page = make(U.UFP4_E2M1, POW2, 32, 32), 2, 8, 64, 16
    prompt, steps = [30, 1, 17], 4
    s = Setup([n + steps for n in prompt], [n + steps for n in prompt], kv, D, page, cfg)
    q, k, v = (rand(s.T, h, D, x).cuda() for h, x in ((heads, 31), (kv, 32), (kv, 33)))
    starts, _, table = s.dev()
    first = [int(x) for x in s.starts[:-1]]
    pick = lambda n0, n1: torch.cat([torch.arange(f + a, f + b) for f, a, b in zip(first, n0, n1)]).cuda()  # noqa: E731
    at = pick([0] * 3, prompt)
    st = torch.tensor([0] + list(np.cumsum(prompt)), dtype=torch.int32).cuda()
    o, _ = U.ufp4_attn_fwd(q[at], k[at], v[at], st, lse=False)
    U.ufp4_kv_write(k[at], v[at], st, torch.tensor(prompt, dtype=torch.int32).cuda(), table, s.cache)
    rows = []
    one = torch.arange(4, dtype=torch.int32).cuda()
    for i in range(steps):
        at = pick([n + i for n in prompt], [n + i + 1 for n in prompt])
        lens = torch.tensor([n + i + 1 for n in prompt], dtype=torch.int32).cuda()
        U.ufp4_kv_write(k[at], v[at], one, lens, table, s.cache)
        rows.append((at, U.ufp4_kv_attn(q[at], one, lens, table, s.cache)))
    want, tol = attended(s, q.cpu(), D ** -0.5)
    for at, x in rows:
        a = at.cpu()
        assert bool(((x.double().cpu() - want[a]).abs() <= tol[a]).all())
    check(s, q.cpu())
    # the prompt's own attention on the keys and values that the cache stands for
    K, V = U.ufp4_kv_read(s.cache, starts, s.lens.cuda(), table, s.T)
    o2, _ = U.ufp4_attn_fwd(q, K, V, starts)
    got = U.ufp4_kv_attn(q, starts, s.lens.cuda(), table, s.cache)
    assert float((o2.double() - got.double()).norm() / got.double().norm()) < 4 * BF16


@pytest.mark.gpu
def test_captured_step():
    """A decoding step in a graph, replayed as the sequences grow, eager work between the replays."""
    cfg, kv, heads, D, page, B = make(U.UFP4_INT4, F32, 16, 16), 2, 4, 64, 16, 3
    s = Setup([200] * B, [1] * B, kv, D, page, cfg)
    filled(s)
    q, k = (rand(B, h, D, 5).cuda() for h in (heads, kv))
    starts, lens, table = s.dev()
    lens.fill_(1)
    out = torch.zeros_like(q)
    ws = torch.empty(U.ufp4_kv_attn_workspace_bytes(B, B, heads, kv, D), dtype=torch.uint8, device="cuda")

    def step():
        U.ufp4_kv_write(k, k, starts, lens, table, s.cache)
        U.ufp4_kv_attn(q, starts, lens, table, s.cache, out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, n in enumerate((1, 16, 17, 64, 130, 200)):
        q.copy_(rand(B, heads, D, 50 + i))
        k.copy_(rand(B, kv, D, 60 + i))
        lens.copy_(torch.tensor([n, max(1, n - 5), 200 - n]))
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, U.ufp4_kv_attn(q, starts, lens, table, s.cache))
        torch.cuda.synchronize()


def test_binding_refuses():
    cfg = make(U.UFP4_INT4, F32, 32, 32)
    c = U.KVCache.empty(4, 2, 16, 64, cfg, device="cpu")
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    st, ln, tb = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 5, dtype=torch.int32)
    w = lambda **a: U.ufp4_kv_write(**{**dict(k=k, v=k, starts=st, lens=ln, table=tb, cache=c), **a})  # noqa: E731
    r = lambda **a: U.ufp4_kv_read(**{**dict(cache=c, starts=st, lens=ln, table=tb, T=3), **a})  # noqa: E731
    t = lambda **a: U.ufp4_kv_attn(**{**dict(q=q, starts=st, lens=ln, table=tb, cache=c), **a})  # noqa: E731
    for f in (w, r, t):
        with pytest.raises(ValueError, match="GPU"):
            f()
        with pytest.raises(ValueError, match="starts"):
            f(starts=st.long())
        with pytest.raises(ValueError, match="lens"):
            f(lens=ln[:1])
        with pytest.raises(ValueError, match="table has 3 rows"):
            f(table=torch.zeros(3, 5, dtype=torch.int32))
        with pytest.raises(ValueError, match="table must have dtype"):
            f(table=tb.long())
        with pytest.raises(ValueError, match="v_scales must be"):
            f(cache=U.KVCache(c.k_codes, c.k_scales, c.v_codes, c.v_scales.double(), cfg))
        with pytest.raises(ValueError, match="v_codes must be"):
            f(cache=U.KVCache(c.k_codes, c.k_scales, c.v_codes[:3], c.v_scales, cfg))
        with pytest.raises(ValueError, match="whole blocks"):
            f(cache=U.KVCache(c.k_codes[..., :24].contiguous(), c.k_scales, c.v_codes, c.v_scales, cfg))
        with pytest.raises(ValueError, match="k_codes must be contiguous"):
            f(cache=U.KVCache(c.k_codes.transpose(0, 0)[:, :, ::1].transpose(1, 2).contiguous().transpose(1, 2), c.k_scales, c.v_codes, c.v_scales, cfg))
    with pytest.raises(ValueError, match="k has shape"):
        w(k=k[:, :1])
    with pytest.raises(ValueError, match="v has shape"):
        w(v=k[:2])
    with pytest.raises(ValueError, match="k has shape"):
        r(out=(k[:2], k))
    with pytest.raises(ValueError, match="heads of"):
        t(q=torch.zeros(3, 3, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="heads of"):
        t(q=torch.zeros(3, 4, 32, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="out has shape"):
        t(out=q[:2])


def test_library_refuses():
    """Every check of the three calls, before any HIP call (pointers are numbers that nobody follows)."""
    import ctypes
    L = U.lib_handle()
    A = 1 << 20
    cfg = make(U.UFP4_INT4, F32, 32, 32)
    base = dict(k_codes=A, k_scales=A, v_codes=A, v_scales=A, pages=4, page_tokens=16, kv_heads=2, D=64, cfg=cfg)

    def cache(**kw):
        return U.KVCacheC(*{**base, **kw}.values())

    size = U.ufp4_kv_attn_workspace_bytes(3, 2, 4, 2, 64)
    good = dict(c=cache(), starts=A, B=2, T=3, lens=A, table=A, ldt=5, width=5, x=A, ldx=256, y=A, ldy=256, heads=4, scale=1.0, ws=A, size=size)

    def calls(**kw):
        a = {**good, **kw}
        c = ctypes.byref(a["c"]) if a["c"] is not None else None
        return (L.ufp4_kv_write(a["x"], a["ldx"], a["y"], a["ldy"], a["starts"], a["B"], a["T"], a["lens"], a["table"], a["ldt"], a["width"], c, None),
                L.ufp4_kv_read(c, a["starts"], a["B"], a["T"], a["lens"], a["table"], a["ldt"], a["width"], a["x"], a["ldx"], a["y"], a["ldy"], None),
                L.ufp4_kv_attn(a["x"], a["ldx"], a["starts"], a["B"], a["T"], a["heads"], a["lens"], a["table"], a["ldt"], a["width"], c, a["scale"],
                               a["y"], a["ldy"], a["ws"], a["size"], None))

    for kw, st in [(dict(c=None), -1), (dict(T=-1), -1), (dict(B=-1), -1), (dict(width=-1), -1), (dict(starts=None), -1), (dict(lens=None), -1),
                   (dict(table=None), -1), (dict(table=A + 2), -1), (dict(ldt=4), -1), (dict(x=None), -1), (dict(y=A + 8), -1), (dict(ldx=120), -1),
                   (dict(ldy=132 + 256), -1), (dict(T=(1 << 30) + 1), -4), (dict(B=(1 << 20) + 1), -4), (dict(width=(1 << 22) + 1, ldt=1 << 23), -4),
                   (dict(c=cache(page_tokens=24)), -1), (dict(c=cache(page_tokens=0)), -1), (dict(c=cache(pages=-1)), -1),
                   (dict(c=cache(kv_heads=0)), -1), (dict(c=cache(D=48)), -2), (dict(c=cache(D=160), ldx=1024, ldy=1024), -4),
                   (dict(c=cache(k_codes=None)), -1), (dict(c=cache(v_scales=A + 4)), -1), (dict(c=cache(v_codes=A + 8)), -1),
                   (dict(c=cache(cfg=make(U.UFP4_E4M3, POW2, 32, 32))), -4), (dict(c=cache(cfg=cfg.copy(rounding=U.UFP4_SR))), -4),
                   (dict(c=cache(cfg=make(U.UFP4_E2M1, POW2, 32, 32).copy(tensor_scale=2.0))), -4), (dict(c=cache(cfg=cfg.copy(rht_n=24))), -2),
                   (dict(c=cache(cfg=U.make_cfg(U.UFP4_E2M1, U.UFP4_RTNE, POW2, 32, 32, 1))), -4), (dict(c=cache(cfg=cfg.copy(grid=9))), -1)]:
        assert calls(**kw) == (st,) * 3, kw
    for kw in (dict(heads=3), dict(heads=0), dict(scale=math.nan), dict(ws=None), dict(ws=A + 16), dict(size=size - 1), dict(heads=8)):
        assert calls(**kw)[2] == U.UFP4_ERR_INVALID_ARG, kw
    assert calls(T=0, x=None) == (0, 0, 0) and calls(B=0, y=None, starts=None) == (0, 0, 0)
    assert U.ufp4_kv_attn_workspace_bytes(0, 2, 4, 2, 64) == 0 and U.ufp4_kv_attn_workspace_bytes(3, 2, 4, 3, 64) == 0
