"""Causal attention over packed sequences and its gradients, against the formulas in 64
bits.

Tolerances, elementwise.  Scores: products of bf16 are exact in fp32, summed over D, (D +
16) 2^-24 of the sum of magnitudes, and two roundings of the result; an error of z is a
relative error of p, to which the hardware exponential adds 2^-20.  p is rounded to bf16,
2^-8 relative, as is ds.  Sums over n terms: (n + 16) 2^-24 of their magnitudes.  delta
carries o's rounding.  Every output is rounded once, 2^-8 (bf16) or 2^-24 (fp32)."""
import math

import pytest
import torch

import rht_bit_block_amd as U

BF16 = torch.finfo(torch.bfloat16).eps / 2
EPS = 2.0 ** -24


def formulas(q, k, v, lens, scale, do=None):
    """{name: (value, tolerance)} in 64 bits; q, k, v, do [T, heads, D]."""
    q, k, v = (x.double() for x in (q, k, v))
    T, H, D = q.shape
    G = H // k.shape[1]
    names = ["o", "lse"] + (["dq", "dk", "dv"] if do is not None else [])
    shape = dict(o=q, lse=q[..., 0], dq=q, dk=k, dv=v)
    out = {x: (torch.zeros_like(shape[x]), torch.zeros_like(shape[x])) for x in names}

    def put(name, rows, h, value, err, add=False):
        a, b = out[name]
        a[rows, h] = a[rows, h] + value if add else value
        b[rows, h] = b[rows, h] + err if add else err

    at = 0
    for n in lens:
        rows = slice(at, at + n)
        at += n
        for h in range(H if n else 0):
            Q, K, V = q[rows, h], k[rows, h // G], v[rows, h // G]
            z = scale * (Q @ K.t())
            ez = abs(scale) * (D + 16) * EPS * (Q.abs() @ K.abs().t()) + 3 * EPS * z.abs()
            hide = torch.ones(n, n, dtype=torch.bool).triu(1)
            z[hide] = -math.inf
            lse = torch.logsumexp(z, 1)
            p = torch.exp(z - lse[:, None])
            ep = ez.masked_fill(hide, 0) + 2.0 ** -20
            ep = ep + (p * ep).sum(1, keepdim=True) + (n + 16) * EPS   # and of the whole
            o = p @ V
            eo = (p * (BF16 + ep + (n + 16) * EPS)) @ V.abs()
            put("o", rows, h, o, eo + BF16 * (o.abs() + eo))
            put("lse", rows, h, lse, ez.masked_fill(hide, 0).amax(1) + (n + 16) * EPS + 2.0 ** -20 + 4 * EPS * lse.abs())
            if do is None:
                continue
            dO = do[rows, h].double()
            dv = p.t() @ dO
            edv = (p * (BF16 + ep + (n + 16) * EPS)).t() @ dO.abs()
            dp = dO @ V.t()
            edp = (D + 16) * EPS * (dO.abs() @ V.abs().t())
            delta = (dO * o).sum(1, keepdim=True)
            edelta = (dO.abs() * (eo + BF16 * o.abs())).sum(1, keepdim=True) + (D + 16) * EPS * (dO * o).abs().sum(1, keepdim=True)
            ds = p * (dp - delta)
            eds = p * (edp + edelta + ep * (dp - delta).abs()) + 2 * EPS * p * (dp.abs() + delta.abs())
            eds = eds + BF16 * (ds.abs() + eds) + (n + 16) * EPS * ds.abs()
            dq = scale * (ds @ K)
            edq = abs(scale) * (eds @ K.abs())
            put("dq", rows, h, dq, edq + BF16 * (dq.abs() + edq))
            put("dk", rows, h // G, scale * (ds.t() @ Q), abs(scale) * (eds.t() @ Q.abs()), add=True)
            put("dv", rows, h // G, dv, edv, add=True)
    for x in ("dk", "dv"):
        if x in out:
            a, b = out[x]
            out[x] = a, b + BF16 * (a.abs() + b)
    return out


def packed(lens, before=0):
    s = [before]
    for n in lens:
        s.append(s[-1] + n)
    return torch.tensor(s, dtype=torch.int32)


def rand(T, H, D, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, H, D, generator=g) * spread).to(torch.bfloat16)


def near(name, got, want):
    value, tol = want
    got = got.double().cpu()
    assert got.shape == value.shape
    off = (got - value).abs()
    bad = ~(off <= tol + 1e-30)
    assert not bad.any(), (name, int(bad.sum()), float((off / (tol + 1e-30)).max()),
                           torch.nonzero(bad)[:3].tolist())


CASES = [
    # lens, heads, key heads, D
    ([1], 1, 1, 128), ([2], 2, 1, 64), ([19], 4, 2, 128), ([64], 2, 2, 128), ([65], 1, 1, 64),
    ([127, 1, 0, 130], 4, 1, 128), ([0, 0, 33], 2, 2, 64), ([300], 3, 3, 80), ([129, 257], 6, 2, 8),
    ([257], 2, 1, 72), ([31, 32, 33, 63, 64, 65], 5, 5, 104), ([500], 2, 1, 120),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,heads,kv,D", CASES)
def test_forward_and_backward(lens, heads, kv, D):
    T = sum(lens)
    q, k, v = rand(T, heads, D, 1), rand(T, kv, D, 2), rand(T, kv, D, 3)
    do = rand(T, heads, D, 4, 1e-2)
    scale = D ** -0.5
    want = formulas(q, k, v, lens, scale, do)
    starts = packed(lens).cuda()
    Q, K, V, dO = (x.cuda() for x in (q, k, v, do))
    o, lse = U.ufp4_attn_fwd(Q, K, V, starts)
    near("o", o, want["o"])
    near("lse", lse, want["lse"])
    for name, x in zip(("dq", "dk", "dv"), U.ufp4_attn_bwd(Q, K, V, starts, o, lse, dO)):
        near(name, x, want[name])


@pytest.mark.gpu
@pytest.mark.parametrize("empty", [0, 600])
@pytest.mark.parametrize("lens,heads,kv,D", [([200, 70], 2, 1, 32), ([129, 257], 2, 2, 64), ([300, 1], 3, 1, 96), ([31, 450], 4, 2, 128)])
def test_few_and_many_workgroups(lens, heads, kv, D, empty):
    """Launches of few workgroups, whose tiles two sets of waves share, and (empty sequences
    count) of many; a group's heads of odd and even number of steps."""
    T = sum(lens)
    q, k, v, do = rand(T, heads, D, 51), rand(T, kv, D, 52), rand(T, kv, D, 53), rand(T, heads, D, 54)
    want = formulas(q, k, v, lens, 0.2, do)
    starts = packed(lens + [0] * empty).cuda()
    Q, K, V, dO = (x.cuda() for x in (q, k, v, do))
    o, lse = U.ufp4_attn_fwd(Q, K, V, starts, scale=0.2)
    near("o", o, want["o"])
    near("lse", lse, want["lse"])
    got = U.ufp4_attn_bwd(Q, K, V, starts, o, lse, dO, scale=0.2)
    for name, x in zip(("dq", "dk", "dv"), got):
        near(name, x, want[name])
    again = U.ufp4_attn_bwd(Q, K, V, starts, o, lse, dO, scale=0.2)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.gpu
@pytest.mark.parametrize("scale,spread", [(-0.3, 1.0), (0.0, 1.0), (1.0, 3.0), (0.02, 30.0)])
def test_scales(scale, spread):
    """Factors of any sign, rows that one key wins."""
    lens, heads, kv, D = [150, 70], 4, 2, 64
    q, k, v, do = rand(220, heads, D, 5, spread), rand(220, kv, D, 6, spread), rand(220, kv, D, 7), rand(220, heads, D, 8)
    want = formulas(q, k, v, lens, scale, do)
    starts = packed(lens).cuda()
    Q, K, V, dO = (x.cuda() for x in (q, k, v, do))
    o, lse = U.ufp4_attn_fwd(Q, K, V, starts, scale=scale)
    near("o", o, want["o"])
    near("lse", lse, want["lse"])
    for name, x in zip(("dq", "dk", "dv"), U.ufp4_attn_bwd(Q, K, V, starts, o, lse, dO, scale=scale)):
        near(name, x, want[name])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_one_matrix_strides_and_rows_of_no_sequence(D):
    """q, k and v as slices of one product, gradients into slices of one matrix, rows before the
    first and behind the last sequence, which keep what they hold."""
    lens, heads, kv = [70, 5, 129], 4, 2
    T, before = sum(lens) + 11, 4
    W = (heads + 2 * kv) * D
    qkv = rand(T, 1, W, 9).view(T, W)
    qkv[:before], qkv[before + sum(lens):] = math.nan, math.nan
    cut = lambda m: (m[:, :heads * D].unflatten(1, (heads, D)),  # noqa: E731
                     m[:, heads * D:(heads + kv) * D].unflatten(1, (kv, D)),
                     m[:, (heads + kv) * D:].unflatten(1, (kv, D)))
    live = slice(before, before + sum(lens))
    q, k, v = cut(qkv[live])
    do = rand(sum(lens), heads, D, 10)
    want = formulas(q, k, v, lens, D ** -0.5, do)
    starts = packed(lens, before).cuda()
    dev = qkv.cuda()
    Q, K, V = cut(dev)
    out = torch.full((T, heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, heads), 7.0, device="cuda")
    U.ufp4_attn_fwd(Q, K, V, starts, out=out, lse=lse)
    dO = torch.full((T, heads, D), math.nan, dtype=torch.bfloat16, device="cuda")
    dO[live] = do.cuda()
    grads = torch.full((T, W), 7.0, dtype=torch.bfloat16, device="cuda")
    got = U.ufp4_attn_bwd(Q, K, V, starts, out, lse, dO, out=cut(grads))
    near("o", out[live], want["o"])
    near("lse", lse[live], want["lse"])
    for name, x in zip(("dq", "dk", "dv"), got):
        near(name, x[live], want[name])
    for x in (out, lse, grads):
        assert bool((x[:before] == 7).all()) and bool((x[before + sum(lens):] == 7).all())


@pytest.mark.gpu
def test_other_sequences_never_matter():
    """NaN and infinities of one sequence stay there; repeated calls give the same bits, with and
    without lse."""
    lens, heads, kv, D = [100, 64, 90], 4, 2, 128
    T = sum(lens)
    starts = packed(lens).cuda()
    Q, K, V, dO = (rand(T, h, D, s).cuda() for h, s in ((heads, 1), (kv, 2), (kv, 3), (heads, 4)))
    o, lse = U.ufp4_attn_fwd(Q, K, V, starts)
    g = U.ufp4_attn_bwd(Q, K, V, starts, o, lse, dO)
    o2, none = U.ufp4_attn_fwd(Q, K, V, starts, lse=False)
    assert none is None and torch.equal(o, o2)
    mid = slice(100, 164)
    for x, bad in ((Q, math.inf), (K, math.nan), (V, math.inf), (dO, math.nan)):
        x[mid] = bad
    o3, lse3 = U.ufp4_attn_fwd(Q, K, V, starts)
    g3 = U.ufp4_attn_bwd(Q, K, V, starts, o3, lse3, dO)
    keep = torch.ones(T, dtype=torch.bool)
    keep[mid] = False
    for a, b in zip((o, lse, *g), (o3, lse3, *g3)):
        assert torch.equal(a[keep.cuda()], b[keep.cuda()])


@pytest.mark.gpu
def test_later_tokens_never_matter():
    """Scores of later tokens are not looked at, however large: finite values past a token leave
    its output as it is, bit for bit."""
    n, heads, kv, D = 200, 2, 1, 64
    starts = packed([n]).cuda()
    Q, K, V = (rand(n, h, D, s).cuda() for h, s in ((heads, 1), (kv, 2), (kv, 3)))
    o, lse = U.ufp4_attn_fwd(Q, K, V, starts)
    for at in (1, 77, 128, 150):
        K2, V2 = K.clone(), V.clone()
        K2[at:] = 1e4
        V2[at:] = -1e30
        o2, lse2 = U.ufp4_attn_fwd(Q, K2, V2, starts)
        assert torch.equal(o[:at], o2[:at]) and torch.equal(lse[:at], lse2[:at])


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv,D", [(1, 1, 64), (6, 2, 128), (3, 3, 80), (2, 1, 24)])
def test_a_single_key_has_no_gradient_of_scores(heads, kv, D):
    """Sequences of one token: o = v and ds = 0, exactly."""
    T = 37
    starts = packed([1] * T).cuda()
    Q, K, V, dO = (rand(T, h, D, s).cuda() for h, s in ((heads, 1), (kv, 2), (kv, 3), (heads, 4)))
    o, lse = U.ufp4_attn_fwd(Q, K, V, starts)
    assert torch.equal(o, V.repeat_interleave(heads // kv, 1))
    dq, dk, dv = U.ufp4_attn_bwd(Q, K, V, starts, o, lse, dO)
    assert not bool(dq.any()) and not bool(dk.any()) and bool(dv.any())


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[9000, 130, 17000, 1, 0, 8300], [20011], [64 * 128, 64 * 128 + 1, 128, 127], [40 * 128] * 64, [300] * 70 + [9000, 2]])
def test_every_tile_is_found(lens):
    """Keys of zeros and values of ones, so that row i has lse = log(i + 1) and o = 1, and with a
    gradient of ones dv[j] = sum over i >= j of 1 / (i + 1): p rounded to bf16, 2^-8 relative, with the
    exponential's 2^-20, a sum of n terms, and the result's own rounding."""
    T = sum(lens)
    starts = packed(lens).cuda()
    K, V = torch.zeros(T, 1, 8, dtype=torch.bfloat16, device="cuda"), torch.ones(T, 1, 8, dtype=torch.bfloat16, device="cuda")
    o, lse = U.ufp4_attn_fwd(rand(T, 1, 8, 31).cuda(), K, V, starts, out=torch.full_like(V, 7.0), lse=torch.full((T, 1), 7.0, device="cuda"))
    dq, dk, dv = U.ufp4_attn_bwd(K, K, V, starts, o, lse, V, out=tuple(torch.full_like(V, 7.0) for _ in range(3)))
    i = torch.cat([torch.arange(n, dtype=torch.float64) for n in lens])
    top = max(lens)
    assert bool((o.cpu() == 1).all())
    near("lse", lse[:, 0], (torch.log(i + 1), (top + 16) * EPS + 2.0 ** -20 + 4 * EPS * torch.log(i + 1)))
    want = torch.cat([torch.flip(torch.cumsum(torch.flip(1 / torch.arange(1, n + 1, dtype=torch.float64), (0,)), 0), (0,)) for n in lens])
    for d in (0, 7):
        near("dv", dv[:, 0, d], (want, want * (2 * BF16 + 2.0 ** -16 + 2 * (top + 16) * EPS)))
    assert bool((dq == 0).all())   # sums of keys that are 0
    # q is 0 in the backward call
    assert bool((dk == 0).all())


@pytest.mark.gpu
def test_many_sequences_and_one_long():
    """More sequences than a wave has lanes, and a sequence of several dozen tiles."""
    lens = [(7 * i) % 23 for i in range(150)]
    heads, kv, D = 2, 1, 64
    T = sum(lens)
    q, k, v, do = rand(T, heads, D, 1), rand(T, kv, D, 2), rand(T, kv, D, 3), rand(T, heads, D, 4)
    want = formulas(q, k, v, lens, D ** -0.5, do)
    starts = packed(lens).cuda()
    Q, K, V, dO = (x.cuda() for x in (q, k, v, do))
    o, lse = U.ufp4_attn_fwd(Q, K, V, starts)
    near("o", o, want["o"])
    for name, x in zip(("dq", "dk", "dv"), U.ufp4_attn_bwd(Q, K, V, starts, o, lse, dO)):
        near(name, x, want[name])
    lens = [2500]
    q, k, v, do = rand(2500, 1, 128, 1), rand(2500, 1, 128, 2), rand(2500, 1, 128, 3), rand(2500, 1, 128, 4)
    want = formulas(q, k, v, lens, 128 ** -0.5, do)
    starts = packed(lens).cuda()
    Q, K, V, dO = (x.cuda() for x in (q, k, v, do))
    o, lse = U.ufp4_attn_fwd(Q, K, V, starts)
    near("o", o, want["o"])
    near("lse", lse, want["lse"])
    for name, x in zip(("dq", "dk", "dv"), U.ufp4_attn_bwd(Q, K, V, starts, o, lse, dO)):
        near(name, x, want[name])


@pytest.mark.gpu
def test_rows_past_32_bits():
    """The last rows of tensors of more than 2^32 elements."""
    T, W, heads, kv, D, n = 530000, 8192, 4, 2, 64, 200
    assert (T - n) * W > 1 << 32
    big, grads = (torch.empty(T, W, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cut = lambda m: (m[:, :256].unflatten(1, (4, 64)), m[:, 256:384].unflatten(1, (2, 64)),  # noqa: E731
                     m[:, 8064:].unflatten(1, (2, 64)), m[:, 512:768].unflatten(1, (4, 64)), m[:, 1024:1280].unflatten(1, (4, 64)))
    q, k, v, do = rand(n, heads, D, 61), rand(n, kv, D, 62), rand(n, kv, D, 63), rand(n, heads, D, 64)
    Q, K, V, dO, out = cut(big)
    for x, y in ((Q, q), (K, k), (V, v), (dO, do)):
        x[T - n:] = y.cuda()
    starts = packed([n], T - n).cuda()
    o, lse = U.ufp4_attn_fwd(Q, K, V, starts, out=out)
    got = U.ufp4_attn_bwd(Q, K, V, starts, o, lse, dO, out=cut(grads)[:3])
    want = formulas(q, k, v, [n], D ** -0.5, do)
    for name, x in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *got)):
        near(name, x[T - n:], want[name])


@pytest.mark.gpu
def test_two_streams_at_once():
    """Calls on two streams, each with memory of its own, give what they give one after another."""
    lens, heads, kv, D = [700, 800], 8, 2, 128
    T = sum(lens)
    starts = packed(lens).cuda()
    sets = [[rand(T, h, D, 70 + 4 * i + j).cuda() for j, h in enumerate((heads, kv, kv, heads))] for i in range(2)]

    def run(Q, K, V, dO):
        o, lse = U.ufp4_attn_fwd(Q, K, V, starts)
        return (o, lse, *U.ufp4_attn_bwd(Q, K, V, starts, o, lse, dO))

    want = [run(*x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = []
        for s, x in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(run(*x))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
def test_nothing_to_do():
    z = lambda t, h: torch.zeros(t, h, 64, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    o, lse = U.ufp4_attn_fwd(z(0, 2), z(0, 1), z(0, 1), packed([0]).cuda())
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2)
    for x in U.ufp4_attn_bwd(z(0, 2), z(0, 1), z(0, 1), packed([0]).cuda(), o, lse, z(0, 2)):
        assert x.shape[0] == 0
    out = torch.full((5, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    U.ufp4_attn_fwd(z(5, 2), z(5, 1), z(5, 1), packed([0, 0]).cuda(), out=out)
    U.ufp4_attn_fwd(z(5, 2), z(5, 1), z(5, 1), packed([]).cuda(), out=out)
    assert bool((out == 3).all())


@pytest.mark.gpu
def test_captured_with_eager_work_between():
    """Forward and backward in a graph, replayed with other inputs and other lengths, eager calls
    and synchronizations between the replays, and on a stream of their own."""
    heads, kv, D, T = 4, 2, 64, 192
    new = lambda s: [rand(T, h, D, s + i).cuda() for i, h in enumerate((heads, kv, kv, heads))]  # noqa: E731
    Q, K, V, dO = new(1)
    starts = packed([100, 92]).cuda()
    out, lse = torch.zeros_like(Q), torch.zeros(T, heads, device="cuda")
    grads = tuple(torch.zeros_like(x) for x in (Q, K, V))
    ws = torch.empty(U.ufp4_attn_workspace_bytes(T, heads), dtype=torch.uint8, device="cuda")

    def step():
        U.ufp4_attn_fwd(Q, K, V, starts, out=out, lse=lse)
        U.ufp4_attn_bwd(Q, K, V, starts, out, lse, dO, out=grads, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, lens in enumerate(([100, 92], [1, 191], [192, 0], [64, 128])):
        for x, y in zip((Q, K, V, dO), new(10 * i)):
            x.copy_(y)
        starts.copy_(packed(lens))
        graph.replay()
        got = [x.clone() for x in (out, lse, *grads)]
        torch.cuda.synchronize()
        o, l2 = U.ufp4_attn_fwd(Q, K, V, starts)
        want = (o, l2, *U.ufp4_attn_bwd(Q, K, V, starts, o, l2, dO))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_formulas_against_differences():
    """The reference's gradients against central differences of its own forward pass."""
    lens, heads, kv, D, scale = [5, 9], 4, 2, 8, 0.7
    T = sum(lens)
    q, k, v, do = (rand(T, h, D, s).double() for h, s in ((heads, 1), (kv, 2), (kv, 3), (heads, 4)))
    want = formulas(q, k, v, lens, scale, do)
    value = lambda q, k, v: float((formulas(q, k, v, lens, scale)["o"][0] * do).sum())  # noqa: E731
    for name, i in (("dq", 0), ("dk", 1), ("dv", 2)):
        x = [q, k, v]
        for seed in range(3):
            d = rand(*x[i].shape, 20 + seed).double()
            e = 1e-5
            up, down = list(x), list(x)
            up[i], down[i] = x[i] + e * d, x[i] - e * d
            slope = (value(*up) - value(*down)) / (2 * e)
            assert abs(slope - float((want[name][0] * d).sum())) < 1e-6 * (1 + abs(slope))


@pytest.mark.gpu
def test_gradients_against_differences():
    """The kernel's gradients along random directions against central differences of the formulas'
    forward pass: within the elementwise tolerances summed along the direction."""
    lens, heads, kv, D = [40, 25], 4, 2, 64
    T, scale = sum(lens), D ** -0.5
    q, k, v, do = (rand(T, h, D, s) for h, s in ((heads, 1), (kv, 2), (kv, 3), (heads, 4)))
    want = formulas(q, k, v, lens, scale, do)
    starts = packed(lens).cuda()
    Q, K, V, dO = (x.cuda() for x in (q, k, v, do))
    o, lse = U.ufp4_attn_fwd(Q, K, V, starts)
    got = U.ufp4_attn_bwd(Q, K, V, starts, o, lse, dO)
    x = [q.double(), k.double(), v.double()]
    value = lambda x: float((formulas(*x, lens, scale)["o"][0] * do.double()).sum())  # noqa: E731
    for i, name in enumerate(("dq", "dk", "dv")):
        d = rand(*x[i].shape, 30 + i).double()
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + 1e-4 * d, x[i] - 1e-4 * d
        slope = (value(up) - value(down)) / 2e-4
        mine = float((got[i].double().cpu() * d).sum())
        assert abs(mine - slope) <= float((want[name][1] * d.abs()).sum()) + 1e-6


def test_binding_refuses():
    q, k = torch.zeros(4, 4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    s = torch.zeros(2, dtype=torch.int32)
    f = U.ufp4_attn_fwd
    with pytest.raises(ValueError, match="3-D bfloat16"):
        f(q.float(), k, k, s)
    with pytest.raises(ValueError, match="3-D bfloat16"):
        f(q[0], k, k, s)
    with pytest.raises(ValueError, match="v has shape"):
        f(q, k, k[:3], s)
    with pytest.raises(ValueError, match="share"):
        f(q, torch.zeros(4, 3, 64, dtype=torch.bfloat16), torch.zeros(4, 3, 64, dtype=torch.bfloat16), s)
    with pytest.raises(ValueError, match="one after another"):
        f(q.transpose(1, 2).contiguous().transpose(1, 2), k, k, s)
    with pytest.raises(ValueError, match="starts"):
        f(q, k, k, s.long())
    with pytest.raises(ValueError, match="starts"):
        f(q, k, k, torch.zeros(0, dtype=torch.int32))
    with pytest.raises(ValueError, match="out has shape"):
        f(q, k, k, s, out=q[:, :2])
    with pytest.raises(ValueError, match="lse holds"):
        f(q, k, k, s, lse=torch.zeros(4, 3))
    with pytest.raises(ValueError, match="GPU"):
        f(q, k, k, s)
    b = lambda **kw: U.ufp4_attn_bwd(**{**dict(q=q, k=k, v=k, starts=s, o=q, lse=torch.zeros(4, 4), dout=q), **kw})  # noqa: E731
    with pytest.raises(ValueError, match="lse must have dtype"):
        b(lse=torch.zeros(4, 4, dtype=torch.float64))
    with pytest.raises(ValueError, match="dout has shape"):
        b(dout=q[:3])
    with pytest.raises(ValueError, match="dk has shape"):
        b(out=(q, q, k))
    with pytest.raises(ValueError, match="GPU"):
        b()


def test_library_refuses():
    """Every check of the two calls, before any HIP call (pointers are numbers that nobody follows)."""
    L = U.lib_handle()
    A = 1 << 20
    good = dict(q=A, ldq=256, k=A, ldk=128, v=A, ldv=128, starts=A, B=2, T=10, heads=4, kv=2, D=64, scale=1.0, o=A, ldo=256)

    def fwd(**kw):
        a = {**good, "lse": A, **kw}
        return L.ufp4_attn_fwd(a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["starts"], a["B"], a["T"], a["heads"], a["kv"],
                               a["D"], a["scale"], a["o"], a["ldo"], a["lse"], None)

    def bwd(**kw):
        a = {**good, "lse": A, "do": A, "lddo": 256, "dq": A, "lddq": 256, "dk": A, "lddk": 128, "dv": A, "lddv": 128, "ws": A,
             "size": U.ufp4_attn_workspace_bytes(10, 4), **kw}
        return L.ufp4_attn_bwd(a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["starts"], a["B"], a["T"], a["heads"], a["kv"],
                               a["D"], a["scale"], a["o"], a["ldo"], a["lse"], a["do"], a["lddo"], a["dq"], a["lddq"], a["dk"], a["lddk"],
                               a["dv"], a["lddv"], a["ws"], a["size"], None)

    both = [(dict(T=-1), -1), (dict(B=-1), -1), (dict(heads=0), -1), (dict(kv=3), -1), (dict(kv=0), -1), (dict(D=0), -1), (dict(D=60), -2),
            (dict(D=136, ldq=1024, ldk=512, ldv=512, ldo=1024), -4), (dict(T=(1 << 30) + 1), -4), (dict(B=(1 << 20) + 1), -4),
            (dict(heads=2048, kv=2), -4), (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(o=None), -1), (dict(starts=None), -1),
            (dict(q=A + 8), -1), (dict(starts=A + 2), -1), (dict(ldq=248), -1), (dict(ldk=132), -1), (dict(ldv=120), -1), (dict(ldo=252), -1),
            (dict(ldk=(1 << 22) + 8), -4), (dict(scale=math.nan), -1), (dict(scale=math.inf), -1), (dict(lse=A + 1), -1)]
    for kw, st in both:
        assert fwd(**kw) == st, kw
        assert bwd(**kw) == st, kw
    for kw in (dict(lse=None), dict(do=None), dict(dq=A + 4), dict(dk=None), dict(lddk=120), dict(dv=None), dict(ws=None), dict(ws=A + 16),
               dict(size=U.ufp4_attn_workspace_bytes(10, 4) - 1)):
        assert bwd(**kw) == U.UFP4_ERR_INVALID_ARG, kw
    assert fwd(T=0, q=None) == U.UFP4_OK and bwd(B=0, q=None) == U.UFP4_OK
    assert U.ufp4_attn_workspace_bytes(0, 4) == 0 and U.ufp4_attn_workspace_bytes(5, 0) == 0
    assert U.ufp4_attn_workspace_bytes(5, 4096) == 0
