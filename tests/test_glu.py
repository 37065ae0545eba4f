"""Gated activation with MXFP8 checkpoints and its backward pass, against the
formulas in 64 bits.

Tolerances.  h, dgate, dup are rounded once to bf16: half a step, 2^-8 of the
value as torch.finfo(bfloat16).eps / 2.  Before that they are fp32 chains of
about ten operations, the hardware exponential and reciprocal among them: 2^-20
of the value covers them, plus the argument y of the exponential: GELU's cubic
carries about 3 roundings, 3 2^-24 |y| in the logistic function, which is 0 or 1
for |y| above 104, so below 2^-15.6 in all; 2^-15 is allowed for everything.
Where act' passes zero its terms cancel: an absolute 2^-18 of |dh u| (1 - s is
off by 2^-24, times g y' of at most about 16 where it matters).
The row sum is 64-term lane sums and a tree over at most 1536 products: 2^-18
of the sum of magnitudes.  The checkpoint itself is exact arithmetic: its codes
and scales are compared with the oracle's, bit for bit."""
import math

import numpy as np
import pytest
import torch

import oracle as O
import rht_bit_block_amd as U

BF16 = torch.finfo(torch.bfloat16).eps / 2
ACTS = [U.UFP4_ACT_SILU, U.UFP4_ACT_GELU]


def act64(g, act):
    if act == U.UFP4_ACT_SILU:
        y, dy = g, torch.ones_like(g)
    else:
        k = 2.0 * math.sqrt(2.0 / math.pi)
        y, dy = k * (g + 0.044715 * g ** 3), k * (1.0 + 3 * 0.044715 * g ** 2)
    s = torch.sigmoid(y)
    return g * s, s * (1.0 + g * torch.sigmoid(-y) * dy)


def values64(codes, scales, cols):
    """What E4M3 codes [rows, cols] and their E8M0 scales stand for."""
    v = codes.cpu().view(torch.float8_e4m3fn).double()
    e = scales.cpu().double() - 127
    return v * torch.exp2(e).repeat_interleave(32, 1)[:, :cols]


def inputs(rows, cols, dtype, seed, spread=True):
    g = torch.Generator().manual_seed(seed)
    a = torch.randn(rows, cols, generator=g) * 2
    b = torch.randn(rows, cols, generator=g)
    if spread:   # blocks of very different sizes, and empty ones
        a *= torch.exp2(torch.randint(-6, 4, (rows, 1), generator=g).float())
        b[:, 32:64] = 0
    d = torch.randn(rows, cols, generator=g) * 1e-3
    r = torch.rand(rows, generator=g)
    if rows > 2:
        r[1] = 0.0   # a padding row
    return a.to(dtype), b.to(dtype), d.to(dtype), r


def close(got, want, rel, floor):
    got, want = got.double().cpu(), want
    bad = (got - want).abs() > rel * want.abs() + floor
    assert not bad.any(), (int(bad.sum()), (got - want).abs().max().item())


def check_case(rows, cols, dtype, act, scaled, again, seed, ld=None):
    print("case: glu", rows, cols, dtype, act, scaled, again, ld, flush=True)
    a, b, d, r = inputs(rows, cols, dtype, seed)

    def dev(t):
        if ld is None:
            return t.cuda()
        big = torch.full((rows, ld), float("nan"), dtype=t.dtype, device="cuda")
        big[:, :cols] = t.cuda()
        return big[:, :cols]

    ga, gb, gd = dev(a), dev(b), dev(d)
    row = r.cuda() if scaled else None
    h, kept = U.ufp4_glu_fwd(ga, gb, act=act, row_scale=row)
    h0, none = U.ufp4_glu_fwd(ga, gb, act=act, row_scale=row, checkpoint=False)
    dg, du, dr, hh = U.ufp4_glu_bwd(kept, gd, row_scale=row, recompute=again)
    torch.cuda.synchronize()
    assert none is None and torch.equal(h.view(torch.int16), h0.view(torch.int16))
    assert (dr is not None) == scaled and (hh is not None) == again

    A, B, D = a.double(), b.double(), d.double()
    R = r.double()[:, None] if scaled else torch.ones(rows, 1, dtype=torch.float64)
    rel = BF16 + 2.0 ** -15
    want, _ = act64(A, act)
    close(h, R * want * B, rel, 1e-38)
    A, B = (values64(c, s, cols) for c, s in ((kept.gate_codes, kept.gate_scales),
                                              (kept.up_codes, kept.up_scales)))
    f, df = act64(A, act)
    close(dg, R * D * B * df, rel, 2.0 ** -18 * (R * D * B).abs() + 1e-38)
    close(du, R * D * f, rel, 1e-38)
    if again:
        close(hh, R * f * B, rel, 1e-38)
    if scaled:
        close(dr, (D * f * B).sum(1), 0.0, 2.0 ** -18 * (D * f * B).abs().sum(1) + 1e-38)
    return kept, (a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,cols,scaled,again", [
    (1, 1408, True, False), (3, 1, True, True), (5, 7, False, False), (2, 31, True, False),
    (4, 33, True, True), (129, 96, False, True), (17, 1411, True, False), (64, 256, True, True),
    (1, 8, False, True), (300, 40, True, True), (257, 520, False, False)])
def test_glu_matches_formulas(rows, cols, scaled, again, dtype, act):
    check_case(rows, cols, dtype, act, scaled, again, seed=rows * 7 + cols)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols,ld", [(96, 104), (96, 101), (40, 41), (33, 64)])
def test_glu_strided_inputs(cols, ld, dtype):
    """Rows inside wider matrices whose other columns are NaN."""
    check_case(9, cols, dtype, U.UFP4_ACT_SILU, True, True, seed=cols + ld, ld=ld)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(33, 256), (7, 1408)])
def test_checkpoint_equals_oracle_quantizer(rows, cols):
    """bf16 inputs: codes and scales are the oracle's MXFP8 quantization bit for
    bit, and ufp4_dequant reads them."""
    print("case: glu checkpoint oracle", rows, cols, flush=True)
    a, b, _, _ = inputs(rows, cols, torch.bfloat16, 5)
    _, kept = U.ufp4_glu_fwd(a.cuda(), b.cuda())
    spec = O.QuantSpec(U.UFP4_E4M3, U.UFP4_RTNE, U.UFP4_SCALE_POW2, 1, 32, 1, 0)
    qa, qb = kept.qtensors()
    for x, q in ((a, qa), (b, qb)):
        ref = O.quantize(x.view(torch.int16).numpy().view(np.uint16), 0, spec)
        assert np.array_equal(q.codes.cpu().numpy(), ref["codes"])
        assert np.array_equal(q.scales.cpu().numpy(), ref["scales"])
        got = U.ufp4_dequant(q)
        assert torch.equal(got.cpu().double(), values64(q.codes, q.scales, cols))


@pytest.mark.gpu
def test_checkpoint_scale_borders():
    """absmax exactly at, just above and just below 448 2^e; zeros; subnormals;
    the largest float: the least scale that holds the block, by definition."""
    tops = [448.0, 448.00003, 447.99997, 0.0, 1e-45, 2.0 ** -126, 1.75 * 2.0 ** -119, 3.4028234e38,
            1.0, 1.75, 1.7500001, 2.0 ** 100]
    x = torch.zeros(len(tops), 32)
    for i, t in enumerate(tops):
        x[i, i] = -t
        x[i, (i + 5) % 32] = t / 3
    print("case: glu checkpoint borders", flush=True)
    _, kept = U.ufp4_glu_fwd(x.cuda(), x.cuda())
    for i in range(len(tops)):
        m = float(x[i].abs().max().double())
        e = -127
        while m > 448.0 * 2.0 ** e:
            e += 1
        assert int(kept.gate_scales[i, 0]) == e + 127, (i, tops[i])
        v = (x[i].double() * 2.0 ** -e)
        q = v.float().to(torch.float8_e4m3fn)
        q = torch.where(q.float() == 0, torch.zeros_like(q.float()), q.float())
        got = kept.gate_codes[i].cpu().view(torch.float8_e4m3fn).float()
        assert torch.equal(got, q), (i, tops[i])
        assert not (kept.gate_codes[i] == 0x80).any()


@pytest.mark.gpu
def test_glu_nonfinite():
    """A NaN stays where it is; an infinity survives the checkpoint; other
    blocks and rows are untouched."""
    print("case: glu nonfinite", flush=True)
    x = torch.ones(3, 96)
    x[0, 3] = float("nan")
    x[1, 40] = float("inf")
    x[1, 41] = -float("inf")
    _, kept = U.ufp4_glu_fwd(x.cuda(), torch.ones(3, 96).cuda())
    v = values64(kept.gate_codes, kept.gate_scales, 96).float()
    assert torch.isnan(v[0, 3]) and int(torch.isnan(v).sum()) == 1
    assert v[1, 40] == float("inf") and v[1, 41] == -float("inf")
    assert (v[0, 4:] == 1).all() and (v[1, :32] == 1).all() and (v[1, 64:] == 1).all()
    assert (v[2] == 1).all()
    dg, du, dr, _ = U.ufp4_glu_bwd(kept, torch.ones(3, 96).cuda(), row_scale=torch.ones(3).cuda())
    assert torch.isnan(dr[0]) and torch.isfinite(dr[2])
    assert int(torch.isnan(dg[0]).sum()) == 1 and torch.isfinite(dg[2]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_glu_extreme_gates(act):
    """Gates far out on both sides: act is 0 or g, its slope 0 or 1, no NaN."""
    print("case: glu extremes", act, flush=True)
    g = torch.tensor([[-1e30, -1e4, -200.0, -90.0, 90.0, 200.0, 1e4, 1e30]]).repeat(2, 4)
    u = torch.ones_like(g)
    h, kept = U.ufp4_glu_fwd(g.cuda(), u.cuda(), act=act)
    want = torch.where(g > 0, g, torch.zeros_like(g))
    got = h.float().cpu()
    assert torch.isfinite(got).all()
    assert ((got - want).abs() <= BF16 * want.abs() + 1e-30).all()
    one = torch.full((2, 32), 1e4)
    _, kept = U.ufp4_glu_fwd(one.cuda(), u.cuda(), act=act)
    dg, _, _, _ = U.ufp4_glu_bwd(kept, u.cuda())
    assert (dg.float() == 1).all()
    _, kept = U.ufp4_glu_fwd(-one.cuda(), u.cuda(), act=act)
    dg, _, _, _ = U.ufp4_glu_bwd(kept, u.cuda())
    assert (dg.float() == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_glu_gradient_against_differences(act):
    """The backward formulas are the derivative of the forward pass at the
    checkpointed values: central differences in 64 bits of the sum of dh * h."""
    print("case: glu differences", act, flush=True)
    a, b, d, r = inputs(6, 64, torch.float32, 77, spread=False)
    _, kept = U.ufp4_glu_fwd(a.cuda(), b.cuda(), act=act, row_scale=r.cuda())
    dg, du, dr, _ = U.ufp4_glu_bwd(kept, d.cuda(), row_scale=r.cuda())
    A, B = (values64(c, s, 64) for c, s in ((kept.gate_codes, kept.gate_scales),
                                            (kept.up_codes, kept.up_scales)))
    D, R, e = d.double(), r.double()[:, None], 1e-5
    f = lambda x: act64(x, act)[0]  # noqa: E731
    diff = R * D * B * (f(A + e) - f(A - e)) / (2 * e)
    # the differences' own error: e^2 |act'''| / 6 and 2^-53 |act| / e, both below 1e-9
    close(dg, diff, BF16 + 2.0 ** -15, (2.0 ** -18 + 1e-8) * (R * D * B).abs() + 1e-30)
    close(du, R * D * f(A), BF16 + 2.0 ** -15, 1e-30)
    close(dr, (D * f(A) * B).sum(1), 0.0, 2.0 ** -18 * (D * f(A) * B).abs().sum(1) + 1e-30)


@pytest.mark.gpu
def test_glu_repeats_on_a_side_stream_and_in_a_graph():
    """The same bits on another stream and from a captured graph replayed
    between eager calls."""
    print("case: glu stream and graph", flush=True)
    a, b, d, r = (t.cuda() for t in inputs(200, 1408, torch.float32, 9))
    ref = U.ufp4_glu_fwd(a, b, row_scale=r)
    rb = U.ufp4_glu_bwd(ref[1], d, row_scale=r, recompute=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        h, kept = U.ufp4_glu_fwd(a, b, row_scale=r)
        out = U.ufp4_glu_bwd(kept, d, row_scale=r, recompute=True)
    torch.cuda.current_stream().wait_stream(s)
    same = lambda x, y: torch.equal(x.view(torch.uint8), y.view(torch.uint8))  # noqa: E731
    assert same(h, ref[0]) and all(same(x, y) for x, y in zip(out, rb))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gh, gk = U.ufp4_glu_fwd(a, b, row_scale=r)
        gout = U.ufp4_glu_bwd(gk, d, row_scale=r, recompute=True)
    for _ in range(3):
        for t in (gh, *gout):
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        U.ufp4_glu_fwd(b, a)
        assert same(gh, ref[0]) and all(same(x, y) for x, y in zip(gout, rb))


@pytest.mark.gpu
def test_glu_empty():
    print("case: glu empty", flush=True)
    z = torch.empty(0, 64, device="cuda")
    h, kept = U.ufp4_glu_fwd(z, z)
    assert h.shape == (0, 64)
    dg, du, dr, hh = U.ufp4_glu_bwd(kept, z, row_scale=torch.empty(0, device="cuda"), recompute=True)
    assert dg.shape == (0, 64) and dr.shape == (0,)
    z = torch.empty(5, 0, device="cuda")
    h, kept = U.ufp4_glu_fwd(z, z)
    _, _, dr, _ = U.ufp4_glu_bwd(kept, z, row_scale=torch.ones(5, device="cuda"))
    assert torch.equal(dr.cpu(), torch.zeros(5))


# --- refusals (no GPU) -------------------------------------------------------
FAKE = 0x10000


def raw_fwd(lib, **kw):
    a = dict(gate=FAKE, up=FAKE, dtype=1, rows=4, cols=64, ld=64, act=0, row=0, h=FAKE, ldh=64,
             gc=FAKE, gs=FAKE, uc=FAKE, us=FAKE)
    a.update(kw)
    return lib.ufp4_glu_fwd(a["gate"], a["up"], a["dtype"], a["rows"], a["cols"], a["ld"], a["act"],
                            a["row"], a["h"], a["ldh"], a["gc"], a["gs"], a["uc"], a["us"], None)


def raw_bwd(lib, **kw):
    a = dict(gc=FAKE, gs=FAKE, uc=FAKE, us=FAKE, rows=4, cols=64, act=0, row=FAKE, dh=FAKE, dtype=1,
             lddh=64, dg=FAKE, du=FAKE, ldd=64, dr=FAKE, h=FAKE, ldh=64)
    a.update(kw)
    return lib.ufp4_glu_bwd(a["gc"], a["gs"], a["uc"], a["us"], a["rows"], a["cols"], a["act"],
                            a["row"], a["dh"], a["dtype"], a["lddh"], a["dg"], a["du"], a["ldd"],
                            a["dr"], a["h"], a["ldh"], None)


def test_glu_abi_refusals():
    lib = U.lib_handle()
    bad = U.UFP4_ERR_INVALID_ARG
    for kw in (dict(dtype=2), dict(dtype=-1), dict(act=2), dict(rows=-1), dict(cols=-1), dict(ld=63),
               dict(ldh=63), dict(gate=0), dict(up=0), dict(h=0), dict(gs=0), dict(uc=0),
               dict(gc=0, gs=0, uc=0), dict(gate=FAKE + 2), dict(up=FAKE + 1, dtype=0),
               dict(h=FAKE + 1), dict(row=FAKE + 2), dict(rows=1 << 60),
               dict(rows=1 << 40, ld=1 << 40)):
        assert raw_fwd(lib, **kw) == bad, kw
    assert raw_fwd(lib, rows=0, gate=0, h=0) == U.UFP4_OK
    assert raw_fwd(lib, cols=0, gate=0, h=0) == U.UFP4_OK
    big = (1 << 30) + 1
    assert raw_fwd(lib, rows=1, cols=big, ld=big, ldh=big) == U.UFP4_ERR_UNSUPPORTED
    for kw in (dict(dtype=2), dict(act=-1), dict(rows=-1), dict(cols=-1), dict(lddh=63), dict(ldd=63),
               dict(ldh=63), dict(row=0), dict(gc=0), dict(gs=0), dict(uc=0), dict(us=0), dict(dh=0),
               dict(dg=0), dict(du=0), dict(dh=FAKE + 2), dict(dg=FAKE + 1), dict(du=FAKE + 1),
               dict(h=FAKE + 1), dict(dr=FAKE + 1), dict(row=FAKE + 2), dict(rows=1 << 60)):
        assert raw_bwd(lib, **kw) == bad, kw
    assert raw_bwd(lib, rows=0, gc=0, dh=0) == U.UFP4_OK
    assert raw_bwd(lib, cols=0, dr=0, gc=0, dh=0) == U.UFP4_OK
    assert raw_bwd(lib, rows=1, cols=big, lddh=big, ldd=big, ldh=big) == U.UFP4_ERR_UNSUPPORTED


def test_glu_binding_refusals():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="GPU"):
        U.ufp4_glu_fwd(x, x)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        U.ufp4_glu_fwd(x.half(), x.half())
    with pytest.raises(ValueError, match="up must have dtype"):
        U.ufp4_glu_fwd(x, x.bfloat16())
    with pytest.raises(ValueError, match="up has shape"):
        U.ufp4_glu_fwd(x, x[:3])
    with pytest.raises(ValueError, match="same row pitch"):
        U.ufp4_glu_fwd(torch.zeros(4, 128)[:, :64], x)
    with pytest.raises(ValueError, match="unit column stride"):
        U.ufp4_glu_fwd(torch.zeros(64, 4).t(), x)
    with pytest.raises(ValueError, match="row_scale"):
        U.ufp4_glu_fwd(x, x, row_scale=torch.ones(3))
    with pytest.raises(ValueError, match="out has shape"):
        U.ufp4_glu_fwd(x, x, out=torch.zeros(4, 63, dtype=torch.bfloat16))
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    ok = U.GluCheckpoint(u8(4, 64), u8(4, 2), u8(4, 64), u8(4, 2), U.UFP4_ACT_SILU)
    with pytest.raises(ValueError, match="GPU"):
        U.ufp4_glu_bwd(ok, x)
    with pytest.raises(ValueError, match="dh has shape"):
        U.ufp4_glu_bwd(ok, x[:, :63])
    with pytest.raises(ValueError, match="up_scales"):
        U.ufp4_glu_bwd(U.GluCheckpoint(u8(4, 64), u8(4, 2), u8(4, 64), u8(4, 1), 0), x)
    with pytest.raises(ValueError, match="contiguous"):
        U.ufp4_glu_bwd(U.GluCheckpoint(u8(4, 128)[:, ::2], u8(4, 2), u8(4, 64), u8(4, 2), 0), x)
    with pytest.raises(ValueError, match="32"):
        U.GluCheckpoint(u8(4, 33), u8(4, 2), u8(4, 33), u8(4, 2), 0).qtensors()
