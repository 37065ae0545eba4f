"""The mixture-of-experts layer for a few tokens on 4-bit weights, against the
formulas in 64 bits on the dequantized weights.

Tolerances, elementwise, each step's error carried through the next by the
magnitudes of what it is multiplied with.  Rotation: at most 8 fp32 roundings
against the sum of magnitudes, 2^-20.  Split into two bf16 pieces: half a step
of half a step, 2^-16.  Products: exact, summed in fp32 over K, (K + 16) 2^-24
of the sum of magnitudes.  Activation: its slope is below 1.13, its own error
2^-18 of itself (hardware exponential and reciprocal; arguments below 32 here).
The router's shares: 2^-19.  The output is rounded once to bf16, 2^-8."""
import math

import numpy as np
import pytest
import torch

import oracle as O
import rht_bit_block_amd as U
from gpu_helpers import spec_of

BF16 = torch.finfo(torch.bfloat16).eps / 2
EPS = 2.0 ** -24


def bits(x):
    return x.contiguous().view(torch.int16).numpy().view(np.uint16)


def quantized(P, K, cfg, seed):
    """A quantized weight: the device operand and its values in 64 bits, in
    the rotated basis."""
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(P, K, generator=g) / math.sqrt(K)).to(torch.bfloat16)
    ref = O.quantize(bits(w), 0, spec_of(cfg))
    q = U.QTensor(torch.from_numpy(ref["codes"]), torch.from_numpy(np.ascontiguousarray(ref["scales"])),
                  P, K, cfg)
    if torch.cuda.is_available():
        q = U.QTensor(q.codes.cuda(), q.scales.cuda(), P, K, cfg)
    _, v = O.dequant(ref["codes"], ref["scales"], spec_of(cfg), P, K)
    return q, torch.from_numpy(np.asarray(v, dtype=np.float64)).reshape(P, K), w


def rotation(cfg):
    """S H / sqrt(n) of a configuration, the signs from the oracle."""
    n = cfg.rht_n
    if n == 1:
        return torch.ones(1, 1, dtype=torch.float64)
    m = torch.ones(1, 1, dtype=torch.float64)
    while m.shape[0] < n:
        m = torch.cat([torch.cat([m, m], 1), torch.cat([m, -m], 1)], 0)
    s = torch.from_numpy(np.asarray(O.rht_signs(cfg.sign_seed, n), dtype=np.float64).reshape(-1)[:n])
    return s[:, None] * m / math.sqrt(n)


def turn(x, R):
    n = R.shape[0]
    return (x.reshape(-1, n) @ R).reshape(x.shape)


def act64(g, act):
    if act == U.UFP4_ACT_SILU:
        return g * torch.sigmoid(g)
    return g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))


def choices(logits, k, renorm):
    """[(token, expert, share)], by the definition."""
    out = []
    for t, row in enumerate(logits.double().tolist()):
        open_ = [e for e in range(len(row)) if row[e] > -math.inf]
        got = sorted(open_, key=lambda e: (-row[e], e))[:k]
        over = got if renorm else open_
        if got:
            top = max(row[e] for e in over)
            den = sum(math.exp(row[e] - top) for e in over)
            out += [(t, e, math.exp(row[e] - top) / den) for e in got]
    return out


def formulas(x, logits, wg, wu, wd, cfg, dcfg, k, renorm, act):
    """y and the bound on its error."""
    T, H = x.shape
    E = logits.shape[1]
    F = wd.shape[1]
    R, D = rotation(cfg), rotation(dcfg)
    X = x.double()
    xr, xa = turn(X, R), turn(X.abs(), R.abs())
    dx = 2.0 ** -16 * xr.abs() + 2.0 ** -20 * xa
    y, tol = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for t, e, p in choices(logits, k, renorm):
        G, Uw, Dw = wg[e * F:(e + 1) * F], wu[e * F:(e + 1) * F], wd[e * H:(e + 1) * H]
        g, u = G @ xr[t], Uw @ xr[t]
        dg, du = (M.abs() @ dx[t] + (H + 16) * EPS * (M.abs() @ xr[t].abs()) for M in (G, Uw))
        a = act64(g, act)
        h = p * a * u
        dh = p * (1.13 * dg * (u.abs() + du) + a.abs() * du) + 2.0 ** -17 * h.abs()
        hr, ha = turn(h, D), turn(h.abs(), D.abs())
        dr = turn(dh, D.abs()) + 2.0 ** -16 * hr.abs() + 2.0 ** -20 * ha
        y[t] += Dw @ hr
        tol[t] += Dw.abs() @ dr + (F + 64) * EPS * (Dw.abs() @ hr.abs())
    return y, tol + BF16 * (y.abs() + tol)


def inputs(T, E, H, seed, masked=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    logits = torch.randn(T, E, generator=g) * 2
    if masked:
        logits[torch.rand(T, E, generator=g) < 0.5] = -math.inf
        logits[T // 2] = -math.inf
    return x, logits


def build(E, H, F, cfg, dcfg, seed):
    qg, vg, _ = quantized(E * F, H, cfg, seed)
    qu, vu, _ = quantized(E * F, H, cfg, seed + 1)
    qd, vd, _ = quantized(E * H, F, dcfg, seed + 2)
    return (qg, qu, qd), (vg, vu, vd)


def check(y, want, tol):
    off = (y.double().cpu() - want).abs()
    bad = off > tol
    assert not bad.any(), (int(bad.sum()), bad.numel(), off.max().item(),
                           (off / want.norm() * want.numel() ** 0.5).max().item())


def mk(grid, block, n, seed, pow2=False, rows=1, ts=0.0):
    return U.make_cfg(grid, U.UFP4_RTNE, U.UFP4_SCALE_POW2 if pow2 else U.UFP4_SCALE_F32, rows, block,
                      n, sign_seed=seed, tensor_scale=ts)


def run_case(T, E, k, H, F, cfg, dcfg, renorm=True, act=U.UFP4_ACT_SILU, masked=False, seed=1):
    print("case: moe", T, E, k, H, F, cfg.grid, cfg.block_cols, cfg.rht_n, dcfg.rht_n, renorm, act,
          masked, flush=True)
    q, v = build(E, H, F, cfg, dcfg, seed)
    x, logits = inputs(T, E, H, seed + 9, masked)
    y = U.ufp4_moe_tokens(x.cuda(), logits.cuda(), *q, k, renorm=renorm, act=act)
    torch.cuda.synchronize()
    check(y, *formulas(x, logits, *v, cfg, dcfg, k, renorm, act))
    return q, x, logits, y


@pytest.mark.gpu
@pytest.mark.parametrize("grid", [U.UFP4_E1M2, U.UFP4_INT4, U.UFP4_E2M1])
@pytest.mark.parametrize("block,n,pow2,rows", [
    (16, 16, False, 1), (32, 32, False, 1), (16, 128, False, 1), (32, 64, False, 1),
    (32, 1, False, 1), (16, 2, False, 1), (32, 32, True, 1), (32, 128, True, 1), (32, 8, True, 32),
    (16, 4, True, 16)])
def test_moe_formats(grid, block, n, pow2, rows):
    cfg, dcfg = mk(grid, block, n, 5, pow2, rows), mk(grid, block, n, 6, pow2, rows)
    run_case(3, 4, 2, 256, 256, cfg, dcfg)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,H,F,renorm,act,masked", [
    (1, 1, 1, 32, 32, True, 0, False), (1, 64, 6, 128, 64, True, 0, False),
    (2, 8, 8, 96, 96, False, 1, False), (16, 4, 2, 160, 32, True, 1, True),
    (17, 3, 3, 128, 96, True, 0, False), (33, 5, 2, 64, 160, False, 0, True),
    (64, 2, 2, 64, 64, True, 1, False), (64, 130, 4, 64, 32, True, 0, True),
    (5, 256, 16, 64, 32, False, 0, False), (64, 16, 8, 128, 128, True, 0, False)])
def test_moe_sizes(T, E, k, H, F, renorm, act, masked):
    run_case(T, E, k, H, F, mk(U.UFP4_INT4, 32, 32, 5), mk(U.UFP4_INT4, 16, 16, 6), renorm, act,
             masked, seed=T + E)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(1, 8, 4), (20, 8, 4), (64, 16, 3)])
def test_moe_split_down(T, E, k):
    """Sizes at which the down product is split over workgroups, twice with the
    same bits."""
    cfg = mk(U.UFP4_INT4, 16, 128, 5)
    q, x, logits, y = run_case(T, E, k, 256, 1408, cfg, mk(U.UFP4_INT4, 16, 128, 9))
    for _ in range(3):
        assert torch.equal(y, U.ufp4_moe_tokens(x.cuda(), logits.cuda(), *q, k))


@pytest.mark.gpu
def test_moe_tensor_scales_and_mixed_weights():
    """Two-level scales, another grid and rotation for the down weights."""
    run_case(4, 4, 2, 128, 64, mk(U.UFP4_E2M1, 32, 32, 1, True, 1, 0.37),
             mk(U.UFP4_E1M2, 16, 64, 2))
    run_case(4, 4, 2, 128, 64, mk(U.UFP4_INT4, 32, 16, 1),
             mk(U.UFP4_E2M1, 32, 1, 2, True, 32, 3.1))


@pytest.mark.gpu
def test_moe_choices():
    """Ties go to the lowest index; -inf and NaN are never chosen; a token with
    nothing open is 0; fewer open experts than top_k."""
    print("case: moe choices", flush=True)
    E, H, F, k = 70, 64, 32, 3
    cfg, dcfg = mk(U.UFP4_INT4, 32, 32, 5), mk(U.UFP4_INT4, 32, 32, 6)
    q, v = build(E, H, F, cfg, dcfg, 3)
    x, _ = inputs(6, E, H, 4)
    logits = torch.zeros(6, E)                       # row 0: all equal -> 0, 1, 2
    logits[1] = -5.0
    logits[1, [69, 64, 5, 66]] = 1.0                 # -> 5, 64, 66
    logits[2] = -math.inf
    logits[2, 68] = -3.0                             # one open
    logits[3] = -math.inf                            # none
    logits[4] = -1.0
    logits[4, :66] = float("nan")                    # -> 66, 67, 68
    logits[5] = torch.arange(E).float() * 1e30       # far apart -> 69 takes it all
    for renorm in (True, False):
        y = U.ufp4_moe_tokens(x.cuda(), logits.cuda(), *q, k, renorm=renorm)
        torch.cuda.synchronize()
        assert not y[3].any()
        check(y, *formulas(x, logits, *v, cfg, dcfg, k, renorm, U.UFP4_ACT_SILU))


@pytest.mark.gpu
def test_moe_matches_the_unquantized_layer_through_the_quantizer():
    """Weights through ufp4_rht_quant: the layer is that of the weights'
    dequantized values turned back into the unrotated basis."""
    print("case: moe through quantizer", flush=True)
    E, H, F, T, k = 4, 256, 128, 5, 2
    cfg, dcfg = mk(U.UFP4_E1M2, 16, 64, 11), mk(U.UFP4_E1M2, 16, 128, 12)
    g = torch.Generator().manual_seed(8)
    ws = [(torch.randn(*s, generator=g) / 16).to(torch.bfloat16) for s in
          ((E * F, H), (E * F, H), (E * H, F))]
    qs = [U.ufp4_rht_quant(w.cuda(), 0, c)[0] for w, c in zip(ws, (cfg, cfg, dcfg))]
    vs = [U.ufp4_dequant(q).double().cpu() for q in qs]
    x, logits = inputs(T, E, H, 3)
    y = U.ufp4_moe_tokens(x.cuda(), logits.cuda(), *qs, k)
    check(y, *formulas(x, logits, *vs, cfg, dcfg, k, True, U.UFP4_ACT_SILU))
    # E1M2 at 4 bits: the layer of the original weights within the quantization's error
    back = [turn(v, rotation(c).t().contiguous()) for v, c in zip(vs, (cfg, cfg, dcfg))]
    for b, w in zip(back, ws):
        assert (b - w.double()).norm() < 0.2 * w.double().norm()


@pytest.mark.gpu
def test_moe_strided_rows():
    print("case: moe strided", flush=True)
    T, E, H, F, k = 5, 4, 64, 64, 2
    cfg, dcfg = mk(U.UFP4_INT4, 32, 32, 5), mk(U.UFP4_INT4, 32, 32, 6)
    q, v = build(E, H, F, cfg, dcfg, 3)
    x, logits = inputs(T, E, H, 4)
    wide = torch.full((T, 80), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :H] = x.cuda()
    lw = torch.full((T, 9), float("nan"), device="cuda")
    lw[:, :E] = logits.cuda()
    out = torch.full((T, 70), 7.0, dtype=torch.bfloat16, device="cuda")
    U.ufp4_moe_tokens(wide[:, :H], lw[:, :E], *q, k, out=out[:, :H])
    check(out[:, :H], *formulas(x, logits, *v, cfg, dcfg, k, True, U.UFP4_ACT_SILU))
    assert (out[:, H:] == 7).all()


@pytest.mark.gpu
def test_moe_on_a_side_stream_and_in_a_graph():
    print("case: moe stream and graph", flush=True)
    cfg = mk(U.UFP4_INT4, 16, 128, 5)
    q, x, logits, ref = run_case(20, 8, 4, 256, 1408, cfg, mk(U.UFP4_INT4, 16, 128, 9))
    x, logits = x.cuda(), logits.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = U.ufp4_moe_tokens(x, logits, *q, 4)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = U.ufp4_moe_tokens(x, logits, *q, 4)
    for _ in range(3):
        y.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        U.ufp4_moe_tokens(x[:3], logits[:3], *q, 2)
        assert torch.equal(y, ref)


@pytest.mark.gpu
def test_moe_no_tokens():
    cfg = mk(U.UFP4_INT4, 32, 32, 5)
    q, _ = build(2, 64, 32, cfg, cfg, 3)
    y = U.ufp4_moe_tokens(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"),
                          torch.empty(0, 2, device="cuda"), *q, 1)
    assert y.shape == (0, 64)


# --- refusals (no GPU) -------------------------------------------------------
FAKE = 0x10000


def raw(lib, **kw):
    cfg = kw.pop("cfg", None) or mk(U.UFP4_INT4, 32, 32, 5)
    a = dict(x=FAKE, ldx=64, T=4, lg=FAKE, ldl=8, E=8, k=2, act=0, g=(8 * 32, 64, cfg),
             u=(8 * 32, 64, cfg), d=(8 * 64, 32, cfg), y=FAKE, ldy=64, ws=FAKE, n=1 << 40,
             codes=FAKE)
    a.update(kw)
    import ctypes
    q = [None if a[n] is None else U.QTensorC(a["codes"], FAKE, *a[n]) for n in ("g", "u", "d")]
    ref = [None if x is None else ctypes.byref(x) for x in q]
    return lib.ufp4_moe_tokens(a["x"], a["ldx"], a["T"], a["lg"], a["ldl"], a["E"], a["k"], 1,
                               a["act"], *ref, a["y"], a["ldy"], a["ws"], a["n"], None)


def test_moe_abi_refusals():
    lib = U.lib_handle()
    bad, shape = U.UFP4_ERR_INVALID_ARG, U.UFP4_ERR_SHAPE
    no, mismatch = U.UFP4_ERR_UNSUPPORTED, U.UFP4_ERR_MISMATCH
    c = mk(U.UFP4_INT4, 32, 32, 5)
    e4m3 = U.make_cfg(U.UFP4_E4M3, U.UFP4_RTNE, U.UFP4_SCALE_POW2, 1, 32, 32)
    c16 = mk(U.UFP4_INT4, 16, 16, 5)
    for kw, want in [
            (dict(act=2), bad), (dict(g=None), bad), (dict(d=None), bad), (dict(E=0), bad),
            (dict(x=0), bad), (dict(lg=0), bad), (dict(y=0), bad), (dict(ws=0), bad),
            (dict(x=FAKE + 8), bad), (dict(ldx=60), bad), (dict(ldx=68), bad), (dict(ldl=7), bad),
            (dict(ldy=62), bad), (dict(ldy=65), bad), (dict(y=FAKE + 2), bad), (dict(T=-1), bad),
            (dict(k=0), bad), (dict(k=9), bad), (dict(n=64), bad), (dict(ws=FAKE + 128), bad),
            (dict(codes=FAKE + 8), bad), (dict(T=65), no), (dict(E=7), shape),
            (dict(g=(8 * 32, 80, c16), u=(8 * 32, 80, c16)), shape),
            (dict(g=(8 * 48, 64, c16), u=(8 * 48, 64, c16)), shape),
            (dict(d=(8 * 64, 64, c)), shape), (dict(d=(8 * 32, 32, c)), shape),
            (dict(u=(8 * 64, 64, c)), shape), (dict(u=(8 * 32, 32, c)), mismatch),
            (dict(u=(8 * 32, 64, mk(U.UFP4_E1M2, 32, 32, 5))), mismatch),
            (dict(u=(8 * 32, 64, mk(U.UFP4_INT4, 16, 32, 5))), mismatch),
            (dict(u=(8 * 32, 64, mk(U.UFP4_INT4, 32, 64, 5))), mismatch),
            (dict(u=(8 * 32, 64, mk(U.UFP4_INT4, 32, 32, 6))), mismatch),
            (dict(g=(8 * 32, 64, e4m3), u=(8 * 32, 64, e4m3)), no), (dict(d=(8 * 64, 32, e4m3)), no)]:
        assert raw(lib, **kw) == want, kw
    big = (17 * 32, 64, c)
    assert raw(lib, E=17, k=17, ldl=17, g=big, u=big, d=(17 * 64, 32, c)) == no
    wide = (257 * 32, 64, c)
    assert raw(lib, E=257, ldl=257, g=wide, u=wide, d=(257 * 64, 32, c)) == no
    assert raw(lib, T=0, x=0, lg=0, y=0, ws=0, n=0) == U.UFP4_OK
    size = U.ufp4_moe_tokens_workspace_bytes
    assert size(0, 8, 2, 64, 32) == 0 and size(65, 8, 2, 64, 32) == 0 and size(4, 8, 9, 64, 32) == 0
    need = size(4, 8, 2, 64, 32)
    assert need > 0 and raw(lib, n=need - 1) == bad


def test_moe_binding_refusals():
    cfg = mk(U.UFP4_INT4, 32, 32, 5)

    def q(P, K):
        return U.QTensor(torch.zeros(P, K // 2, dtype=torch.uint8), torch.zeros(P, K // 32), P, K, cfg)

    x, lg = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 8)
    w = (q(256, 64), q(256, 64), q(512, 32))
    with pytest.raises(ValueError, match="GPU"):
        U.ufp4_moe_tokens(x, lg, *w, 2)
    with pytest.raises(ValueError, match="x must have dtype"):
        U.ufp4_moe_tokens(x.float(), lg, *w, 2)
    with pytest.raises(ValueError, match="logits must have dtype"):
        U.ufp4_moe_tokens(x, lg.double(), *w, 2)
    with pytest.raises(ValueError, match="rows"):
        U.ufp4_moe_tokens(x, lg[:3], *w, 2)
    with pytest.raises(ValueError, match="contracts"):
        U.ufp4_moe_tokens(x[:, :32], lg, *w, 2)


class _Cycle:
    """The rows of a few experts, repeated for all."""

    def __init__(self, v, rows, experts):
        self.v, self.rows, self.experts = v, rows, experts

    def __getitem__(self, s):
        e = s.start // self.rows % self.experts
        return self.v[e * self.rows:(e + 1) * self.rows]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,H,F", [
    (33, 16, 4, 3200, 1472), (17, 32, 8, 512, 800), (34, 64, 4, 512, 800), (3, 32, 4, 1024, 1024)])
def test_moe_runs(T, E, k, H, F):
    """Sizes at which a workgroup takes two, three, four or eight pairs of tiles,
    the last one of an expert fewer. Over such long sums the elementwise bound is
    wide; the error of the whole is below a bf16 rounding of every element and, for
    all that is summed in fp32 and split in two pieces, (K + 16) 2^-24 < 2^-12 and
    2^-16 of the whole per product, together below 2^-10."""
    print("case: moe runs", T, E, k, H, F, flush=True)
    cfg, dcfg = mk(U.UFP4_INT4, 32, 32, 5), mk(U.UFP4_E2M1, 32, 16, 6, True)
    some = 3
    q, v = build(some, H, F, cfg, dcfg, T)
    turns = (E + some - 1) // some
    q = [U.QTensor(w.codes.repeat(turns, 1)[:E * P], w.scales.repeat(turns, 1)[:E * P], E * P, w.K, c)
         for w, P, c in zip(q, (F, F, H), (cfg, cfg, dcfg))]
    x, logits = inputs(T, E, H, 7)
    y = U.ufp4_moe_tokens(x.cuda(), logits.cuda(), *q, k)
    torch.cuda.synchronize()
    v = [_Cycle(w, P, some) for w, P in zip(v, (F, F, H))]
    v[2].shape = (E * H, F)
    want, tol = formulas(x, logits, *v, cfg, dcfg, k, True, U.UFP4_ACT_SILU)
    check(y, want, tol)
    assert (y.double().cpu() - want).norm() <= (BF16 + 2.0 ** -10) * want.norm()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 12])
@pytest.mark.parametrize("E", [8, 64, 70, 130])
def test_moe_signed_zeros_tie(E, T):
    """-0 and +0 are equal logits, so the lower index is chosen of the two, on
    both sides of the 64 experts that one register per lane holds and with
    routing inside the up product (few tokens) or in front of it."""
    print("case: moe signed zeros", E, T, flush=True)
    H, F = 64, 32
    cfg, dcfg = mk(U.UFP4_INT4, 32, 32, 5), mk(U.UFP4_INT4, 32, 32, 6)
    q, v = build(E, H, F, cfg, dcfg, 3)
    x, logits = inputs(T, E, H, 4)
    logits[0] = 0.0
    logits[0, ::2] = -0.0                                   # -0 +0 -0 +0 ..
    logits[1] = 0.0
    logits[1, 1::2] = -0.0                                  # +0 -0 +0 -0 ..
    logits[2] = -1.0
    logits[2, [2, E - 2]] = -0.0
    logits[2, [5, E - 1]] = 0.0                             # -> 2, 5, E - 2 in this order
    for k in (1, 2, 3):
        for renorm in (True, False):
            y = U.ufp4_moe_tokens(x.cuda(), logits.cuda(), *q, k, renorm=renorm)
            torch.cuda.synchronize()
            check(y, *formulas(x, logits, *v, cfg, dcfg, k, renorm, U.UFP4_ACT_SILU))


def plain_weight(P, K, cfg, level, scale):
    """A weight whose codes all stand for the same level (INT4)."""
    q = U.QTensor(torch.full((P, K // 2), level * 17, dtype=torch.uint8),
                  torch.full((P, K // cfg.block_cols), scale), P, K, cfg)
    return U.QTensor(q.codes.cuda(), q.scales.cuda(), P, K, cfg)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 12])
@pytest.mark.parametrize("block", [16, 32])
def test_moe_infinite_and_largest_activations(block, T):
    """An infinity in x gives infinities (positive weights, no rotation), not
    NaN, a NaN gives NaN, and both only in their own tokens.  An intermediate
    between the largest bf16 and the largest fp32 value, 2^128 (1 - 2^-10), times
    2^-100 is 2^28 to within bf16's half step 2^-8."""
    print("case: moe infinities", block, T, flush=True)
    H, F, E = 64, 64, 2
    c = mk(U.UFP4_INT4, block, 1, 0)
    w = [plain_weight(E * P, K, c, 1, s) for P, K, s in ((F, H, 2.0 ** -6), (F, H, 2.0 ** -6), (H, F, 2.0 ** -6))]
    x, logits = inputs(T, E, H, 4)
    x = x.abs()
    ref = U.ufp4_moe_tokens(x.cuda(), logits.cuda(), *w, 2)
    x[0, 5] = float("inf")
    x[1, 40] = float("nan")
    y = U.ufp4_moe_tokens(x.cuda(), logits.cuda(), *w, 2)
    torch.cuda.synchronize()
    assert (y[0] == float("inf")).all()
    assert torch.isnan(y[1]).all()
    assert torch.isfinite(ref).all() and torch.equal(y[2:], ref[2:])

    big = 2.0 ** 64
    w = [plain_weight(P, K, c, 1, s) for P, K, s in ((F, H, big), (F, H, big * (1 - 2.0 ** -10)), (H, F, 2.0 ** -100))]
    w[1].codes[1:] = 0                    # one column of the intermediate
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    x[:, 3] = 1.0
    y = U.ufp4_moe_tokens(x.cuda(), torch.zeros(T, 1).cuda(), *w, 1)
    torch.cuda.synchronize()
    assert ((y.double() - 2.0 ** 28 * (1 - 2.0 ** -10)).abs() <= BF16 * 2.0 ** 28).all()


@pytest.mark.parametrize("T,E,k,H,F", [(1, 64, 6, 2048, 1408), (61, 64, 6, 2048, 1408), (16, 16, 8, 5120, 1536),
                                       (64, 256, 16, 1 << 20, 1 << 20), (64, 256, 1, 64, 32)])
def test_moe_workspace_holds_the_choices(T, E, k, H, F):
    """A row of the intermediate and of the down products for each of the T k
    choices (fp32), the rotated tokens (4 bytes an element) and small arrays."""
    need = U.ufp4_moe_tokens_workspace_bytes(T, E, k, H, F)
    rows = 4 * T * k * (H + F)
    assert rows <= need <= rows + 4 * T * H + 16 * T * k + 16 * E + 8 * 256


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 12])
def test_moe_infinite_logits(T):
    """A softmax over +inf is NaN, in its own token only."""
    print("case: moe infinite logits", T, flush=True)
    E, H, F, k = 8, 64, 32, 2
    cfg, dcfg = mk(U.UFP4_INT4, 32, 32, 5), mk(U.UFP4_INT4, 32, 32, 6)
    q, _ = build(E, H, F, cfg, dcfg, 3)
    x, logits = inputs(T, E, H, 4)
    ref = U.ufp4_moe_tokens(x.cuda(), logits.cuda(), *q, k)
    logits[1, 5] = float("inf")
    y = U.ufp4_moe_tokens(x.cuda(), logits.cuda(), *q, k)
    torch.cuda.synchronize()
    assert torch.isnan(y[1]).all()
    rest = [t for t in range(T) if t != 1]
    assert torch.isfinite(ref).all() and torch.equal(y[rest], ref[rest])


@pytest.mark.gpu
@pytest.mark.parametrize("T,k", [(16, 4), (33, 2)])
def test_moe_three_pairs_of_the_down_product(T, k):
    """47 pairs of column tiles of 16 experts over a contraction of 3200: a
    workgroup of the down product takes three of them, the last one two.  Bounds
    as for the runs of the other sizes."""
    E, H, F, some = 16, 1504, 3200, 3
    print("case: moe three pairs", T, k, flush=True)
    cfg, dcfg = mk(U.UFP4_E2M1, 32, 16, 6, True), mk(U.UFP4_INT4, 32, 32, 5)
    q, v = build(some, H, F, cfg, dcfg, T)
    turns = (E + some - 1) // some
    q = [U.QTensor(w.codes.repeat(turns, 1)[:E * P], w.scales.repeat(turns, 1)[:E * P], E * P, w.K, c)
         for w, P, c in zip(q, (F, F, H), (cfg, cfg, dcfg))]
    x, logits = inputs(T, E, H, 7)
    y = U.ufp4_moe_tokens(x.cuda(), logits.cuda(), *q, k)
    torch.cuda.synchronize()
    v = [_Cycle(w, P, some) for w, P in zip(v, (F, F, H))]
    v[2].shape = (E * H, F)
    want, tol = formulas(x, logits, *v, cfg, dcfg, k, True, U.UFP4_ACT_SILU)
    check(y, want, tol)
    assert (y.double().cpu() - want).norm() <= (BF16 + 2.0 ** -10) * want.norm()
