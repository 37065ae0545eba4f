"""Linear softmax cross entropy without stored logits, and its gradients,
against the formulas in 64 bits.

Tolerances.  A logit is an fp32 sum of D exact products: off by at most
D 2^-24 sum |h w| =: E.  Its exponential: E, the rounded argument (2^-23 times
at most 128 for terms that are not 0) and the instruction's 2^-22: p is off by
e_p = 2 E + 2^-15 of itself (lse included).  lse and loss: E + 2^-16 absolute for
the sum of up to V terms in a tree whose longest chain is below 256, and 2^-22
of |lse| and |z|.  G is rounded to bf16, half a step 2^-8 of its value; dh and dw
add V (T) 2^-24 of the sum of magnitudes and one rounding to bf16.  Those are
worst cases; the sums average the independent roundings, so the relative
Frobenius error must also be below 3 2^-8, (two roundings of at most 2^-8 and a
third for what the worst case holds in reserve)."""
import pytest
import torch

import rht_bit_block_amd as U

BF16 = torch.finfo(torch.bfloat16).eps / 2


def inputs(T, V, D, seed, ignored=0.2, size=1.0, device="cpu"):
    g = torch.Generator(device=device).manual_seed(seed)
    w = (torch.randn(V, D, generator=g, device=device) / D ** 0.5 * size).to(torch.bfloat16)
    t = torch.randint(0, V, (T,), generator=g, device=device)
    h = torch.randn(T, D, generator=g, device=device) + 4 * w[t].float()
    out = torch.rand(T, generator=g, device=device) < ignored
    t = torch.where(out, torch.full_like(t, -100), t)
    if T > 3:
        t[T // 2] = V            # past the last class: ignored as well
        t[0], t[1] = 0, V - 1    # the first and the last class
    dloss = torch.rand(T, generator=g, device=device) / T
    dlse = torch.randn(T, generator=g, device=device) * 1e-2 / T
    return h.to(torch.bfloat16), w, t, dloss, dlse


def formulas(h, w, t, dloss, dlse):
    h, w = h.double(), w.double()
    V = w.shape[0]
    z = h @ w.t().contiguous()
    lse = torch.logsumexp(z, 1)
    live = (t >= 0) & (t < V)
    at = torch.where(live, t, torch.zeros_like(t))[:, None]
    zt = z.gather(1, at)[:, 0]
    loss = torch.where(live, lse - zt, torch.zeros_like(lse))
    b = torch.where(live, dloss.double(), torch.zeros_like(lse))
    a = b + (dlse.double() if dlse is not None else 0)
    p = torch.exp(z - lse[:, None]) * a[:, None]
    G = p.clone()
    G.scatter_add_(1, at, -b[:, None])
    E = h.shape[1] * 2.0 ** -24 * (h.abs() @ w.abs().t().contiguous())
    return dict(z=z, lse=lse, loss=loss, zt=zt, G=G, p=p.abs(), E=E, dh=G @ w,
                dw=G.t().contiguous() @ h)


def assert_near(got, want, tol, what):
    bad = (got.double().cpu() - want.cpu()).abs() > tol.cpu()
    assert not bad.any(), (what, int(bad.sum()), int(bad.numel()),
                           (got.double().cpu() - want.cpu()).abs().max().item())


def check_fwd(loss, lse, f):
    e = f["E"].amax(1) + 2.0 ** -16
    assert_near(lse, f["lse"], e + 2.0 ** -22 * f["lse"].abs(), "lse")
    assert_near(loss, f["loss"],
                torch.where(f["loss"] == 0, torch.zeros_like(e),
                            2 * e + 2.0 ** -22 * (f["lse"].abs() + f["zt"].abs())), "loss")


def check_bwd(dh, dw, f, h, w):
    h, w = h.double(), w.double()
    ep = (2 * f["E"].amax(1) + 2.0 ** -15)[:, None] * f["p"]
    G = f["G"].abs()
    slack = BF16 * (G + ep) + ep
    tol = slack @ w.abs() + w.shape[0] * 2.0 ** -24 * (G @ w.abs()) + BF16 * f["dh"].abs()
    assert_near(dh, f["dh"], tol * 1.01 + 1e-38, "dh")
    tol = (slack.t().contiguous() @ h.abs() + h.shape[0] * 2.0 ** -24 * (G.t().contiguous() @ h.abs())
           + BF16 * f["dw"].abs())
    assert_near(dw, f["dw"], tol * 1.01 + 1e-38, "dw")
    for got, want, name in ((dh, f["dh"], "dh"), (dw, f["dw"], "dw")):
        norm = want.norm()
        off = (got.double().to(want.device) - want).norm()
        assert off <= 3 * BF16 * norm + 1e-30, (name, (off / norm).item())


SIZES = [(1, 1, 8), (1, 7, 64), (2, 256, 72), (7, 1003, 256), (33, 255, 136), (65, 257, 64),
         (130, 513, 200), (256, 256, 128), (300, 2000, 328), (257, 31, 520)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,D", SIZES)
def test_xent_matches_formulas(T, V, D):
    print("case: xent", T, V, D, flush=True)
    h, w, t, dloss, dlse = inputs(T, V, D, seed=T + V + D)
    g = [x.cuda() for x in (h, w, t, dloss, dlse)]
    loss, lse = U.ufp4_linear_xent_fwd(*g[:3])
    torch.cuda.synchronize()
    f = formulas(h, w, t, dloss, None)
    check_fwd(loss, lse, f)
    dh, dw = U.ufp4_linear_xent_bwd(*g[:3], lse, g[3])
    torch.cuda.synchronize()
    check_bwd(dh, dw, f, h, w)
    dh, dw = U.ufp4_linear_xent_bwd(*g[:3], lse, g[3], dlse=g[4])
    torch.cuda.synchronize()
    check_bwd(dh, dw, formulas(h, w, t, dloss, dlse), h, w)


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,D", [(8200, 9001, 64), (4, 70001, 64), (1500, 50021, 32)])
def test_xent_in_pieces_and_splits(T, V, D):
    """Vocabularies of several pieces, and a dh product split over K."""
    print("case: xent pieces", T, V, D, flush=True)
    h, w, t, dloss, dlse = inputs(T, V, D, seed=T, device="cuda")
    loss, lse = U.ufp4_linear_xent_fwd(h, w, t)
    dh, dw = U.ufp4_linear_xent_bwd(h, w, t, lse, dloss, dlse)
    torch.cuda.synchronize()
    f = formulas(h, w, t, dloss, dlse)
    check_fwd(loss, lse, f)
    check_bwd(dh, dw, f, h, w)


@pytest.mark.gpu
def test_xent_strided_rows():
    """Rows of wider matrices whose other columns are NaN, outputs too."""
    print("case: xent strided", flush=True)
    T, V, D, ld = 70, 300, 72, 96
    h, w, t, dloss, _ = inputs(T, V, D, seed=3)

    def wide(x):
        big = torch.full((x.shape[0], ld), float("nan"), dtype=torch.bfloat16, device="cuda")
        big[:, :D] = x.cuda()
        return big[:, :D]

    H, W = wide(h), wide(w)
    loss, lse = U.ufp4_linear_xent_fwd(H, W, t.cuda())
    oh, ow = wide(h), wide(w)
    U.ufp4_linear_xent_bwd(H, W, t.cuda(), lse, dloss.cuda(), out=(oh, ow))
    torch.cuda.synchronize()
    f = formulas(h, w, t, dloss, None)
    check_fwd(loss, lse, f)
    check_bwd(oh, ow, f, h, w)
    assert torch.isnan(oh._base[:, D:]).all() and torch.isnan(ow._base[:, D:]).all()


@pytest.mark.gpu
def test_xent_all_ignored_and_dead_rows():
    """No target at all: losses, dh and dw are exactly 0; a token without any
    gradient may hold NaN and changes nothing else."""
    print("case: xent ignored", flush=True)
    T, V, D = 100, 700, 128
    h, w, t, dloss, _ = inputs(T, V, D, seed=11, ignored=0.0)
    none = torch.full_like(t, -100)
    loss, lse = U.ufp4_linear_xent_fwd(h.cuda(), w.cuda(), none.cuda())
    dh, dw = U.ufp4_linear_xent_bwd(h.cuda(), w.cuda(), none.cuda(), lse, dloss.cuda())
    assert not loss.any() and not dh.any() and not dw.any() and torch.isfinite(lse).all()
    t2 = t.clone()
    t2[40] = -1
    loss, lse = U.ufp4_linear_xent_fwd(h.cuda(), w.cuda(), t2.cuda())
    ref = U.ufp4_linear_xent_bwd(h.cuda(), w.cuda(), t2.cuda(), lse, dloss.cuda())
    bad = h.clone()
    bad[40] = float("nan")
    loss2, lse2 = U.ufp4_linear_xent_fwd(bad.cuda(), w.cuda(), t2.cuda())
    got = U.ufp4_linear_xent_bwd(bad.cuda(), w.cuda(), t2.cuda(), lse2, dloss.cuda())
    assert torch.equal(loss, loss2) and loss2[40] == 0 and torch.isnan(lse2[40])
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert not got[0][40].any()


@pytest.mark.gpu
def test_xent_large_logits_and_infinities():
    """Logits of several hundred keep their statistics; a class at -inf counts
    nothing; a NaN shows."""
    print("case: xent large", flush=True)
    T, V, D = 64, 600, 128
    h, w, t, dloss, _ = inputs(T, V, D, seed=21, size=60.0)
    f = formulas(h, w, t, dloss, None)
    assert f["z"].abs().max() > 300
    loss, lse = U.ufp4_linear_xent_fwd(h.cuda(), w.cuda(), t.cuda())
    check_fwd(loss, lse, f)
    check_bwd(*U.ufp4_linear_xent_bwd(h.cuda(), w.cuda(), t.cuda(), lse, dloss.cuda()), f, h, w)
    h2, w2 = h.clone(), w.clone()
    h2[:, 0], w2[:, 0] = 1.0, 0.0
    w2[300:, 0] = -float("inf")     # the last classes closed, whole tiles of them among these
    t2 = t.clamp(0, 299)
    loss, lse = U.ufp4_linear_xent_fwd(h2.cuda(), w2.cuda(), t2.cuda())
    f = formulas(h2, w2[:300].contiguous(), t2, dloss, None)
    check_fwd(loss, lse, f)
    h2[5, 3] = float("nan")
    loss, lse = U.ufp4_linear_xent_fwd(h2.cuda(), w2.cuda(), t2.cuda())
    assert torch.isnan(lse[5]) and torch.isnan(loss[5]) and int(torch.isnan(lse).sum()) == 1


@pytest.mark.gpu
def test_xent_gradient_against_differences():
    """dh and dw are the derivative of sum dloss loss + dlse lse: central
    differences in 64 bits (own error below 1e-9) along random directions."""
    print("case: xent differences", flush=True)
    T, V, D = 24, 130, 64
    h, w, t, dloss, dlse = inputs(T, V, D, seed=31)
    loss, lse = U.ufp4_linear_xent_fwd(h.cuda(), w.cuda(), t.cuda())
    dh, dw = U.ufp4_linear_xent_bwd(h.cuda(), w.cuda(), t.cuda(), lse, dloss.cuda(), dlse.cuda())
    H, W = h.double(), w.double()
    live = (t >= 0) & (t < V)
    at = torch.where(live, t, torch.zeros_like(t))[:, None]

    def value(H, W):
        z = H @ W.t()
        s = torch.logsumexp(z, 1)
        return (torch.where(live, s - z.gather(1, at)[:, 0], torch.zeros_like(s)) * dloss.double()
                + s * dlse.double()).sum()

    g = torch.Generator().manual_seed(1)
    f = formulas(h, w, t, dloss, dlse)
    for _ in range(4):
        u, v = torch.randn(T, D, generator=g).double(), torch.randn(V, D, generator=g).double()
        e = 1e-6
        for got, du, dv, want in ((dh, u, 0, f["dh"]), (dw, 0, v, f["dw"])):
            diff = (value(H + e * du, W + e * dv) - value(H - e * du, W - e * dv)) / (2 * e)
            x = u if got is dh else v
            # independent roundings of 2 steps each: 3 2^-8 of the norm, at 4 deviations
            tol = 4 * 3 * BF16 * want.norm() + 1e-8
            assert abs((got.double().cpu() * x).sum() - diff) <= tol
            assert abs((want * x).sum() - diff) <= 1e-8 + 1e-6 * want.norm()


@pytest.mark.gpu
def test_xent_repeats_on_a_side_stream_and_in_a_graph():
    print("case: xent stream and graph", flush=True)
    T, V, D = 300, 3000, 256
    h, w, t, dloss, dlse = (x.cuda() for x in inputs(T, V, D, seed=41))
    loss, lse = U.ufp4_linear_xent_fwd(h, w, t)
    ref = (loss, lse, *U.ufp4_linear_xent_bwd(h, w, t, lse, dloss, dlse))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        l2, e2 = U.ufp4_linear_xent_fwd(h, w, t)
        got = (l2, e2, *U.ufp4_linear_xent_bwd(h, w, t, e2, dloss, dlse))
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(x, y) for x, y in zip(got, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        l3, e3 = U.ufp4_linear_xent_fwd(h, w, t)
        got = (l3, e3, *U.ufp4_linear_xent_bwd(h, w, t, e3, dloss, dlse))
    for _ in range(3):
        for x in got:
            x.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        U.ufp4_linear_xent_fwd(w, h, torch.zeros(V, dtype=torch.int64, device="cuda"))
        assert all(torch.equal(x, y) for x, y in zip(got, ref))


@pytest.mark.gpu
def test_xent_no_tokens():
    print("case: xent empty", flush=True)
    h = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.randn(100, 64, device="cuda").to(torch.bfloat16)
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = U.ufp4_linear_xent_fwd(h, w, t)
    dh, dw = U.ufp4_linear_xent_bwd(h, w, t, lse, torch.empty(0, device="cuda"))
    assert loss.shape == (0,) and dh.shape == (0, 64) and dw.shape == (100, 64) and not dw.any()


# --- refusals (no GPU) -------------------------------------------------------
FAKE = 0x10000


def raw_fwd(lib, **kw):
    a = dict(h=FAKE, ldh=64, w=FAKE, ldw=64, t=FAKE, T=4, V=100, D=64, loss=FAKE, lse=FAKE, ws=FAKE,
             n=1 << 40)
    a.update(kw)
    return lib.ufp4_linear_xent_fwd(a["h"], a["ldh"], a["w"], a["ldw"], a["t"], a["T"], a["V"],
                                    a["D"], a["loss"], a["lse"], a["ws"], a["n"], None)


def raw_bwd(lib, **kw):
    a = dict(h=FAKE, ldh=64, w=FAKE, ldw=64, t=FAKE, T=4, V=100, D=64, lse=FAKE, dl=FAKE, de=0,
             dh=FAKE, lddh=64, dw=FAKE, lddw=64, ws=FAKE, n=1 << 40)
    a.update(kw)
    return lib.ufp4_linear_xent_bwd(a["h"], a["ldh"], a["w"], a["ldw"], a["t"], a["T"], a["V"],
                                    a["D"], a["lse"], a["dl"], a["de"], a["dh"], a["lddh"], a["dw"],
                                    a["lddw"], a["ws"], a["n"], None)


def test_xent_abi_refusals():
    lib = U.lib_handle()
    bad, shape, no = U.UFP4_ERR_INVALID_ARG, U.UFP4_ERR_SHAPE, U.UFP4_ERR_UNSUPPORTED
    both = [(dict(T=-1), bad), (dict(V=0), bad), (dict(D=0), bad), (dict(D=60), shape),
            (dict(T=(1 << 21) + 1), no), (dict(V=(1 << 30) + 1), no),
            (dict(D=(1 << 20) + 8), no), (dict(ldh=56), bad), (dict(ldw=68), bad),
            (dict(ldh=(1 << 20) + 8), no), (dict(h=0), bad), (dict(w=FAKE + 8), bad),
            (dict(t=0), bad), (dict(t=FAKE + 4), bad), (dict(lse=0), bad), (dict(lse=FAKE + 2), bad),
            (dict(ws=0), bad), (dict(ws=FAKE + 64), bad), (dict(n=100), bad)]
    for kw, want in both + [(dict(loss=0), bad), (dict(loss=FAKE + 2), bad)]:
        assert raw_fwd(lib, **kw) == want, kw
    for kw, want in both + [(dict(dl=0), bad), (dict(dl=FAKE + 1), bad), (dict(de=FAKE + 1), bad),
                            (dict(dh=0), bad), (dict(dw=0), bad), (dict(lddh=56), bad),
                            (dict(lddw=60), bad), (dict(dw=FAKE + 8), bad),
                            (dict(T=0, dw=0), bad)]:
        assert raw_bwd(lib, **kw) == want, kw
    assert raw_fwd(lib, T=0, h=0, t=0, loss=0, lse=0, ws=0, n=0) == U.UFP4_OK
    size = U.ufp4_linear_xent_workspace_bytes
    assert size(0, 100, 64) == 0 and size(4, 100, 60) == 0 and size(4, 0, 64, True) == 0
    need = size(4, 100, 64, True)
    assert need > 0 and raw_bwd(lib, n=need - 1) == bad
    # one piece of G and its transpose at most, whatever the vocabulary
    assert size(8192, 1 << 20, 64, True) < 2 * 2 * (1 << 26) + (1 << 24) + 8192 * 64 * 16


def test_xent_binding_refusals():
    h, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(9, 64, dtype=torch.bfloat16)
    t, f = torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    with pytest.raises(ValueError, match="GPU"):
        U.ufp4_linear_xent_fwd(h, w, t)
    with pytest.raises(ValueError, match="GPU"):
        U.ufp4_linear_xent_bwd(h, w, t, f, f)
    with pytest.raises(ValueError, match="h must have dtype"):
        U.ufp4_linear_xent_fwd(h.float(), w, t)
    with pytest.raises(ValueError, match="columns"):
        U.ufp4_linear_xent_fwd(h, w[:, :56], t)
    with pytest.raises(ValueError, match="targets"):
        U.ufp4_linear_xent_fwd(h, w, t.int())
    with pytest.raises(ValueError, match="targets"):
        U.ufp4_linear_xent_fwd(h, w, t[:3])
    with pytest.raises(ValueError, match="unit column stride"):
        U.ufp4_linear_xent_fwd(torch.zeros(64, 4, dtype=torch.bfloat16).t(), w, t)
    with pytest.raises(ValueError, match="dloss"):
        U.ufp4_linear_xent_bwd(h, w, t, f, f.double())
    with pytest.raises(ValueError, match="dlse"):
        U.ufp4_linear_xent_bwd(h, w, t, f, f, dlse=f[:2])
    with pytest.raises(ValueError, match="dw has shape"):
        U.ufp4_linear_xent_bwd(h, w, t, f, f, out=(h, w[:8]))


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,D", [(5, 270001, 16), (40, 262200, 8), (70, 262401, 8)])
def test_xent_few_tokens_in_pieces(T, V, D):
    """Vocabularies of several pieces with each of the tile shapes of few tokens."""
    print("case: xent few tokens in pieces", T, V, D, flush=True)
    h, w, t, dloss, dlse = inputs(T, V, D, seed=T, device="cuda")
    loss, lse = U.ufp4_linear_xent_fwd(h, w, t)
    dh, dw = U.ufp4_linear_xent_bwd(h, w, t, lse, dloss, dlse)
    torch.cuda.synchronize()
    f = formulas(h, w, t, dloss, dlse)
    check_fwd(loss, lse, f)
    check_bwd(dh, dw, f, h, w)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [9, 50, 300])
def test_xent_gradients_with_classes_at_minus_infinity(T):
    """Classes whose logits fall below fp32's range (-2^200) have no probability:
    their rows of dw are exactly 0 and the other gradients are those of the open
    classes alone."""
    print("case: xent closed classes", T, flush=True)
    V, D, open_ = 700, 64, 300
    h, w, t, dloss, dlse = inputs(T, V, D, seed=51)
    t = torch.where(t >= 0, t.clamp(max=open_ - 1), t)
    h[:, 0], w[:, 0] = 2.0 ** 100, 0.0
    w[open_:, 0] = -2.0 ** 100
    g = [x.cuda() for x in (h, w, t, dloss, dlse)]
    loss, lse = U.ufp4_linear_xent_fwd(*g[:3])
    dh, dw = U.ufp4_linear_xent_bwd(*g[:3], lse, g[3], dlse=g[4])
    torch.cuda.synchronize()
    few = w[:open_].contiguous()
    f = formulas(h, few, t, dloss, dlse)
    check_fwd(loss, lse, f)
    check_bwd(dh, dw[:open_], f, h, few)
    assert not dw[open_:].any()
