"""The language-model operators that stand around the 4-bit GEMMs, as cases to be timed and compared.

Three operators, each in its plain form (elementary torch operations in 32 bits) and, where
`own` is true, through the package's entry points:

  xent  softmax cross entropy of a linear head over a large vocabulary, without keeping the
        logits, and its gradients (ufp4_linear_xent_fwd, ufp4_linear_xent_bwd);
  glu   an expert's gated activation, saving its inputs as MXFP8 checkpoints, and its backward
        pass from them (ufp4_glu_fwd, ufp4_glu_bwd);
  moe   a whole mixture-of-experts layer for a few tokens on 4-bit weights (ufp4_moe_tokens).
"""
import math

import torch

own = False

E1M2, INT4, E2M1 = 0, 1, 2
LEVELS = {
    E1M2: [0.25 * k for k in range(8)] + [-0.25 * k for k in range(8)],
    INT4: [0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1],
    E2M1: [0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6],
}


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the log-probabilities of a handful of tokens (a request that is scored): reading W is all there is
        dict(name="xent score 7 tokens", op="xent", T=7, V=32003, D=2048, grad=False, ignored=0.0),
        # perplexity of held-out text: forward only, vocabulary that no tile divides, part of the text not scored
        dict(name="xent eval 4099 tokens", op="xent", T=4099, V=100003, D=2048, grad=False, ignored=0.3),
        # a small micro-batch of fine-tuning: prompts carry no loss
        dict(name="xent step 509 tokens", op="xent", T=509, V=32003, D=4096, grad=True, ignored=0.5),
        # a training micro-batch at the 16-expert layer's width
        dict(name="xent step 4096 tokens", op="xent", T=4096, V=65536, D=5120, grad=True, ignored=0.02),
        # the largest: a long-sequence batch over a large vocabulary
        dict(name="xent step 8192 tokens", op="xent", T=8192, V=131072, D=4096, grad=True, ignored=0.02),
        # generation: the activations of one token's six experts, nothing kept for a backward pass
        dict(name="glu serve 6 rows", op="glu", rows=6, F=1408, act="silu", dtype="bf16", grad=False, scaled=True, again=False),
        # an odd micro-batch in bf16 with the other activation; rows end inside a 32-element block
        dict(name="glu step odd", op="glu", rows=4093, F=1411, act="gelu", dtype="bf16", grad=True, scaled=False, again=True),
        # the 64-expert layer's token rows, straight from the fp32 GEMM outputs, expert weights folded in
        dict(name="glu step 64 experts", op="glu", rows=98304, F=1408, act="silu", dtype="fp32", grad=True, scaled=True, again=False),
        # the 16-expert share: every token eight times
        dict(name="glu step 16 experts", op="glu", rows=262144, F=1536, act="silu", dtype="fp32", grad=True, scaled=True, again=True),
        # one token generated through the 64-expert layer
        dict(name="moe 1 token", op="moe", T=1, E=64, H=2048, F=1408, k=6, grid=INT4, scale="fp32", block=32, n=32, act="silu", renorm=True, masked=False),
        # a small decoding batch on the 16-expert share
        dict(name="moe 16 tokens", op="moe", T=16, E=16, H=5120, F=1536, k=8, grid=INT4, scale="fp32", block=16, n=128, act="silu", renorm=True, masked=False),
        # a full decoding batch, MX blocks, some experts closed to some tokens
        dict(name="moe 61 tokens", op="moe", T=61, E=64, H=2048, F=1408, k=6, grid=E2M1, scale="pow2", block=32, n=32, act="silu", renorm=False, masked=True),
    ]


def _between(rng, low, high):
    """A whole number between the two, evenly over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["xent", "glu", "moe"])
    if op == "xent":
        while True:
            c = dict(op="xent", T=_between(rng, 1, 8192), V=_between(rng, 1000, 131072), D=8 * _between(rng, 32, 640),
                     grad=rng.random() < 0.6, ignored=rng.choice([0.0, 0.02, 0.5, 1.0]))
            if c["T"] * c["V"] * c["D"] <= 8192 * 131072 * 4096 and 3072 not in c.values():
                return c
    if op == "glu":
        while True:
            c = dict(op="glu", rows=_between(rng, 1, 262144), F=rng.choice([rng.randint(33, 1536), 8 * rng.randint(5, 192), 1408, 1536]),
                     act=rng.choice(["silu", "gelu"]), dtype=rng.choice(["bf16", "fp32"]), grad=rng.random() < 0.7,
                     scaled=rng.random() < 0.5, again=rng.random() < 0.5)
            if 3072 not in c.values():
                return c
    while True:
        block, pow2 = rng.choice([16, 32]), rng.random() < 0.4
        n = rng.choice([1, 16, 32, 64, 128])
        E = rng.choice([8, 16, 32, 64])
        c = dict(op="moe", T=_between(rng, 1, 64), E=E, H=128 * rng.randint(4, 40), F=max(n, 32) * rng.randint(2, 1536 // max(n, 32)),
                 k=rng.randint(1, min(8, E)), grid=rng.choice([E1M2, INT4, E2M1]), scale="pow2" if pow2 else "fp32", block=32 if pow2 else block,
                 n=n, act=rng.choice(["silu", "gelu"]), renorm=rng.random() < 0.5, masked=rng.random() < 0.3)
        if c["E"] * c["H"] * c["F"] <= 64 * 2048 * 1536 and 3072 not in c.values():
            return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _weights(P, K, case, gen, dev):
    """Codes and scales of a quantized weight [P, K]: bell-shaped values whose blocks fill the grid."""
    grid, block = case["grid"], case["block"]
    x = torch.randn(P, K, generator=gen, device=dev)
    if grid == INT4:
        c = (x * 3.0).round().clamp(-7, 7).to(torch.int32) & 15
    elif grid == E1M2:
        c = (x.abs() * 3.0).round().clamp(0, 7).to(torch.int32)
        c = c + 8 * ((x < 0) & (c > 0))
    else:
        c = (x.abs() * 2.5).clamp(0, 7).to(torch.int32)
        c = c + 8 * ((x < 0) & (c > 0))
    c = c.view(P, K // 2, 2)
    codes = (c[..., 0] | (c[..., 1] << 4)).to(torch.uint8)
    top = {E1M2: 1.75, INT4: 7.0, E2M1: 6.0}[grid]
    size = (0.5 + torch.rand(P, K // block, generator=gen, device=dev)) * (2.5 / top / math.sqrt(K))
    if case["scale"] == "pow2":
        return codes, (torch.log2(size).round() + 127).to(torch.uint8)
    return codes, size


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * seed + 17)
    s = dict(case)
    if case["op"] == "xent":
        T, V, D = case["T"], case["V"], case["D"]
        w = torch.randn(V, D, generator=g, device=dev, dtype=torch.float32).mul_(1.0 / math.sqrt(D))
        # frequent tokens come first; a trained head scores the right one well above the rest
        t = (torch.rand(T, generator=g, device=dev).double() ** 3 * V).long().clamp_(0, V - 1)
        h = torch.randn(T, D, generator=g, device=dev)
        sure = torch.rand(T, 1, generator=g, device=dev) * 8
        h = h + w[t] * sure
        s["h"], s["w"] = h.to(torch.bfloat16), w.to(torch.bfloat16)
        out = torch.rand(T, generator=g, device=dev) < case["ignored"]
        s["targets"] = torch.where(out, torch.full_like(t, -100), t)
        kept = T * (1.0 - case["ignored"])
        s["dloss"] = torch.full((T,), 1.0 / max(1.0, kept), device=dev)
    elif case["op"] == "glu":
        R, F = case["rows"], case["F"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["gate"] = torch.randn(R, F, generator=g, device=dev).mul_(1.5).to(dt)
        s["up"] = torch.randn(R, F, generator=g, device=dev).to(dt)
        s["dh"] = torch.randn(R, F, generator=g, device=dev).mul_(1e-3).to(dt) if case["grad"] else None
        s["row"] = torch.rand(R, generator=g, device=dev) if case["scaled"] else None
    else:
        T, E, H, F, n = case["T"], case["E"], case["H"], case["F"], case["n"]
        s["x"] = torch.randn(T, H, generator=g, device=dev).to(torch.bfloat16)
        s["logits"] = torch.randn(T, E, generator=g, device=dev) * 1.5
        if case["masked"]:
            closed = torch.rand(T, E, generator=g, device=dev) < 0.6
            closed[T // 2] = True  # a slot of the batch that holds no token
            s["logits"] = torch.where(closed, torch.full_like(s["logits"], -math.inf), s["logits"])
        s["sign_seed"] = 4101 + seed
        s["wg"] = _weights(E * F, H, case, g, dev)
        s["wu"] = _weights(E * F, H, case, g, dev)
        s["wd"] = _weights(E * H, F, case, g, dev)
        s["levels"] = torch.tensor(LEVELS[case["grid"]], dtype=torch.float32, device=dev)
        # the random signs that a seed stands for: the first n bits of one Philox4x32-10 block
        c, key = [0, 0, 0xFFFFFFFF, 0], [s["sign_seed"], 0]
        for _ in range(10):
            a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
            c = [(b >> 32) ^ c[1] ^ key[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ key[1], a & 0xFFFFFFFF]
            key = [(key[0] + 0x9E3779B9) & 0xFFFFFFFF, (key[1] + 0xBB67AE85) & 0xFFFFFFFF]
        signs = [1.0 - 2.0 * ((c[i // 32] >> (i % 32)) & 1) for i in range(n)] if n > 1 else [1.0]
        m = torch.ones(1, 1, dtype=torch.float64)
        while m.shape[0] < n:
            m = torch.cat([torch.cat([m, m], 1), torch.cat([m, -m], 1)], 0)
        s["turn"] = (torch.tensor(signs, dtype=torch.float64)[:, None] * m).to(dev)  # S H, without its 1 / sqrt(n)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _plain_xent(s):
    h, w, t = s["h"].float(), s["w"].float(), s["targets"]
    z = h @ w.t()
    top = z.amax(1, keepdim=True)
    lse = (torch.exp(z - top).sum(1, keepdim=True).log() + top).squeeze(1)
    live = (t >= 0) & (t < w.shape[0])
    at = torch.where(live, t, torch.zeros_like(t))[:, None]
    loss = torch.where(live, lse - z.gather(1, at).squeeze(1), torch.zeros_like(lse))
    if not s["grad"]:
        return dict(loss=loss, lse=lse)
    scale = torch.where(live, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
    G = torch.exp(z.sub_(lse[:, None])).mul_(scale)
    G.scatter_add_(1, at, -scale)
    return dict(loss=loss, lse=lse, dh=(G @ w).to(torch.bfloat16), dw=(G.t() @ h).to(torch.bfloat16))


def _plain_act(g, act):
    """The activation and its derivative."""
    if act == "silu":
        q = 1.0 / (1.0 + torch.exp(-g))
        return g * q, q * (1.0 + g * (1.0 - q))
    c, b = math.sqrt(2.0 / math.pi), 0.044715
    t = torch.tanh(c * (g + b * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * (c * (1.0 + 3.0 * b * g * g))


def _plain_eight_bits(x):
    """x as 1 x 32 blocks of E4M3 values under the least power of two that keeps the block within +-448."""
    R, F = x.shape
    wide = -(-F // 32) * 32
    b = torch.nn.functional.pad(x, (0, wide - F)).view(R, wide // 32, 32)
    m, e = torch.frexp(b.abs().amax(2, keepdim=True))  # amax = m 2^e, 1/2 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(-127, 127)
    e = torch.where(m == 0, torch.full_like(e, -127), e)
    q = torch.ldexp(b, -e).to(torch.float8_e4m3fn).float()
    return torch.ldexp(q, e).view(R, wide)[:, :F]


def _plain_glu(s):
    g, u = s["gate"].float(), s["up"].float()
    r = s["row"][:, None] if s["scaled"] else 1.0
    a, _ = _plain_act(g, s["act"])
    out = dict(h=(a * u * r).to(torch.bfloat16))
    if not s["grad"]:
        return out
    g, u, dh = _plain_eight_bits(g), _plain_eight_bits(u), s["dh"].float()
    a, da = _plain_act(g, s["act"])
    out["dgate"] = (dh * u * da * r).to(torch.bfloat16)
    out["dup"] = (dh * a * r).to(torch.bfloat16)
    if s["scaled"]:
        out["drow"] = (dh * a * u).sum(1)
    if s["again"]:
        out["again"] = (a * u * r).to(torch.bfloat16)
    return out


def _plain_dequant(w, s, slots):
    """The weights of the experts in `slots`, one after another."""
    codes, scales = (x.view(s["E"], -1, x.shape[1])[slots].flatten(0, 1) for x in w)
    c = torch.stack([codes & 15, codes >> 4], 2).view(codes.shape[0], -1)
    v = torch.take(s["levels"], c.long()).view(codes.shape[0], -1, s["block"])
    size = torch.exp2(scales.float() - 127.0) if s["scale"] == "pow2" else scales
    return (v * size[..., None]).view(codes.shape[0], -1)


def _plain_rotate(x, s):
    n = s["n"]
    return ((x.reshape(-1, n) @ s["turn"].float()) * (1.0 / math.sqrt(n))).view(x.shape)


def _plain_moe(s):
    T, E, H, F = s["T"], s["E"], s["H"], s["F"]
    z = s["logits"]
    z, at = torch.sort(z, dim=1, descending=True, stable=True)
    p = torch.where(z > -math.inf, torch.exp(z - z[:, :1]), torch.zeros_like(z))
    p, whole = p[:, :s["k"]], p.sum(1, keepdim=True)
    whole = p.sum(1, keepdim=True) if s["renorm"] else whole
    p = torch.where(whole > 0, p / whole, torch.zeros_like(p))
    at = at[:, :s["k"]]
    if T * s["k"] < E:  # every token's choices one after another; else all experts
        slots, to = at.reshape(-1), torch.arange(T * s["k"], device=z.device).view(T, -1)
    else:
        slots, to = torch.arange(E, device=z.device), at
    S = slots.shape[0]
    share = torch.zeros(T, S, device=z.device).scatter_(1, to, p)
    x = _plain_rotate(s["x"].float(), s)
    gate, up = x @ _plain_dequant(s["wg"], s, slots).t(), x @ _plain_dequant(s["wu"], s, slots).t()
    h = (_plain_act(gate, s["act"])[0] * up).view(T, S, F) * share[..., None]
    down = _plain_dequant(s["wd"], s, slots).view(S, H, F).permute(0, 2, 1).reshape(S * F, H)
    return dict(y=(_plain_rotate(h, s).view(T, S * F) @ down).to(torch.bfloat16))


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    s = state
    if not own:
        return {"xent": _plain_xent, "glu": _plain_glu, "moe": _plain_moe}[s["op"]](s)
    import rht_bit_block_amd as U
    if s["op"] == "xent":
        loss, lse = U.ufp4_linear_xent_fwd(s["h"], s["w"], s["targets"])
        if not s["grad"]:
            return dict(loss=loss, lse=lse)
        dh, dw = U.ufp4_linear_xent_bwd(s["h"], s["w"], s["targets"], lse, s["dloss"])
        return dict(loss=loss, lse=lse, dh=dh, dw=dw)
    act = U.UFP4_ACT_SILU if s["act"] == "silu" else U.UFP4_ACT_GELU
    if s["op"] == "glu":
        h, kept = U.ufp4_glu_fwd(s["gate"], s["up"], act=act, row_scale=s["row"], checkpoint=s["grad"])
        out = dict(h=h)
        if s["grad"]:
            out["dgate"], out["dup"], drow, again = U.ufp4_glu_bwd(kept, s["dh"], row_scale=s["row"], recompute=s["again"])
            if s["scaled"]:
                out["drow"] = drow
            if s["again"]:
                out["again"] = again
        return out
    cfg = U.make_cfg(s["grid"], U.UFP4_RTNE, U.UFP4_SCALE_POW2 if s["scale"] == "pow2" else U.UFP4_SCALE_F32, 1, s["block"], s["n"],
                     sign_seed=s["sign_seed"])
    E, H, F = s["E"], s["H"], s["F"]
    wg, wu = U.QTensor(*s["wg"], E * F, H, cfg), U.QTensor(*s["wu"], E * F, H, cfg)
    wd = U.QTensor(*s["wd"], E * H, F, cfg)
    return dict(y=U.ufp4_moe_tokens(s["x"], s["logits"], wg, wu, wd, s["k"], renorm=s["renorm"], act=act))


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "xent":
        T, V, D = case["T"], case["V"], case["D"]
        read = 2 * (T + V) * D + 8 * T
        if not case["grad"]:
            return {"bytes": read + 8 * T, "flops": 2.0 * T * V * D}
        # three products: the logits, dh and dw (the logits a second time are this path's own price)
        return {"bytes": read + 12 * T + 2 * (T + V) * D, "flops": 6.0 * T * V * D}
    if case["op"] == "glu":
        n, size = case["rows"] * case["F"], 2 if case["dtype"] == "bf16" else 4
        row = 4 * case["rows"] if case["scaled"] else 0
        if not case["grad"]:
            return {"bytes": n * (2 * size + 2) + row, "flops": 8.0 * n}
        # h, dgate, dup (and h again) written; the checkpoints, 33 bytes for 32 values, written and read
        again = 2 if case["again"] else 0
        return {"bytes": n * (3 * size + 6 + again + 4 * 33 / 32) + 3 * row, "flops": 30.0 * n}
    T, E, H, F, k = case["T"], case["E"], case["H"], case["F"], case["k"]
    met = E * (1.0 - (1.0 - k / E) ** T)  # experts that some token of the batch goes to
    weight = 0.5 + (1.0 if case["scale"] == "pow2" else 4.0) / case["block"]
    return {"bytes": met * 3 * H * F * weight + T * (4 * H + 4 * E), "flops": 6.0 * T * k * H * F}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_act(g, act):
    if act == "silu":
        sig = torch.sigmoid(g)
        return g * sig, sig + g * sig * torch.sigmoid(-g)
    k = math.sqrt(8.0 / math.pi)  # (1 + tanh x) / 2 = sigmoid(2 x)
    arg, darg = k * (g + 0.044715 * g ** 3), k * (1 + 0.134145 * g ** 2)
    sig = torch.sigmoid(arg)
    return g * sig, sig + g * darg * sig * torch.sigmoid(-arg)


def _exact_eight_bits(x):
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], 32):
        b = x[:, c:c + 32]
        m = b.abs().amax(1, keepdim=True)
        e = torch.full_like(m, -127.0)
        ok = m > 0
        e[ok] = torch.ceil(torch.log2(m[ok] / 448.0) - 1e-9)
        e = torch.where(m > 448.0 * torch.exp2(e), e + 1, e)
        e = torch.where(ok & (m <= 448.0 * torch.exp2(e - 1)), e - 1, e).clamp(-127, 127)
        v = b * torch.exp2(-e)
        # spacing 2^(floor(log2 |v|) - 3), and 2^-9 below 2^-6
        ex = torch.frexp(v)[1].double() - 1
        step = torch.exp2(ex.clamp(min=-6) - 3)
        out[:, c:c + 32] = torch.round(v / step) * step * torch.exp2(e)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "xent":
        h, w, t = s["h"].double(), s["w"].double(), s["targets"]
        z = torch.matmul(h, w.t())
        lse = torch.logsumexp(z, 1)
        rows = torch.nonzero((t >= 0) & (t < w.shape[0])).squeeze(1)
        loss = torch.zeros_like(lse)
        loss[rows] = lse[rows] - z[rows, t[rows]]
        if not case["grad"]:
            return dict(loss=loss, lse=lse)
        z = torch.exp(z - lse[:, None])
        z[rows, t[rows]] -= 1.0
        weight = torch.zeros_like(lse)
        weight[rows] = s["dloss"].double()[rows]
        z *= weight[:, None]
        return dict(loss=loss, lse=lse, dh=torch.matmul(z, w), dw=torch.matmul(z.t(), h))
    if case["op"] == "glu":
        g, u = s["gate"].double(), s["up"].double()
        r = s["row"].double()[:, None] if case["scaled"] else torch.ones(1, 1, dtype=torch.float64, device=g.device)
        out = dict(h=r * u * _exact_act(g, case["act"])[0])
        if case["grad"]:
            g, u, dh = _exact_eight_bits(g), _exact_eight_bits(u), s["dh"].double()
            a, da = _exact_act(g, case["act"])
            out["dgate"], out["dup"] = r * dh * (u * da), r * dh * a
            if case["scaled"]:
                out["drow"] = torch.sum(dh * a * u, 1)
            if case["again"]:
                out["again"] = r * a * u
        return out
    T, E, H, F, n, k = (case[x] for x in ("T", "E", "H", "F", "n", "k"))

    def weight(w, e, P):
        codes, scales = w[0][e * P:(e + 1) * P], w[1][e * P:(e + 1) * P]
        v = torch.empty(P, codes.shape[1] * 2, dtype=torch.float64, device=codes.device)
        lv = s["levels"].double()
        v[:, 0::2], v[:, 1::2] = lv[(codes & 15).long()], lv[(codes >> 4).long()]
        size = 2.0 ** (scales.double() - 127) if case["scale"] == "pow2" else scales.double()
        return v * size.repeat_interleave(case["block"], 1)

    def rotate(x):
        return (x.reshape(x.shape[0], -1, n) @ s["turn"] / math.sqrt(n)).reshape(x.shape)

    x, z = rotate(s["x"].double()), s["logits"].double().cpu()
    pairs = [[] for _ in range(E)]
    for t in range(T):
        row = z[t].tolist()
        chosen = [e for e in sorted(range(E), key=lambda e: (-row[e], e))[:k] if row[e] > -math.inf]
        over = chosen if case["renorm"] else [e for e in range(E) if row[e] > -math.inf]
        top = max((row[e] for e in over), default=0.0)
        total = sum(math.exp(row[e] - top) for e in over)
        for e in chosen:
            pairs[e].append((t, math.exp(row[e] - top) / total))
    y = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    for e, p in enumerate(pairs):
        if not p:
            continue
        ts = torch.tensor([t for t, _ in p], device=x.device)
        ws = torch.tensor([v for _, v in p], dtype=torch.float64, device=x.device)
        a = _exact_act(x[ts] @ weight(s["wg"], e, F).t(), case["act"])[0] * (x[ts] @ weight(s["wu"], e, F).t())
        y.index_add_(0, ts, (rotate(a) @ weight(s["wd"], e, H).t()) * ws[:, None])
    return dict(y=y)
