"""Attention around the 4-bit GEMMs, as cases to be timed and compared.

Three groups of calls, each in its plain form (elementary torch operations in 32 bits) and, where
`own` is true, through the package's entry points:

  attn   causal attention over packed sequences with grouped heads, and its gradients
         (ufp4_attn_fwd, ufp4_attn_bwd);
  kv     keys and values quantized into the pages of a 4-bit cache as they are written, and read
         back (ufp4_kv_write, ufp4_kv_read);
  cache  attention of a few new tokens over a cache held in 4 bits (ufp4_kv_attn).
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
TOP = {E1M2: 1.75, INT4: 7.0, E2M1: 6.0}


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a short request's prompt in a server that is otherwise idle: the launch is all there is
        dict(name="attn 19 tokens", op="attn", lens="19", heads=16, kv=4, D=128, grad=False),
        # prompts of several users in one batch, one of them a single token, one slot empty, at the 16-expert layer's width
        dict(name="attn 7 prompts", op="attn", lens="1237,1,2048,0,333,1000,384", heads=40, kv=8, D=128, grad=False),
        # a long document as one prompt, every head on one key head
        dict(name="attn 32768 tokens", op="attn", lens="32768", heads=8, kv=1, D=128, grad=False),
        # a small fine-tuning batch of odd texts, head width that no tile has, no shared heads
        dict(name="attn step odd", op="attn", lens="701,1300,17,983", heads=20, kv=20, D=80, grad=True),
        # a training micro-batch at the 16-expert layer's width
        dict(name="attn step 4 x 4096", op="attn", lens="4096,4096,4096,4096", heads=40, kv=8, D=128, grad=True),
        # a decoding batch writes a token each
        dict(name="kv 32 x 1 token", op="kv", lens=",".join("%d" % (100 + 37 * i) for i in range(32)), new=",".join(["1"] * 32), kv=8, D=128, page=64,
             grid=INT4, scale="fp32", block=16, n=128),
        # odd prompts into small pages, behind what the sequences hold already
        dict(name="kv odd", op="kv", lens="1000,3,77,2049", new="901,3,1,1496", kv=5, D=96, page=16, grid=E1M2, scale="fp32", block=32, n=32),
        # a long prompt in MX blocks
        dict(name="kv 16381 tokens", op="kv", lens="16381", new="16381", kv=8, D=128, page=128, grid=E2M1, scale="pow2", block=32, n=32),
        # one user's next token after a short conversation
        dict(name="cache 1 of 1000", op="cache", lens="1000", new="1", heads=16, kv=4, D=128, page=64, grid=INT4, scale="fp32", block=32, n=32),
        # draft tokens that are checked five at a time, every key head under five heads
        dict(name="cache 16 x 5 tokens", op="cache", lens=",".join("%d" % (4001 + 251 * i) for i in range(16)), new=",".join(["5"] * 16), heads=40, kv=8, D=128,
             page=64, grid=INT4, scale="fp32", block=16, n=128),
        # a full decoding batch of conversations of every length
        dict(name="cache 64 ragged", op="cache", lens=",".join("%d" % (1 + (i * i * 16383) // 3969) for i in range(64)), new=",".join(["1"] * 64), heads=40,
             kv=8, D=128, page=64, grid=E2M1, scale="pow2", block=32, n=32),
        # four long documents are asked about
        dict(name="cache 4 x 131072", op="cache", lens="131072,131072,131072,131072", new="1,1,1,1", heads=32, kv=8, D=128, page=128, grid=E1M2, scale="fp32",
             block=32, n=64),
    ]


def _between(rng, low, high):
    """A whole number between the two, evenly over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _text(values):
    return ",".join("%d" % v for v in values)


def draw(rng):
    op = rng.choice(["attn", "kv", "cache"])
    kv = rng.choice([1, 2, 4, 5, 8])
    if op == "attn":
        group = rng.choice([1, 2, 4, 5, 8])
        c = dict(op="attn", heads=kv * group, kv=kv, D=rng.choice([64, 128, 8 * rng.randint(4, 16)]), grad=rng.random() < 0.5)
        lens = [_between(rng, 1, 4096) for _ in range(rng.randint(1, 7))]
        if rng.random() < 0.3:
            lens[rng.randrange(len(lens))] = rng.randint(0, 1)
        if rng.random() < 0.15:
            lens = [_between(rng, 4096, 16384)]
        while sum(n * n for n in lens) * c["heads"] > 4 * 4096 * 4096 * 40:
            lens = [n // 2 for n in lens]
        return dict(c, lens=_text(lens))
    # the quantizer takes whole blocks and whole rotations along a head
    n = rng.choice([1, 16, 32, 64, 128])
    scale, block = rng.choice([("fp32", 16), ("fp32", 32), ("pow2", 32)])
    D = rng.choice([d for d in (32, 64, 80, 96, 112, 128) if d % n == 0 and d % block == 0] + ([128] if n < 64 else []))
    c = dict(op=op, kv=kv, D=D, page=2 ** rng.randint(4, 8), grid=rng.choice([E1M2, INT4, E2M1]), scale=scale, block=block, n=n)
    B = _between(rng, 1, 64)
    if op == "kv":
        new = [_between(rng, 1, 2048) if rng.random() < 0.5 else 1 for _ in range(B)]
        while sum(new) > 16384:
            new = [max(1, x // 2) for x in new]
        return dict(c, new=_text(new), lens=_text([x + rng.choice([0, rng.randint(1, 500)]) for x in new]))
    most = rng.choice([1, 1, 1, 4, 16])
    new = [rng.randint(1, most) for _ in range(B)]
    lens = [max(x, _between(rng, 1, 65536 if B <= 4 else 8192)) for x in new]
    while sum(lens) * kv > 4 * 131072 * 8 or max(lens) * B > 64 * 16384:
        lens = [max(x, n // 2) for x, n in zip(new, lens)]
    return dict(c, heads=kv * rng.choice([1, 4, 5, 8]), new=_text(new), lens=_text(lens))


def _numbers(text):
    return [int(x) for x in text.split(",")]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _signs(seed, n):
    """The random signs that a seed stands for: the first n bits of one Philox4x32-10 block."""
    c, key = [0, 0, 0xFFFFFFFF, 0], [seed, 0]
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ key[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ key[1], a & 0xFFFFFFFF]
        key = [(key[0] + 0x9E3779B9) & 0xFFFFFFFF, (key[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return [1.0 - 2.0 * ((c[i // 32] >> (i % 32)) & 1) for i in range(n)] if n > 1 else [1.0]


def _rows(T, heads, D, gen, dev, spread):
    """Activations of T tokens: some heads and tokens are louder than others, a few channels stand out."""
    x = torch.randn(T, heads, D, generator=gen, device=dev)
    x = x * (0.5 + spread * torch.rand(T, heads, 1, generator=gen, device=dev))
    loud = 1.0 + 3.0 * (torch.rand(1, heads, D, generator=gen, device=dev) > 0.97).float()
    return (x * loud).to(torch.bfloat16)


def _pages(case, pages, gen, dev):
    """Codes and scales of a cache that is in use: bell-shaped values whose blocks fill the grid."""
    grid, block, shape = case["grid"], case["block"], (pages, case["kv"], case["page"])
    x = torch.randn(*shape, case["D"], generator=gen, device=dev)
    if grid == INT4:
        c = (x * 3.0).round().clamp(-7, 7).to(torch.int8) & 15
    elif grid == E1M2:
        c = (x.abs() * 3.0).round().clamp(0, 7).to(torch.int8)
        c = c + 8 * ((x < 0) & (c > 0)).to(torch.int8)
    else:
        c = (x.abs() * 2.5).clamp(0, 7).to(torch.int8)
        c = c + 8 * ((x < 0) & (c > 0)).to(torch.int8)
    del x
    c = c.view(*shape, case["D"] // 2, 2)
    codes = (c[..., 0] | (c[..., 1] << 4)).view(torch.uint8)
    size = (0.5 + torch.rand(*shape, case["D"] // block, generator=gen, device=dev)) * (2.0 / TOP[grid])
    if case["scale"] == "pow2":
        return codes, (torch.log2(size).round() + 127).to(torch.uint8)
    return codes, size


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * seed + 29)
    s = dict(case)
    lens = _numbers(case["lens"])
    new = _numbers(case["new"]) if "new" in case else lens
    T, D, kv = sum(new), case["D"], case["kv"]
    starts = [0]
    for x in new:
        starts.append(starts[-1] + x)
    s["T"], s["new_list"], s["len_list"], s["start_list"] = T, new, lens, starts
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    s["factor"] = D ** -0.5
    if case["op"] != "kv":
        s["q"] = _rows(T, case["heads"], D, g, dev, 1.5)
    if case["op"] != "cache":
        s["k"], s["v"] = _rows(T, kv, D, g, dev, 1.0), _rows(T, kv, D, g, dev, 1.0)
    if case["op"] == "attn":
        s["do"] = (torch.randn(T, case["heads"], D, generator=g, device=dev) * 1e-3).to(torch.bfloat16) if case["grad"] else None
        return s
    # the sequences' pages lie anywhere in the cache, as a server that has run for a while hands them out
    page, wide = case["page"], max(1, max(-(-x // case["page"]) for x in lens))
    need = sum(-(-x // page) for x in lens)
    pages = need + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)[:need]
    table = torch.full((len(lens), wide), -1, dtype=torch.int32, device=dev)
    held = torch.tensor([-(-x // page) for x in lens], device=dev)
    table[torch.arange(wide, device=dev)[None, :] < held[:, None]] = order
    s["table"], s["lens"] = table, torch.tensor(lens, dtype=torch.int32, device=dev)
    s["sign_seed"] = 5101 + seed
    s["signs"] = torch.tensor(_signs(s["sign_seed"], case["n"]), dtype=torch.float32, device=dev)
    s["levels"] = torch.tensor(LEVELS[case["grid"]], dtype=torch.float32, device=dev)
    s["kc"], s["ks"] = _pages(case, pages, g, dev)
    s["vc"], s["vs"] = _pages(case, pages, g, dev)
    # where every packed row lies in its sequence
    seq = torch.repeat_interleave(torch.arange(len(new), device=dev), torch.tensor(new, device=dev))
    s["seq"] = seq
    s["at"] = torch.arange(T, device=dev) - s["starts"].long()[seq] + (s["lens"].long() - torch.tensor(new, device=dev))[seq]
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _plain_attn(s):
    T, D, heads, kv = s["T"], s["D"], s["heads"], s["kv"]
    G = heads // kv
    dev = s["q"].device
    out = dict(o=torch.zeros(T, heads, D, dtype=torch.bfloat16, device=dev), lse=torch.zeros(T, heads, device=dev))
    if s["grad"]:
        out |= dict(dq=torch.zeros_like(s["q"]), dk=torch.zeros_like(s["k"]), dv=torch.zeros_like(s["v"]))
    for a, n in zip(s["start_list"], s["new_list"]):
        if n == 0:
            continue
        # [key heads, group * tokens, D]
        turn = lambda x: x[a:a + n].float().view(n, kv, G, D).permute(1, 2, 0, 3).reshape(kv, G * n, D)  # noqa: E731
        back = lambda x: x.view(kv, G, n, D).permute(2, 0, 1, 3).reshape(n, heads, D)  # noqa: E731
        q, k, v = turn(s["q"]), s["k"][a:a + n].float().transpose(0, 1).contiguous(), s["v"][a:a + n].float().transpose(0, 1).contiguous()
        z = torch.matmul(q, k.transpose(1, 2).contiguous()).mul_(s["factor"]).view(kv, G, n, n)
        later = torch.ones(n, n, dtype=torch.bool, device=dev).triu_(1)
        z.masked_fill_(later, -math.inf)
        top = z.amax(3, keepdim=True)
        p = torch.exp(z.sub_(top), out=z)
        whole = p.sum(3, keepdim=True)
        p.div_(whole)
        out["lse"][a:a + n] = (top + whole.log()).view(heads, n).t()
        p = p.view(kv, G * n, n)
        out["o"][a:a + n] = back(torch.matmul(p, v)).to(torch.bfloat16)
        if not s["grad"]:
            continue
        do = turn(s["do"])
        out["dv"][a:a + n] = torch.matmul(p.transpose(1, 2).contiguous(), do).transpose(0, 1).to(torch.bfloat16)
        dp = torch.matmul(do, v.transpose(1, 2).contiguous())
        ds = dp.sub_((p * dp).sum(2, keepdim=True)).mul_(p).mul_(s["factor"])
        out["dq"][a:a + n] = back(torch.matmul(ds, k)).to(torch.bfloat16)
        out["dk"][a:a + n] = torch.matmul(ds.transpose(1, 2).contiguous(), q).transpose(0, 1).to(torch.bfloat16)
    return out


def _plain_butterflies(x, n):
    """The Sylvester transform of whole chunks of n, h = 1, 2, ..., n / 2, in fp32."""
    h, shape = 1, x.shape
    while h < n:
        x = x.reshape(-1, 2, h)
        x = torch.stack([x[:, 0] + x[:, 1], x[:, 0] - x[:, 1]], 1)
        h *= 2
    return x.reshape(shape)


def _plain_rounding(x, s):
    """(codes, scales) of blocks along the last dimension."""
    grid, top = s["grid"], TOP[s["grid"]]
    b = x.view(*x.shape[:-1], -1, s["block"])
    m = b.abs().amax(-1)
    if s["scale"] == "pow2":
        f, e = torch.frexp(m)  # the least e with m <= top 2^e; top = f0 2^e0
        f0, e0 = math.frexp(top)
        e = torch.where(m == 0, torch.full_like(e, -127), torch.where(f > f0, e - e0 + 1, e - e0).clamp(-127, 127))
        scales, v = (e + 127).to(torch.uint8), torch.ldexp(b, -e[..., None])
    else:
        scales = m / top
        v = torch.where(scales[..., None] == 0, torch.zeros_like(b), b / scales[..., None])
    v = v.view(x.shape)
    a = v.abs()
    if grid == INT4:
        return torch.round(v).to(torch.int32).clamp(-7, 7) & 15, scales
    if grid == E1M2:
        k = torch.round(a * 4.0).clamp(max=7)
    else:
        k = torch.where(a < 2, torch.round(a * 2), torch.where(a < 4, torch.round(a) + 2, torch.round(a * 0.5) + 4)).clamp(max=7)
    k = k.to(torch.int32)
    return k + 8 * ((v < 0) & (k > 0)).to(torch.int32), scales


def _plain_values(codes, scales, s):
    """What the codes stand for, in the basis of the rotation."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    v = torch.take(s["levels"], c.long()).view(*scales.shape, s["block"])
    size = torch.exp2(scales.float() - 127.0) if s["scale"] == "pow2" else scales
    return (v * size[..., None]).flatten(-2)


def _plain_back(x, s):
    """Out of the basis of the rotation."""
    n = s["n"]
    if n == 1:
        return x
    y = _plain_butterflies(x, n) * (1.0 / math.sqrt(n))
    return (y.view(-1, n) * s["signs"]).view(x.shape)


def _plain_kv(s):
    page, n = s["page"], s["n"]
    at, seq = s["at"], s["seq"]
    where, row = s["table"][seq, at // page].long(), at % page
    out = {}
    for name, codes, scales in (("k", s["kc"], s["ks"]), ("v", s["vc"], s["vs"])):
        x = s[name].float()
        if n > 1:
            x = _plain_butterflies((x.view(-1, n) * s["signs"]).view(x.shape), n) * (1.0 / math.sqrt(n))
        c, size = _plain_rounding(x, s)
        c = c.view(*c.shape[:-1], -1, 2)
        codes[where, :, row] = (c[..., 0] | (c[..., 1] << 4)).to(torch.uint8)
        scales[where, :, row] = size
        out[name] = _plain_back(_plain_values(codes[where, :, row], scales[where, :, row], s), s).to(torch.bfloat16)
    return out


def _plain_cache(s):
    page, kv, D, heads, T = s["page"], s["kv"], s["D"], s["heads"], s["T"]
    B, G, most, L = len(s["new_list"]), heads // kv, max(s["new_list"]), max(s["len_list"])
    dev = s["q"].device
    t = torch.arange(L, device=dev)
    where = s["table"][:, t // page].long().clamp_(min=0)
    row = (t % page)[None, :].expand(B, L)
    # [sequences, key heads, kept tokens, D]
    k = _plain_back(_plain_values(s["kc"][where, :, row], s["ks"][where, :, row], s), s).transpose(1, 2).contiguous()
    v = _plain_back(_plain_values(s["vc"][where, :, row], s["vs"][where, :, row], s), s).transpose(1, 2).contiguous()
    first = s["lens"].long() - (s["starts"][1:] - s["starts"][:-1]).long()
    slot = s["at"] - first[s["seq"]]
    q = torch.zeros(B, most, heads, D, device=dev)
    q[s["seq"], slot] = s["q"].float()
    q = q.view(B, most, kv, G, D).permute(0, 2, 3, 1, 4).reshape(B, kv, G * most, D)
    z = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(s["factor"]).view(B, kv, G, most, L)
    seen = first[:, None] + torch.arange(most, device=dev)[None, :]
    z.masked_fill_((t[None, None, :] > seen[:, :, None])[:, None, None], -math.inf)
    p = torch.exp(z - z.amax(4, keepdim=True))
    p = (p / p.sum(4, keepdim=True)).view(B, kv, G * most, L)
    o = torch.matmul(p, v).view(B, kv, G, most, D).permute(0, 3, 1, 2, 4).reshape(B, most, heads, D)
    return dict(o=o[s["seq"], slot].to(torch.bfloat16))


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    s = state
    if not own:
        return {"attn": _plain_attn, "kv": _plain_kv, "cache": _plain_cache}[s["op"]](s)
    import rht_bit_block_amd as U
    if s["op"] == "attn":
        o, lse = U.ufp4_attn_fwd(s["q"], s["k"], s["v"], s["starts"])
        if not s["grad"]:
            return dict(o=o, lse=lse)
        dq, dk, dv = U.ufp4_attn_bwd(s["q"], s["k"], s["v"], s["starts"], o, lse, s["do"])
        return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)
    cfg = U.make_cfg(s["grid"], U.UFP4_RTNE, U.UFP4_SCALE_POW2 if s["scale"] == "pow2" else U.UFP4_SCALE_F32, 1, s["block"], s["n"],
                     sign_seed=s["sign_seed"])
    cache = U.KVCache(s["kc"], s["ks"], s["vc"], s["vs"], cfg)
    if s["op"] == "kv":
        U.ufp4_kv_write(s["k"], s["v"], s["starts"], s["lens"], s["table"], cache)
        k, v = U.ufp4_kv_read(cache, s["starts"], s["lens"], s["table"], s["T"])
        return dict(k=k, v=v)
    return dict(o=U.ufp4_kv_attn(s["q"], s["starts"], s["lens"], s["table"], cache))


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    lens = _numbers(case["lens"])
    new = _numbers(case["new"]) if "new" in case else lens
    T, D, kv = sum(new), case["D"], case["kv"]
    if case["op"] == "attn":
        heads = case["heads"]
        pairs = sum(n * (n + 1) // 2 for n in lens)
        read, lse = 2 * T * D * (heads + 2 * kv), 4 * T * heads
        if not case["grad"]:
            return {"bytes": read + 2 * T * D * heads + lse, "flops": 4.0 * pairs * heads * D}
        # two products forward, five backward (the scores again)
        return {"bytes": 2 * read + 4 * T * D * heads + 2 * lse + 2 * T * D * (heads + 2 * kv) + 2 * T * D * heads,
                "flops": 14.0 * pairs * heads * D}
    # two tensors, half a byte a code and the blocks' scales
    held = 2 * kv * D * (0.5 + (1.0 if case["scale"] == "pow2" else 4.0) / case["block"])
    index = 4 * (2 * len(lens) + 1) + 4 * sum(-(-x // case["page"]) for x in lens)
    if case["op"] == "kv":
        return {"bytes": T * (2 * held + 2 * 4 * kv * D) + index, "flops": 2.0 * T * kv * D * (20 + 2 * math.log2(case["n"]))}
    pairs = sum(x * n - x * (x - 1) // 2 for x, n in zip(new, lens))
    return {"bytes": sum(lens) * held + 4 * T * case["heads"] * D + index, "flops": 4.0 * pairs * case["heads"] * D}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_turn(seed, n, dev):
    """S H / sqrt(n) of a seed."""
    i = torch.arange(n, device=dev)
    both, odd = i[:, None] & i[None, :], torch.zeros(n, n, dtype=torch.int64, device=dev)
    for bit in range(7):
        odd = odd ^ ((both >> bit) & 1)
    return torch.tensor(_signs(seed, n), dtype=torch.float64, device=dev)[:, None] * (1.0 - 2.0 * odd.double()) / math.sqrt(n)


def _exact_rows(codes, scales, case, turn):
    """Rows [N, D] of a cache as values out of the rotation's basis."""
    lv = torch.tensor(LEVELS[case["grid"]], dtype=torch.float64, device=codes.device)
    x = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    x[:, 0::2], x[:, 1::2] = lv[(codes & 15).long()], lv[(codes >> 4).long()]
    size = 2.0 ** (scales.double() - 127) if case["scale"] == "pow2" else scales.double()
    x *= size.repeat_interleave(case["block"], 1)
    return (x.view(-1, case["n"]) @ turn.t()).view(x.shape)


def _exact_attn(case, s):
    heads, kv, D = case["heads"], case["kv"], case["D"]
    G = heads // kv
    o, lse = s["q"].double() * 0, torch.zeros(s["T"], heads, dtype=torch.float64, device=s["q"].device)
    dq, dk, dv = s["q"].double() * 0, s["k"].double() * 0, s["v"].double() * 0
    for b, n in enumerate(s["new_list"]):
        rows = slice(s["start_list"][b], s["start_list"][b] + n)
        for h in range(heads if n else 0):
            q, k, v = s["q"][rows, h].double(), s["k"][rows, h // G].double(), s["v"][rows, h // G].double()
            for c in range(0, n, 4096):  # rows c .. of the queries against all keys up to their last
                e = min(n, c + 4096)
                z = (q[c:e] @ k[:e].t()) / math.sqrt(D)
                hide = torch.arange(e, device=z.device)[None, :] > torch.arange(c, e, device=z.device)[:, None]
                z[hide] = -math.inf
                l = torch.logsumexp(z, 1)
                p = torch.exp(z - l[:, None])
                mine = slice(rows.start + c, rows.start + e)
                keys = slice(rows.start, rows.start + e)
                o[mine, h], lse[mine, h] = p @ v[:e], l
                if case["grad"]:
                    do = s["do"][mine, h].double()
                    dv[keys, h // G] += p.t() @ do
                    ds = p * (do @ v[:e].t() - (do * o[mine, h]).sum(1)[:, None]) / math.sqrt(D)
                    dq[mine, h] = ds @ k[:e]
                    dk[keys, h // G] += ds.t() @ q[c:e]
    return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv) if case["grad"] else dict(o=o, lse=lse)


def _exact_quantized(x, case, turn):
    """Rows [N, D] rounded to the grid, out of the rotation's basis again."""
    y = (x.double().view(-1, case["n"]) @ turn).view(-1, case["block"])
    m, top = y.abs().amax(1, keepdim=True), TOP[case["grid"]]
    size = (m / top).float().double()  # a scale is kept in 32 bits
    if case["scale"] == "pow2":
        size = m / top
        e = torch.ceil(torch.log2(size))
        e = torch.where(size <= torch.exp2(e - 1), e - 1, e)
        size = torch.exp2(torch.where(size > torch.exp2(e), e + 1, e).clamp(-127, 127))
    grid = torch.tensor(sorted(set(abs(v) for v in LEVELS[case["grid"]] if abs(v) <= top)), dtype=torch.float64, device=y.device)
    a = torch.where(m > 0, (y.abs() / size).float().double(), torch.zeros_like(y))  # and so is the quotient that is rounded
    up = torch.searchsorted(grid, a.contiguous()).clamp(1, 7)
    low, high = grid[up - 1], grid[up]
    mid = (low + high) / 2
    got = torch.where((a > mid) | ((a == mid) & (up % 2 == 0)), high, low)
    return ((got * torch.sign(y) * size).view(-1, case["n"]) @ turn.t()).view(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(case, s)
    dev = s["kc"].device
    turn = _exact_turn(s["sign_seed"], case["n"], dev)
    if case["op"] == "kv":
        return {x: _exact_quantized(s[x].reshape(-1, case["D"]), case, turn).view(s[x].shape) for x in ("k", "v")}
    heads, kv, page = case["heads"], case["kv"], case["page"]
    o = torch.zeros(s["T"], heads, case["D"], dtype=torch.float64, device=dev)
    for b, (n, have) in enumerate(zip(s["new_list"], s["len_list"])):
        mine = s["table"][b, :-(-have // page)].long()
        for g in range(kv):
            k, v = (_exact_rows(c[mine, g].flatten(0, 1)[:have], z[mine, g].flatten(0, 1)[:have], case, turn)
                    for c, z in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
            for i in range(n):
                end, row = have - n + i + 1, s["start_list"][b] + i
                hs = slice(g * (heads // kv), (g + 1) * (heads // kv))
                w = torch.softmax(s["q"][row, hs].double() @ k[:end].t() / math.sqrt(case["D"]), 1)
                o[row, hs] = w @ v[:end]
    return dict(o=o)
