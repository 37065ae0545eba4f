"""A small mixture-of-experts language model trained with 4-bit GEMMs and then run
token by token on the same 4-bit weights.

    python examples/moe_lm.py [--steps 30]

One block: embedding, a routed expert layer with a residual connection, and a
linear head.  Training goes through the package from end to end: the dual
quantizers and grouped GEMMs of the experts (FPROP, DGRAD, WGRAD), the gated
activation that keeps its inputs as MXFP8 checkpoints (ufp4_glu_fwd,
ufp4_glu_bwd; the router's weights ride along as row factors), and the loss over
the vocabulary without stored logits (ufp4_linear_xent_fwd, _bwd).  Generation
runs the expert layer of a few tokens in ufp4_moe_tokens, on the codes that the
last training step quantized for FPROP.  The text is synthetic: every token is
followed by a fixed other one, most of the time.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import rht_bit_block_amd as U  # noqa: E402
import workloads  # noqa: E402

TOKENS, VOCAB, HIDDEN, FFN, EXPERTS, TOP_K = 512, 1003, 256, 320, 4, 2
N, BLOCK = 32, 32           # Hadamard size and block of every quantization
SIGNS = dict(fprop=11, dgrad=12, wgrad=13)


def cfg(gemm, rounding=U.UFP4_RTNE, seed=0):
    return U.make_cfg(U.UFP4_E1M2, rounding, U.UFP4_SCALE_F32, 1, BLOCK, N, sign_seed=SIGNS[gemm],
                      sr_seed=seed, sr_stream=0 if gemm == "dgrad" else 1)


class Model:
    def __init__(self, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        new = lambda *s, std: torch.randn(*s, generator=g, device=device) * std  # noqa: E731
        self.p = dict(embed=new(VOCAB, HIDDEN, std=1.0), head=new(VOCAB, HIDDEN, std=HIDDEN ** -0.5),
                      router=new(EXPERTS, HIDDEN, std=HIDDEN ** -0.5),
                      gate=new(EXPERTS * FFN, HIDDEN, std=HIDDEN ** -0.5),
                      up=new(EXPERTS * FFN, HIDDEN, std=HIDDEN ** -0.5),
                      down=new(EXPERTS * HIDDEN, FFN, std=FFN ** -0.5))
        self.quantize()

    def quantize(self):
        """4-bit copies of the expert weights: row-wise for FPROP and generation,
        column-wise per expert for DGRAD."""
        self.q = {}
        for name, rows in (("gate", FFN), ("up", FFN), ("down", HIDDEN)):
            w = self.p[name].to(torch.bfloat16)
            row, col = U.ufp4_rht_quant_dual(w, cfg("fprop"), cfg("dgrad"),
                                             [e * rows for e in range(EXPERTS + 1)])
            self.q[name] = row, U.stacked(col, EXPERTS)

    def route(self, x):
        """Router logits, the chosen experts and their softmax weights."""
        logits = x.float() @ self.p["router"].t()
        top = torch.sort(logits, dim=1, descending=True, stable=True)
        ids = top.indices[:, :TOP_K]
        return logits, ids, torch.softmax(top.values[:, :TOP_K], 1)

    def step(self, tokens, targets, seed):
        """Loss and gradients of one batch."""
        x = self.p["embed"][tokens].to(torch.bfloat16)
        logits, ids, share = self.route(x)
        host = ids.cpu()
        gather, offsets, _ = workloads.permute_by_expert(
            host, torch.bincount(host.reshape(-1), minlength=EXPERTS), max(N, BLOCK))
        offsets = offsets.tolist()
        # row r of the experts' batch is choice `choice[r]` of token `gather[r]`; padding has weight 0
        gather = gather.to(x.device)
        real = gather >= 0
        at = gather.clamp(min=0)
        expert = torch.repeat_interleave(torch.arange(EXPERTS, device=x.device),
                                         torch.tensor(offsets, device=x.device).diff())
        choice = (ids[at] == expert[:, None]).int().argmax(1)
        weight = torch.where(real, share[at, choice], torch.zeros_like(share[at, choice]))
        rows = workloads.gather_rows(x, gather)

        sr = lambda gemm: cfg(gemm, U.UFP4_SR, seed)  # noqa: E731
        xr, xc = U.ufp4_rht_quant_dual(rows, cfg("fprop"), cfg("wgrad"), offsets)
        gate = U.ufp4_gemm_fprop_grouped(xr, self.q["gate"][0], offsets)
        up = U.ufp4_gemm_fprop_grouped(xr, self.q["up"][0], offsets)
        h, kept = U.ufp4_glu_fwd(gate, up, row_scale=weight)
        hr, hc = U.ufp4_rht_quant_dual(h, cfg("fprop"), cfg("wgrad"), offsets)
        out = U.ufp4_gemm_fprop_grouped(hr, self.q["down"][0], offsets)
        y = x.float().index_add(0, at, torch.where(real[:, None], out, torch.zeros_like(out)))
        y16, head = y.to(torch.bfloat16), self.p["head"].to(torch.bfloat16)
        loss, lse = U.ufp4_linear_xent_fwd(y16, head, targets)

        live = (targets >= 0).sum().clamp(min=1)
        dloss = torch.full_like(loss, 1.0) / live
        g = {}
        dy, g["head"] = U.ufp4_linear_xent_bwd(y16, head, targets, lse, dloss)
        dout = workloads.gather_rows(dy, gather)
        dr, dc = U.ufp4_rht_quant_dual(dout, sr("dgrad"), sr("wgrad"), offsets)
        dh = U.ufp4_gemm_dgrad_grouped(dr, self.q["down"][1], offsets)
        g["down"] = U.ufp4_gemm_wgrad_grouped(dc, hc, offsets)
        dgate, dup, dweight, _ = U.ufp4_glu_bwd(kept, dh, row_scale=weight)
        dx = dy.float()
        for name, d in (("gate", dgate), ("up", dup)):
            dr, dc = U.ufp4_rht_quant_dual(d, sr("dgrad"), sr("wgrad"), offsets)
            part = U.ufp4_gemm_dgrad_grouped(dr, self.q[name][1], offsets)
            dx = dx.index_add(0, at, torch.where(real[:, None], part, torch.zeros_like(part)))
            g[name] = U.ufp4_gemm_wgrad_grouped(dc, xc, offsets)
        # the router: softmax over the chosen logits
        dshare = torch.zeros_like(share)
        dshare[at[real], choice[real]] = dweight[real]
        dtop = share * (dshare - (share * dshare).sum(1, keepdim=True))
        dlogits = torch.zeros_like(logits).scatter_(1, ids, dtop)
        g["router"] = dlogits.t() @ x.float()
        dx = dx + dlogits @ self.p["router"]
        g["embed"] = torch.zeros_like(self.p["embed"]).index_add_(0, tokens, dx)
        return loss.sum() / live, g, y16

    def update(self, grads, rate):
        for name, d in grads.items():
            d = d.float()
            self.p[name] -= rate * d / (d.square().mean().sqrt() + 1e-12) * self.p[name].square().mean().sqrt()
        self.quantize()

    def generate(self, tokens):
        """The block's output for a few tokens, experts on 4-bit weights."""
        x = self.p["embed"][tokens].to(torch.bfloat16)
        logits, _, _ = self.route(x)
        y = U.ufp4_moe_tokens(x, logits, self.q["gate"][0], self.q["up"][0], self.q["down"][0], TOP_K)
        return x.float() + y.float()


def batch(step, device="cuda"):
    """Tokens and what follows them: a fixed successor nine times in ten; the
    first eighth of the batch carries no loss."""
    g = torch.Generator(device=device).manual_seed(1000 + step)
    t = torch.randint(0, VOCAB, (TOKENS,), generator=g, device=device)
    t = t * t % VOCAB                       # some tokens are much more frequent than others
    after = (t * 7 + 3) % VOCAB
    noise = torch.rand(TOKENS, generator=g, device=device) < 0.1
    after = torch.where(noise, torch.randint(0, VOCAB, (TOKENS,), generator=g, device=device), after)
    after[: TOKENS // 8] = -100
    return t, after


def main(steps=30, say=print):
    """Returns (first loss, last loss, how far the few-token layer is from the
    training forward pass on the same tokens, share of right next tokens)."""
    m = Model()
    losses = []
    for s in range(steps):
        tokens, targets = batch(s)
        loss, grads, _ = m.step(tokens, targets, seed=s)
        losses.append(loss.item())
        m.update(grads, 0.05)
        if s % 5 == 0 or s == steps - 1:
            say(f"step {s:3d}  loss {losses[-1]:.4f}")
    tokens, targets = batch(steps)
    _, _, y = m.step(tokens, targets, seed=0)
    few = tokens[-16:]
    z = m.generate(few)
    x = m.p["embed"][few].to(torch.bfloat16).float()
    off = ((z - y[-16:].float()).norm() / (y[-16:].float() - x).norm()).item()
    right, t = 0, few[:1]
    for _ in range(16):                     # one token after another
        nxt = (m.generate(t) @ m.p["head"].t()).argmax(1)
        right += int(nxt.item() == (t.item() * 7 + 3) % VOCAB)
        t = nxt
    say(f"expert layer of 16 tokens against the training pass: {off:.3f} relative; "
        f"{right} of 16 generated tokens follow the rule")
    return losses[0], losses[-1], off, right / 16


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=30)
    main(ap.parse_args().steps)
