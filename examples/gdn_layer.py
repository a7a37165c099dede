"""A Gated DeltaNet layer on the library's operators: trained over chunks, then
served token by token with drafted tokens.

    python examples/gdn_layer.py        # a few training steps, then generation

Products with weight matrices are torch's; everything between them is the
library's: the block boundary (gdn_res_norm), the short convolution
(gdn_conv), the maps of q, k and the gates (gdn_prep), the chunk transition
(gdn_chunk), the gated norm of its output (gdn_gate_norm); and for serving
gdn_conv_step and gdn_step over caches of states.
"""
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from chunked_linear_recurrence_gated_gb300 import gdn  # noqa: E402


@dataclass
class Config:
    C: int = 256          # width of the residual stream
    H: int = 4            # value heads
    Hk: int = 2           # key heads
    dk: int = 128
    dv: int = 128
    W: int = 4            # width of the short convolution

    @property
    def qk(self):
        return 2 * self.Hk * self.dk

    @property
    def qkv(self):
        return self.qk + self.H * self.dv


class Layer:
    """Parameters (fp32 masters; matrices used in bf16) and the two ways to run them."""

    def __init__(self, cfg, device="cuda", seed=0):
        self.cfg = cfg
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=gen, device=device)
        c = cfg
        self.p = {
            "norm": torch.ones(c.C, device=device),
            "w_in": r(c.C, c.qkv + c.H * c.dv + 2 * c.H) * c.C ** -0.5,   # q k v | z | decay, write
            "conv_w": r(c.qkv, c.W) * c.W ** -0.5,
            "conv_b": torch.zeros(c.qkv, device=device),
            "rate": torch.log(torch.linspace(1.0, 8.0, c.H, device=device)),
            "bias": torch.linspace(-4.0, -1.0, c.H, device=device),
            "gate_norm": torch.ones(c.dv, device=device),
            "w_out": r(c.H * c.dv, c.C) * (c.H * c.dv) ** -0.5,
            "post": torch.ones(c.C, device=device),
            "scale": torch.full((c.C,), 0.5, device=device),
            "norm_out": torch.ones(c.C, device=device),
        }

    def matrix(self, name):
        return self.p[name].to(torch.bfloat16)

    def split(self, u):
        """The parts of one projection [.., qkv + H dv + 2 H]."""
        c = self.cfg
        z = u[..., c.qkv:c.qkv + c.H * c.dv].unflatten(-1, (c.H, c.dv))
        gates = u[..., c.qkv + c.H * c.dv:]
        return u[..., :c.qkv], z, gates[..., :c.H], gates[..., c.H:]

    def heads(self, y):
        """q, k and v in the convolution's output [.., qkv]."""
        c = self.cfg
        n = c.Hk * c.dk
        return (y[..., :n].unflatten(-1, (c.Hk, c.dk)), y[..., n:2 * n].unflatten(-1, (c.Hk, c.dk)),
                y[..., c.qk:].unflatten(-1, (c.H, c.dv)))

    # ------------------------------------------------------------ over a sequence
    def forward(self, h, conv_state=None, S=None):
        """One block over h [B, T, C] (fp32 residual stream). Returns (h, the normed
        stream that a next block or the head reads, what backward needs)."""
        p, c = self.p, self.cfg
        _, x = gdn.gdn_res_norm_fwd(h, None, p["norm"], dtype=torch.bfloat16)
        u = x @ self.matrix("w_in")
        raw, z, xg, xb = self.split(u)
        raw = raw.contiguous()
        y, conv_out = gdn.gdn_conv_fwd(raw, p["conv_w"], p["conv_b"], conv_state)
        q, k, v = self.heads(y)
        v = v.contiguous()
        scale = c.dk ** -0.5
        qn, kn, g, beta = gdn.gdn_prep_fwd(q, k, xg, xb, p["rate"], p["bias"], q_scale=scale)
        o, S_out = gdn.gdn_chunk_fwd(qn, kn, v, g, beta, S)
        n = gdn.gdn_gate_norm_fwd(o, z, p["gate_norm"])
        block = n.flatten(-2) @ self.matrix("w_out")
        h2, out = gdn.gdn_res_norm_fwd(h, block, p["norm_out"], p["post"], p["scale"])
        saved = (h, x, raw, conv_state, y, q, k, z, xg, xb, qn, kn, v, g, beta, S, o, n, block, h2)
        return h2, out, (conv_out, S_out), saved

    def backward(self, dout, dh2, saved):
        """Gradients of every parameter and of h for <dout, out> + <dh2, h2>."""
        p, c = self.p, self.cfg
        h, x, raw, conv_state, y, q, k, z, xg, xb, qn, kn, v, g, beta, S, o, n, block, h2 = saved
        gr = {}
        dh, dblock, gr["norm_out"], gr["post"], gr["scale"] = gdn.gdn_res_norm_bwd(
            h2, block, p["norm_out"], dout, dh2, p["post"], p["scale"])
        flat = lambda t: t.flatten(0, 1)
        gr["w_out"] = (flat(n.flatten(-2)).t() @ flat(dblock)).float()
        dn = (dblock @ self.matrix("w_out").t()).unflatten(-1, (c.H, c.dv))
        do, dz, gr["gate_norm"] = gdn.gdn_gate_norm_bwd(o, z, p["gate_norm"], dn)
        dqn, dkn, dv, dg, dbeta, _ = gdn.gdn_chunk_bwd(qn, kn, v, g, beta, S, do)
        dq, dk, dxg, dxb, gr["rate"], gr["bias"] = gdn.gdn_prep_bwd(
            q, k, xg, xb, p["rate"], p["bias"], dqn, dkn, dg, dbeta, q_scale=c.dk ** -0.5)
        dy = torch.cat([dq.flatten(-2), dk.flatten(-2), dv.flatten(-2)], dim=-1)
        draw, gr["conv_w"], gr["conv_b"], _ = gdn.gdn_conv_bwd(raw, p["conv_w"], p["conv_b"],
                                                               conv_state, dy)
        du = torch.cat([draw, dz.flatten(-2), dxg, dxb], dim=-1)
        gr["w_in"] = (flat(x).t() @ flat(du)).float()
        dx = du @ self.matrix("w_in").t()
        dh, _, gr["norm"], _, _ = gdn.gdn_res_norm_bwd(h, None, p["norm"], dx, dh, dh=dh)
        return dh, gr

    # ------------------------------------------------------------ token by token
    def cache(self, slots, device="cuda"):
        """Zeroed caches: convolution inputs and recurrence states of `slots` sequences."""
        c = self.cfg
        return (torch.zeros(slots, c.W - 1, c.qkv, dtype=torch.bfloat16, device=device),
                torch.zeros(slots, c.H, c.dk, c.dv, device=device))

    def prefill(self, h, cache, slot):
        """A prompt h [1, T, C] through the chunk path, its states into a slot."""
        h, out, (conv, S), _ = self.forward(h)
        cache[0][slot], cache[1][slot] = conv[0], S[0]
        return h, out

    def step(self, h, cache, **seqs):
        """The block for packed new tokens h [n, C] of cached sequences (slot_in,
        slot_out, cu_seqlens, n_commit as gdn_step takes them)."""
        p, c = self.p, self.cfg
        _, x = gdn.gdn_res_norm_fwd(h, None, p["norm"], dtype=torch.bfloat16)
        raw, z, xg, xb = self.split(x @ self.matrix("w_in"))
        y = gdn.gdn_conv_step(raw, p["conv_w"], p["conv_b"], cache[0], **seqs)
        q, k, v = self.heads(y)
        o = gdn.gdn_step(q, k, v, xg, xb, cache[1], **seqs, gate=(p["rate"], p["bias"]),
                         q_scale=c.dk ** -0.5)
        n = gdn.gdn_gate_norm_fwd(o[None], z[None], p["gate_norm"])[0]
        block = n.flatten(-2) @ self.matrix("w_out")
        return gdn.gdn_res_norm_fwd(h, block, p["norm_out"], p["post"], p["scale"])


def train(layer, steps=20, B=4, T=300, lr=0.2, seed=1):
    """A few steps of normalised gradient descent on a small task: out_t is to be
    h_{t - 1}. Returns the losses."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    losses = []
    for _ in range(steps):
        h = torch.randn(B, T, layer.cfg.C, generator=gen, device="cuda")
        target = torch.roll(h, 1, dims=1)
        h2, out, _, saved = layer.forward(h)
        diff = out.float() - target
        diff[:, :1] = 0.0
        losses.append(float(diff.square().mean()))
        dout = (2.0 / diff.numel() * diff).to(out.dtype)
        _, grads = layer.backward(dout, None, saved)
        norm = torch.sqrt(sum(g.square().sum() for g in grads.values()))
        for name, g in grads.items():
            layer.p[name] -= lr * g / norm
    return losses


def main():
    layer = Layer(Config())
    losses = train(layer, steps=40)
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f}")

    # two sequences in a cache of four slots: prompts, then single tokens
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    h = torch.randn(2, 90, layer.cfg.C, generator=gen, device="cuda")
    cache = layer.cache(4)
    for s in range(2):
        layer.prefill(h[s:s + 1, :80], cache, slot=s)
    for t in range(80, 84):
        layer.step(h[:, t].contiguous(), cache, slot_in=i32(0, 1), slot_out=i32(0, 1))
    # four drafted tokens of each are verified (the slots stay), three of the first
    # and one of the second accepted: passed again and committed, with the next
    # drafts behind them
    drafts = h[:, 84:88].reshape(8, -1).contiguous()
    layer.step(drafts, cache, cu_seqlens=i32(0, 4, 8), n_commit=i32(0, 0), slot_in=i32(0, 1),
               slot_out=i32(0, 1))
    packed = torch.cat([h[0, 84:89], h[1, 84:89]])
    _, out = layer.step(packed, cache, cu_seqlens=i32(0, 5, 10), n_commit=i32(3, 1),
                        slot_in=i32(0, 1), slot_out=i32(0, 1))
    whole = layer.forward(h[:, :89].contiguous())[1]
    err = max(float((out[5 * s:5 * s + 5].float() - whole[s, 84:89].float()).abs().max())
              for s in range(2))
    print(f"generation: verified tokens against the whole sequence at once: {err:.3f} of "
          f"{float(whole.float().abs().max()):.1f}")
    # a branch of the first sequence in slot 2
    layer.step(h[0, 87:87], cache, cu_seqlens=i32(0, 0), slot_in=i32(0), slot_out=i32(2))
    print("branched:", bool(torch.equal(cache[1][0], cache[1][2])))
    torch.cuda.synchronize()


if __name__ == "__main__":
    main()
