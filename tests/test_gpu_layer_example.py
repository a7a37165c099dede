"""The layer of examples/gdn_layer.py: gradients against autograd of a plain fp32
layer, and token-by-token serving against the whole sequence at once."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
from gdn_layer import Config, Layer, main  # noqa: E402

pytestmark = pytest.mark.gpu


def plain(p, c, h):
    """The layer in elementary fp32 operations (autograd differentiates it)."""
    rms = lambda x, w: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
    unit = lambda x: x * torch.rsqrt(x.square().sum(-1, keepdim=True) + 1e-6)
    B, T, _ = h.shape
    u = rms(h, p["norm"]) @ p["w_in"]
    raw, z, xg, xb = torch.split(u, [c.qkv, c.H * c.dv, c.H, c.H], dim=-1)
    pad = torch.cat([raw.new_zeros(B, c.W - 1, c.qkv), raw], dim=1)
    y = torch.nn.functional.silu((pad.unfold(1, c.W, 1) * p["conv_w"]).sum(-1) + p["conv_b"])
    q, k, v = torch.split(y, [c.Hk * c.dk, c.Hk * c.dk, c.H * c.dv], dim=-1)
    rep = lambda x: x.unflatten(-1, (c.Hk, c.dk)).repeat_interleave(c.H // c.Hk, dim=2)
    q, k, v = unit(rep(q)) * c.dk ** -0.5, unit(rep(k)), v.unflatten(-1, (c.H, c.dv))
    a = torch.exp(-p["rate"].exp() * torch.nn.functional.softplus(xg + p["bias"]))
    b = torch.sigmoid(xb)
    S, outs = h.new_zeros(B, c.H, c.dk, c.dv), []
    for t in range(T):
        S = a[:, t, :, None, None] * S
        e = b[:, t, :, None] * (v[:, t] - (k[:, t, :, :, None] * S).sum(2))
        S = S + k[:, t, :, :, None] * e[:, :, None]
        outs.append((q[:, t, :, :, None] * S).sum(2))
    n = rms(torch.stack(outs, 1), p["gate_norm"]) * torch.nn.functional.silu(
        z.unflatten(-1, (c.H, c.dv)))
    h2 = h + p["scale"] * rms(n.flatten(-2) @ p["w_out"], p["post"])
    return h2, rms(h2, p["norm_out"])


def test_layer_gradients():
    """bf16 activations through a dozen operators: each tensor within 3e-2 of its
    own 2-norm (2^-8 per rounding, about 60 of them adding up at random)."""
    c = Config()
    layer = Layer(c, seed=3)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    h, dout, dh2 = r(2, 75, c.C), r(2, 75, c.C).to(torch.bfloat16), r(2, 75, c.C)
    h2, out, _, saved = layer.forward(h)
    dh, grads = layer.backward(dout, dh2, saved)
    torch.cuda.synchronize()
    p = {k: v.clone().requires_grad_() for k, v in layer.p.items()}
    hr = h.clone().requires_grad_()
    ref2, ref = plain(p, c, hr)
    want = torch.autograd.grad([ref2, ref], [hr, *p.values()], [dh2, dout.float()])
    off = lambda u, w: float((u.float() - w.detach()).norm() / w.detach().norm())
    errs = {"h2": off(h2, ref2), "out": off(out, ref), "dh": off(dh, want[0])}
    errs |= {k: off(grads[k], w) for k, w in zip(p, want[1:])}
    print({k: f"{e:.1e}" for k, e in errs.items()})
    assert max(errs.values()) <= 3e-2, errs


def test_layer_serves_what_it_computes_at_once():
    c = Config()
    layer = Layer(c, seed=5)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    h = torch.randn(3, 40, c.C, generator=gen, device="cuda")
    whole = layer.forward(h)[1].float()
    cache = layer.cache(5)
    for s, slot in enumerate((4, 0, 2)):
        layer.prefill(h[s:s + 1, :30], cache, slot)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    slots = dict(slot_in=i32(4, 0, 2), slot_out=i32(4, 0, 2))
    for t in range(30, 34):
        _, out = layer.step(h[:, t].contiguous(), cache, **slots)
        assert float((out.float() - whole[:, t]).norm() / whole[:, t].norm()) <= 3e-2
    # six drafts each, none committed, then two, none and six of them
    packed = h[:, 34:].reshape(18, -1).contiguous()
    cu = i32(0, 6, 12, 18)
    for commit in ((0, 0, 0), (2, 0, 6)):
        _, out = layer.step(packed, cache, cu_seqlens=cu, n_commit=i32(*commit), **slots)
        out = out.view(3, 6, -1).float()
        assert float((out - whole[:, 34:]).norm() / whole[:, 34:].norm()) <= 3e-2
    _, out = layer.step(torch.cat([h[0, 36:38], h[1, 34:36]]), cache, cu_seqlens=i32(0, 2, 4, 4),
                        **slots)
    want = torch.cat([whole[0, 36:38], whole[1, 34:36]])
    assert float((out.float() - want).norm() / want.norm()) <= 3e-2


def test_example_runs(capsys):
    main()
    said = capsys.readouterr().out
    assert "branched: True" in said
