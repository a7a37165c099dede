"""Linear attention and the query / key norms (include/gdn_lin.h, gdn_layer.h) in calls that
lie at the edge of what their headers allow. Inputs and tolerances as in test_gpu_lin_ops."""
import subprocess
import sys

import numpy as np
import pytest
import torch

from chunked_linear_recurrence_gated_gb300 import gdn
from oracle import lin_ops as lo
from test_gpu_lin_ops import DT, HALF, check, gen, host, lin_inputs
from test_lin_edges_cpu import turns

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("decay", ["mid", "head"])
def test_no_tokens(dtype, packed, decay):
    """States pass through; a log-decay for each token has no elements, nor has its gradient
    (which torch gives as a null pointer)."""
    x = lin_inputs(1 if packed else 2, 0, 2, 64, 128, DT[dtype], decay, nseq=2)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda") if packed else None
    a = [x[i] for i in "qkvg"]
    o, S = gdn.gdn_lin_fwd(*a, x["S"], cu_seqlens=cu)
    assert o.numel() == 0 and torch.equal(S, x["S"])
    for dS, want in ((x["dS"], x["dS"]), (None, torch.zeros_like(x["dS"]))):
        r = gdn.gdn_lin_bwd(*a, x["S"], x["do"], dS, cu_seqlens=cu)
        torch.cuda.synchronize()
        assert torch.equal(r[4], want)
        assert r[3].shape == (x["g"].shape if decay == "mid" else (2,)) and (r[3] == 0).all()


# ------------------------------------------------------------------ dg by the token
# dg_u is the sum, over the pairs s < u <= t, of A_ts = scale (q_t . k_s) (dO_t . v_s) times
# the decay between them, with the states of the call as a first and a last such token; M_u is
# that sum of magnitudes, the oracle's on absolute values. Whatever is rounded on the way is a
# factor of these terms, so dg_u is off by a multiple of M_u, however large terms of other
# tokens are. fp32: a product of two operands of two TF32 parts, of two such products, decay
# factors of 2^-21, and states good to 2^-17 of their magnitudes: 2^-16 in all. bf16: states
# good to 3 2^-16 of their magnitudes, and one of two states (or a state before it meets a
# token) as two bf16 parts, 2^-16 more: 7 2^-16, and decay factors of 2^-21 and fp32 sums.
DG_TOL = {"f32": 2.0 ** -16, "bf16": 2.0 ** -13}


def dg_inputs(kind, dtype, T, H, dk, dv, cut, seed, decay="weak", nseq=1, B=1):
    """Tokens from `cut` on 1024 times as large in v and dO as those before it."""
    x = lin_inputs(B, T, H, dk, dv, DT[dtype], decay, seed=seed, nseq=nseq)
    x["v"][:, cut:] *= 1024
    x["do"][:, cut:] *= 1024
    x["dS"] *= 1024
    if kind != "decays":
        x["g"][:, cut] = -float("inf")  # a boundary that nothing crosses
    if kind == "no gradient before":
        x["do"][:, :cut] = 0
    return x


def dg_check(x, dtype, cu=None, scale=0.2):
    q, k, v, g, S, do, dS = host(*(x[i] for i in ("q", "k", "v", "g", "S", "do", "dS")))
    d = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    got = gdn.gdn_lin_bwd(*(x[i] for i in "qkvg"), x["S"], x["do"], x["dS"], scale=scale,
                          cu_seqlens=d)[3]
    with np.errstate(invalid="ignore"):
        ref = lo.lin_bwd(q, k, v, g, S, do, dS, scale, cu)[3]
        mag = lo.lin_bwd(*map(np.abs, (q, k, v)), g, *(None if t is None else np.abs(t) for t in (S, do, dS)),
                         scale, cu)[3]
    if x["g"].dim() == 1:
        ref, mag = ref.sum((0, 1)), mag.sum((0, 1))
    check("dg", got, ref, DG_TOL[dtype] * mag)
    return got


@pytest.mark.parametrize("dtype", sorted(DG_TOL))
@pytest.mark.parametrize("kind", ["boundary", "no gradient before", "decays"])
@pytest.mark.parametrize("cut", [40, 64, 300, 511])
@pytest.mark.parametrize("packed", [False, True])
def test_dg_beside_larger_tokens(dtype, kind, cut, packed):
    """Packed: the tokens around the boundary are in one unit of several chunks."""
    x = dg_inputs(kind, dtype, 700, 2, 64, 64, cut, cut)
    got = dg_check(x, dtype, [0, 700] if packed else None)
    if kind == "no gradient before":
        assert (got[:, :cut + 1] == 0).all()


@pytest.mark.parametrize("dtype", sorted(DG_TOL))
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("decay", ["none", "mid", "strong", "mixed", "head"])
def test_dg_of_each_token(dtype, dk, dv, decay):
    x = dg_inputs("decays", dtype, 500, 2, dk, dv, 390, dk, decay, nseq=3)
    dg_check(x, dtype, [0, 13, 400, 500])


@pytest.mark.parametrize("dtype", sorted(DG_TOL))
@pytest.mark.parametrize("S,dS", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("T", [1, 100, 128, 129, 256, 385, 700])
@pytest.mark.parametrize("packed", [False, True])
def test_dg_with_and_without_states(dtype, S, dS, T, packed):
    """Chunks that nothing comes into or goes out of, and ones that only tokens do."""
    x = dg_inputs("decays", dtype, T, 2, 64, 128, T // 2, T, nseq=4 if packed else 2, B=1 if packed else 2)
    if not S:
        x["S"] = None
    if not dS:
        x["dS"] = None
    dg_check(x, dtype, [0, T // 3, T // 3, T // 3 + T // 2, T] if packed else None)


@pytest.mark.parametrize("B,T,H,decay", [(1, 8200, 160, "weak"), (3, 2500, 60, "mid"), (1, 30000, 5, "weak"),
                                         (160, 400, 1, "none"), (1, 8200, 160, "head")])
def test_dg_of_long_units(B, T, H, decay):
    """bf16 against the fp32 kernels (held to the oracle above): units of up to a whole
    sequence, and sequences of many units; tokens behind forgotten states 1024 times as large."""
    x = dg_inputs("decays", "bf16", T, H, 64, 64, T - 200, 4, decay, nseq=B, B=B)
    if decay != "head":
        x["g"][:, T - 200] = -float("inf")
    f = {i: t.float() for i, t in x.items()}

    def dg(x, m=lambda t: t):
        return gdn.gdn_lin_bwd(m(x["q"]), m(x["k"]), m(x["v"]), x["g"], m(x["S"]), m(x["do"]),
                               m(x["dS"]), scale=0.2)[3].double()

    ref, mag = dg(f), dg(f, torch.abs)
    tol = (2.0 ** -13 + 2.0 ** -16) * mag + 1e-30 + (0.0 if decay == "head" else HALF * ref.abs())
    off = (dg(x) - ref).abs() - tol
    assert not (off > 0).any() and not off.isnan().any(), (off.max(), ref.abs().max())


@pytest.mark.parametrize("dtype,T,C", [("f32", 65536, 64), ("bf16", 262144, 128)])
@pytest.mark.parametrize("packed", [False, True])
def test_states_that_hardly_decay(dtype, T, C, packed):
    """Nothing but the decay acts on a state over thousands of chunks. A chunk's factor is
    good to 2^-23 of itself, and it, its product with others and the state's round by 2^-24
    each: 2^-22 a chunk."""
    H = 12
    r = gen(2)
    x = torch.zeros(1, T, H, 64, dtype=DT[dtype], device="cuda")
    S = 1 + r(1, H, 64, 64).abs()
    decay = -torch.logspace(-7, -3.7, H, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda") if packed else None
    got = (gdn.gdn_lin_fwd(x, x, x, decay, S, cu_seqlens=cu)[1],
           gdn.gdn_lin_bwd(x, x, x, decay, S, x, S, cu_seqlens=cu)[4])
    want = S.double() * torch.exp(T * decay.double())[None, :, None, None]
    for t in got:
        assert ((t - want).abs() <= T / C * 2.0 ** -22 * want).all()


@pytest.mark.parametrize("style", ["half", "pairs"])
def test_far_positions_of_large_frequencies(style):
    """Exact angles of the farthest positions at any frequency up to 2^40: below 2^-31 of a
    turn in whole numbers, the fraction of half a turn rounded by 2^-25, sine and cosine by
    2^-23, and the norm's factor by 2^-22: below 2^-20 of the sum of two terms of size 1."""
    f = torch.tensor([1.0, -100.25, 1e4, 1e6, 123456789.0, -2.0 ** 39, 3.3e11, 0.1], dtype=torch.float64)
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, 1 << 30, 7, -1]
    x = torch.ones(1, len(pos), 1, 64, device="cuda")
    y = gdn.gdn_qk_norm_fwd(x, x, None, None, f.cuda(), style=style, eps=1e-30,
                            pos=torch.tensor([pos], dtype=torch.int32, device="cuda"))[0][0, :, 0].cpu()
    at = np.array([[2 * np.pi * float(turns(g, p) % 1) for g in f.tolist()] for p in pos])
    a, b = (y[:, :8], y[:, 8:16]) if style == "half" else (y[:, 0:16:2], y[:, 1:16:2])
    assert np.abs(a.numpy() - (np.cos(at) - np.sin(at))).max() < 2.0 ** -20
    assert np.abs(b.numpy() - (np.cos(at) + np.sin(at))).max() < 2.0 ** -20
    assert (y[:, 16:] - 1).abs().max() < 2.0 ** -20


FIRST_IN_A_GRAPH = """
import torch
from chunked_linear_recurrence_gated_gb300 import gdn
r = lambda *s: torch.randn(*s, device="cuda")
for dt in (torch.bfloat16, torch.float32):
    q, k, v, do = (r(1, 700, 2, 64).to(dt) for _ in range(4))
    g, S, w = -r(1, 700, 2).abs().to(dt), r(1, 2, 64, 64), r(64)
    f = torch.rand(8, dtype=torch.float64, device="cuda")
    call = lambda: (gdn.gdn_lin_fwd(q, k, v, g, S) + gdn.gdn_lin_bwd(q, k, v, g, S, do, S)
                    + gdn.gdn_qk_norm_fwd(q, k, w, w, f) + gdn.gdn_qk_norm_bwd(q, k, w, w, f, q, k)
                    + (gdn.gdn_lin_step(q[0, :1], k[0, :1], v[0, :1], g[0, :1], S.clone()),))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, call()))
print("the same")
"""


def test_first_call_of_a_process_is_captured():
    r = subprocess.run([sys.executable, "-c", FIRST_IN_A_GRAPH], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "the same" in r.stdout, r.stderr[-2000:]
