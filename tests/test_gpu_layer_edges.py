"""Edges of the layer operators (include/gdn_layer.h) on the GPU: waits that run
out, open gates, small eps, empty batches, and the precision of fp32 calls."""
import numpy as np
import pytest
import torch

import step_precision as sp
from chunked_linear_recurrence_gated_gb300 import gdn
from helpers import np64
from oracle import layer_ops as lo
from test_gpu_layer_ops import DT, HALF, check, gen, i32, ref_step, step_inputs
from test_gpu_layer_ops import test_res_norm as check_res_norm

pytestmark = pytest.mark.gpu


# ------------------------------------------------- the exchange within a cluster
def test_exchange_sums_arrive():
    gdn.gdn_layer_status()
    sums = torch.zeros(4, device="cuda")
    assert gdn.diag_exchange(sums) == 0
    assert gdn.gdn_layer_status() == 0
    assert sums.tolist() == [256.0] * 4


@pytest.mark.parametrize("silent", range(4))
def test_exchange_wait_that_runs_out_is_reported(silent):
    """A CTA that sends nothing: every wait of its cluster runs out, the sums are
    NaN, the status says so once, and the context keeps computing."""
    gdn.gdn_layer_status()
    sums = torch.zeros(4, device="cuda")
    assert gdn.diag_exchange(sums, silent=silent, limit_log2=20) == 0
    assert gdn.gdn_layer_status() == 5  # GDN_ERR_TIMEOUT; reading resets it
    assert gdn.gdn_layer_status() == 0
    assert torch.isnan(sums).all()
    check_res_norm(("bf16", "f32"), True, True, 37, 8200)
    assert gdn.gdn_layer_status() == 0

# --------------------------------------------------------------- open and closed gates
def gate_inputs(dtype):
    """z over [-80, 80], the other factors of the gradient fixed, and s(z), 1 - s(z) in fp64."""
    z = torch.linspace(-80, 80, 64 * 40, device="cuda").to(dtype)
    x = np64(z)
    return z, lo.sigmoid(x), lo.sigmoid(-x)


# fp32: expf 2 ulp, reciprocal and products 1 each, rsqrtf 2: below 16 u. bf16 results:
# __expf is good to 2 + 1.2 |x| ulp (98 at 80, 1.2e-5), then the result's rounding.
GATE_TOL = {torch.float32: 1e-6, torch.bfloat16: 2e-5 + HALF}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_gate_norm_gradient_of_open_and_closed_gates(dtype, act):
    """dz element by element: the gate's derivative does not cancel where s is near 1."""
    z, s, t = gate_inputs(dtype)
    z = z.view(1, 40, 1, 64)
    o, w = torch.ones_like(z), torch.ones(64, device="cuda")
    _, dz, _ = gdn.gdn_gate_norm_bwd(o, z, w, o, act)
    torch.cuda.synchronize()
    n, x = 1.0 / np.sqrt(1.0 + 1e-6), np64(z).reshape(-1)
    want = n * (s * t if act == "sigmoid" else s * (1.0 + x * t))
    mag = n * (s * t if act == "sigmoid" else s * (1.0 + np.abs(x) * t))
    off = np.abs(np64(dz).reshape(-1) - want) / mag
    assert off.max() <= GATE_TOL[dtype], (off.max(), x[off.argmax()])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prep_gradient_of_open_and_closed_gates(dtype):
    xb, s, t = gate_inputs(dtype)
    xb = xb.view(1, -1, 4)
    T = xb.shape[1]
    qk = torch.ones(1, T, 4, 64, dtype=dtype, device="cuda")
    one, zero = torch.ones_like(xb), torch.zeros(4, device="cuda")
    dxb = gdn.gdn_prep_bwd(qk, qk, xb, xb, zero, zero, qk, qk, one, one)[3]
    torch.cuda.synchronize()
    off = np.abs(np64(dxb).reshape(-1) - s * t) / (s * t)
    assert off.max() <= 1e-6 + (HALF if dtype == torch.bfloat16 else 0.0), off.max()

# ------------------------------------------------------------------------- small eps
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [1e-30, 1e-40])
def test_small_eps_and_small_rows(dtype, eps):
    """Zero rows, and rows far below sqrt(eps), where 1 / rms is up to 1e20: its square
    and cube must not be formed by themselves (0 times infinity)."""
    dt, r = DT[dtype], gen(51)
    x, h = r(6, 256, dtype=dt), r(6, 256, dtype=dt)
    for u in (x, h):
        u[0] = 0.0
        if eps == 1e-30:
            u[1] *= 1e-17
    w, wp, dy, dh = r(256), r(256), r(6, 256, dtype=dt), r(6, 256, dtype=dt)
    f = lambda *ts: [np64(t) for t in ts]

    def rows(name, got, ref):
        for i in range(got.shape[0]):
            # 1 / rms of both norms is 1e20 in row 0: parts of its dx have no fp32 value
            past = np.abs(ref[i]) > np.finfo(np.float32).max
            assert (np64(got[i])[past] == np.sign(ref[i][past]) * np.inf).all(), (name, i)
            keep = torch.from_numpy(~past)
            mag = np.abs(ref[i]).max()
            check(f"{name} row {i}", got[i].cpu()[keep], ref[i][~past], 5e-5, mag)

    got = gdn.gdn_res_norm_bwd(h, x, w, dy, dh, w_post=wp, eps=eps)
    ref = lo.res_norm_bwd(*f(h, x, w, dy, dh), w_post=np64(wp), eps=eps)[0]
    for name, u, v in zip(("dh", "dx"), got, ref):
        rows(name, u, v)
    rows("y", gdn.gdn_res_norm_fwd(h, x, w, wp, eps=eps)[1],
         lo.res_norm_fwd(*f(h, x, w, wp), eps=eps)[1])
    o = lambda t: t.view(1, 6, 4, 64)
    got = gdn.gdn_gate_norm_bwd(o(h), o(x), w[:64].clone(), o(dy), eps=eps)
    ref = lo.gate_norm_bwd(*f(o(h), o(x), w[:64], o(dy)), eps=eps)[0]
    for name, u, v in zip(("do", "dz"), got, ref):
        rows(name, u.view(24, 64), v.reshape(24, 64))
    gates = r(1, 6, 4, dtype=dt)
    a = (o(h), o(x), gates, gates, r(4), r(4), o(dy), o(dh), gates, gates)
    got = gdn.gdn_prep_bwd(*a, eps=eps)
    ref = lo.prep_bwd(*f(*a), eps=eps)[0]
    for name, u, v in zip(("dq", "dk"), got, ref):
        rows(name, u.view(24, 64), v.reshape(24, 64))

# --------------------------------------------------------------------- empty batches
def test_batches_without_tokens():
    e = lambda *s: torch.empty(*s, device="cuda")
    one = torch.ones(64, device="cuda")
    a = (e(2, 0, 2, 64), e(2, 0, 2, 64), e(2, 0, 2), e(2, 0, 2), one[:2], one[:2])
    assert gdn.gdn_prep_fwd(*a)[0].shape == (2, 0, 2, 64)
    p = gdn.gdn_prep_bwd(*a, e(2, 0, 2, 64), e(2, 0, 2, 64), e(2, 0, 2), e(2, 0, 2))
    assert gdn.gdn_gate_norm_fwd(e(2, 0, 1, 64), e(2, 0, 1, 64), one).shape == (2, 0, 1, 64)
    g = gdn.gdn_gate_norm_bwd(e(2, 0, 1, 64), e(2, 0, 1, 64), one, e(2, 0, 1, 64))
    assert gdn.gdn_res_norm_fwd(e(2, 0, 64), e(2, 0, 64), one)[1].shape == (2, 0, 64)
    r = gdn.gdn_res_norm_bwd(e(2, 0, 64), e(2, 0, 64), one, e(2, 0, 64), None, one, one)
    torch.cuda.synchronize()
    for t in (p[4], p[5], g[2], *r[2:]):
        assert not t.any()

# ------------------------------------------------------------------ the type of a norm
def test_res_norm_refuses_another_type_than_it_returns():
    r = gen(52)
    h, x, w = r(3, 64), r(3, 64, dtype=torch.bfloat16), r(64)
    with pytest.raises(ValueError):
        gdn.gdn_res_norm_fwd(h, x, w, dtype=torch.float32)
    with pytest.raises(ValueError):
        gdn.gdn_res_norm_fwd(h, None, w, y=torch.empty_like(h), dtype=torch.bfloat16)
    assert gdn.gdn_res_norm_fwd(h, x, w, dtype=torch.bfloat16)[1].dtype == torch.bfloat16
    assert gdn.gdn_res_norm_fwd(h, None, w, dtype=torch.bfloat16)[1].dtype == torch.bfloat16

# ------------------------------------------------------- precision of several tokens
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 256), (128, 128), (128, 256)])
@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("wide", [False, True])
def test_step_keeps_fp32(dtype, dk, dv, raw, wide):
    """States of every call, and outputs of fp32 calls, to the bound of operands in two
    TF32 parts (step_precision.py; one part is off by several times that). The wider
    blocks take calls of 466944 columns and more."""
    H, Hk = (32, 8) if wide else (4, 2)
    lens = [2, 3, 8, 9, 16, 1, 0, 33] * (-(-466944 // (8 * H * dv)) if wide else 1)
    q, k, v, g, beta, S, gate, cu = step_inputs(lens, H, Hk, dk, dv, DT[dtype], raw, dk + dv,
                                                len(lens))
    S *= 0.1
    commit = i32([n - i % 3 if n > 2 and i % 2 else n for i, n in enumerate(lens)])
    o = torch.zeros(q.shape[0], H, dv, dtype=DT[dtype], device="cuda")
    ro, rS = ref_step(q, k, v, g, beta, S, None, None, cu, commit, gate, dk ** -0.5, o)
    gdn.gdn_step(q, k, v, g, beta, S, cu_seqlens=cu, n_commit=commit, gate=gate,
                 q_scale=dk ** -0.5, o=o)
    torch.cuda.synchronize()
    S, at = np64(S), cu.tolist()
    for s, n in enumerate(lens):
        assert sp.error(S[s], rS[s]) <= sp.bound([n]), (s, n, sp.error(S[s], rS[s]))
    if dtype == "f32":
        got, ref = sp.by_head(np64(o), at), sp.by_head(ro, at)
        ns = [n for n in lens if n for _ in range(H)]
        off = [sp.error(a, b) / sp.bound([n]) for a, b, n in zip(got, ref, ns)]
        assert max(off) <= 1.0, max(off)

# ------------------------------------------------------------------- eps of each call
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [1e-5, 0.5])
def test_eps_is_used(dtype, eps):
    dt, r = DT[dtype], gen(53)
    f = lambda *ts: [np64(t) for t in ts]
    for lens in ([1, 1, 1], [3, 9, 2]):
        q, k, v, g, beta, S, gate, cu = step_inputs(lens, 2, 1, 64, 64, dt, True, 54, 3)
        q, k = q * 0.05, k * 0.05
        o = torch.zeros(q.shape[0], 2, 64, dtype=dt, device="cuda")
        ro, rS = lo.step(*f(q, k, v, g, beta, S), cu=cu.cpu().numpy(), gate=f(*gate), eps=eps)
        gdn.gdn_step(q, k, v, g, beta, S, cu_seqlens=cu, gate=gate, eps=eps, o=o)
        check("S", S, rS, 2e-5 * (1 + max(lens)))
        check("o", o, ro, 2e-5 * (1 + max(lens)))
    q, k, xg, xb = (r(2, 17, *s, dtype=dt, by=0.05) for s in ((2, 64), (2, 64), (4,), (4,)))
    rate, bias = r(4, by=0.5), r(4)
    for name, u, ref in zip(("q", "k"), gdn.gdn_prep_fwd(q, k, xg, xb, rate, bias, 0.3, eps),
                            lo.prep_fwd(*f(q, k, xg, xb, rate, bias), 0.3, eps)):
        check(name, u, ref, 1e-5)
    d = [r(2, 17, *s, dtype=dt) for s in ((4, 64), (4, 64), (4,), (4,))]
    got = gdn.gdn_prep_bwd(q, k, xg, xb, rate, bias, *d, q_scale=0.3, eps=eps)
    ref, _ = lo.prep_bwd(*f(q, k, xg, xb, rate, bias, *d), q_scale=0.3, eps=eps)
    for name, u, v in zip(("dq", "dk"), got, ref):
        check(name, u, v, 5e-5)
    o, z, dy, w = r(2, 17, 2, 64, dtype=dt, by=0.05), r(2, 17, 2, 64, dtype=dt), r(2, 17, 2, 64, dtype=dt), r(64)
    check("y", gdn.gdn_gate_norm_fwd(o, z, w, eps=eps), lo.gate_norm_fwd(*f(o, z, w), eps=eps), 1e-5)
    got = gdn.gdn_gate_norm_bwd(o, z, w, dy, eps=eps)
    ref, _ = lo.gate_norm_bwd(*f(o, z, w, dy), eps=eps)
    for name, u, v in zip(("do", "dz"), got, ref):
        check(name, u, v, 5e-5)
    for C in (128, 8200):
        h, x, dy, dh = (r(9, C, dtype=dt, by=b) for b in (0.05, 0.05, 1.0, 1.0))
        w, wp, sc = 1.0 + r(C, by=0.2), 1.0 + r(C, by=0.2), 0.5 + r(C, by=0.1)
        got = gdn.gdn_res_norm_fwd(h, x, w, wp, sc, eps)
        for name, u, v in zip(("h", "y"), got, lo.res_norm_fwd(*f(h, x, w, wp, sc), eps)):
            check(name, u, v, 1e-5)
        got = gdn.gdn_res_norm_bwd(h, x, w, dy, dh, wp, sc, eps)
        ref, _ = lo.res_norm_bwd(*f(h, x, w, dy, dh, wp, sc), eps)
        for name, u, v in zip(("dh", "dx"), got, ref):
            check(name, u, v, 5e-5)
    torch.cuda.synchronize()
