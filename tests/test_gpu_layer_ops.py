"""GPU parity of the layer operators (include/gdn_layer.h) against their fp64
oracle, at the sizes, strides and masks where they can go wrong.

Tolerances, with u = 2^-24 (fp32 unit roundoff). A norm's statistic is a sum of
at most 64 terms per thread joined by a tree, so values are exact to about
(64 + 16) u < 1e-5 of the terms they are made of, which max|ref| measures; a
gradient joins two such statistics: 5e-5. A parameter gradient sums its terms in
chains of fewer than 170 additions: 2e-5 of the sum of their magnitudes. A
stored bf16 value (8 significant bits) is off by up to another 2^-8 of itself. Each token of the recurrence
adds the error of dot products of 128 terms, 128 u = 7.6e-6 of the state
column's norm: 2e-5 (1 + tokens) of it."""
import numpy as np
import pytest
import torch

from chunked_linear_recurrence_gated_gb300 import gdn
from helpers import np64
from oracle import layer_ops as lo

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = 2.0 ** -8  # unit roundoff of bf16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s, dtype=torch.float32, by=1.0: (
        torch.randn(*s, generator=g, device="cuda") * by).to(dtype)


def check(name, got, ref, by, mag=None):
    """|got - ref| <= by * (mag, or max|ref|) (+ the rounding of a bf16 result)."""
    if got is None and ref is None:
        return
    r = np.asarray(ref, dtype=np.float64)
    assert tuple(got.shape) == r.shape, name
    if r.size == 0:
        return
    tol = by * (np.abs(r).max() if mag is None else mag) + 1e-30
    if got.dtype == torch.bfloat16:
        tol = tol + HALF * np.abs(r)
    off = np.abs(np64(got) - r) - tol
    assert not (off > 0).any() and not np.isnan(off).any(), (name, off.max(), np.abs(r).max())


# ------------------------------------------------------------------ recurrence
def step_inputs(lens, H, Hk, dk, dv, dtype, raw, seed, slots):
    r = gen(seed)
    n = sum(lens)
    qkv = r(n, 2 * Hk * dk + H * dv, dtype=dtype)
    q, k = (qkv[:, i * Hk * dk:(i + 1) * Hk * dk].unflatten(1, (Hk, dk)) for i in range(2))
    v = qkv[:, 2 * Hk * dk:].unflatten(1, (H, dv))
    gates = r(n, 2 * H, dtype=dtype)
    g, beta = gates[:, :H], gates[:, H:]
    gate = (r(H, by=0.5), r(H)) if raw else None
    if not raw:
        for x in (q, k):
            x.copy_(torch.nn.functional.normalize(x.float(), dim=-1))
        g.copy_(-torch.nn.functional.softplus(g.float()))
        beta.copy_(torch.sigmoid(beta.float()))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    return q, k, v, g, beta, r(slots, H, dk, dv), gate, cu


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def ref_step(q, k, v, g, beta, S, si, so, cu, commit, gate, scale, o):
    c = lambda t: None if t is None else t.cpu().numpy()
    return lo.step(*[np64(t) for t in (q, k, v, g, beta, S)], c(si), c(so), c(cu), c(commit),
                   None if gate is None else [np64(t) for t in gate], scale, o=np64(o))


def run_step(lens, H, Hk, dk, dv, dtype, raw, seed, slots, si=None, so=None, commit=None,
             scale=1.0, packed=True):
    q, k, v, g, beta, S, gate, cu = step_inputs(lens, H, Hk, dk, dv, dtype, raw, seed, slots)
    cu = cu if packed else None
    si, so, commit = i32(si), i32(so), i32(commit)
    o = torch.full((q.shape[0], H, dv), 7.0, dtype=dtype, device="cuda")
    ro, rS = ref_step(q, k, v, g, beta, S, si, so, cu, commit, gate, scale, o)
    before = S.clone()
    gdn.gdn_step(q, k, v, g, beta, S, si, so, cu, commit, gate=gate, q_scale=scale, o=o)
    torch.cuda.synchronize()
    col = max(np.sqrt((x ** 2).sum(-2)).max() for x in (np64(before), rS))
    vmag = np.abs(np64(v)).max()
    by = 2e-5 * (1 + max(lens))
    check("S", S, rS, by, col + vmag)
    check("o", o, ro, by, col + vmag)
    return before, S, rS, o


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 256), (128, 64), (128, 128), (128, 256)])
@pytest.mark.parametrize("raw", [False, True])
def test_step_sizes(dtype, dk, dv, raw):
    run_step([3, 1, 0, 6], 6, 2, dk, dv, DT[dtype], raw, dk + dv, 4, scale=dk ** -0.5 if raw else 1.0)


@pytest.mark.parametrize("N,H", [(1, 1), (1, 16), (5, 3), (70, 2), (33, 7)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_one_token_each(N, H, dtype):
    run_step([1] * N, H, H, 128, 128, DT[dtype], True, N + H, N, packed=False, scale=0.1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv,N", [(64, 64, 230), (64, 128, 116), (64, 256, 58), (128, 64, 230),
                                     (128, 128, 116), (128, 256, 58)])
def test_step_large_calls(dtype, dk, dv, N):
    """Calls of many waves (32 heads): up to 10 tokens, some sequences with none."""
    lens = [(1, 0, 2, 5, 10, 1)[i % 6] for i in range(N)]
    commit = [min(n, i % 4) if i % 3 else n for i, n in enumerate(lens)]
    run_step(lens, 32, 8, dk, dv, DT[dtype], True, dk + dv, N, commit=commit, scale=dk ** -0.5)


@pytest.mark.parametrize("lens", [[1], [2], [5], [7], [8], [9], [16], [17], [33, 4, 70], [64, 1]])
def test_step_token_counts(lens):
    run_step(lens, 2, 1, 128, 128, torch.bfloat16, True, sum(lens), len(lens), scale=0.1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_slots_and_commits(dtype):
    """New sequences, states that are not kept, branches, copies, partial commits
    and out-of-range values; untouched slots keep their bits."""
    lens = [4, 4, 4, 0, 0, 3, 1, 5, 2]
    si = [2, 0, -1, 3, 9, 99, 6, 7, 8]
    so = [2, 0, 1, 4, -1, 5, -7, 10, 8]
    commit = [0, 2, 4, 0, 0, 3, 1, 1, 99]
    before, S, rS, _ = run_step(lens, 3, 3, 128, 128, DT[dtype], True, 11, 12, si, so, commit)
    for slot in (2, 3, 6, 7, 9, 11):      # read only or not named
        assert torch.equal(S[slot], before[slot]), slot
    assert torch.equal(S[4], before[3])   # copied without tokens


def test_step_branch_of_a_missing_state_is_zero():
    _, S, _, _ = run_step([0, 2], 2, 2, 64, 64, torch.float32, False, 12, 3, [-1, 1], [0, 1], [0, 2])
    assert not S[0].any()


def test_step_malformed_offsets_are_skipped():
    q, k, v, g, beta, S, gate, _ = step_inputs([6], 2, 2, 64, 64, torch.float32, False, 13, 4)
    cu = i32([0, 2, 1, 99, 6])            # second decreasing, third and fourth past the end
    o = torch.full((6, 2, 64), 7.0, device="cuda")
    before = S.clone()
    ro, rS = ref_step(q, k, v, g, beta, S, None, None, cu, None, None, 1.0, o)
    gdn.gdn_step(q, k, v, g, beta, S, cu_seqlens=cu, o=o)
    torch.cuda.synchronize()
    check("o", o, ro, 6e-5, 30.0)
    check("S", S, rS, 6e-5, 30.0)
    assert (o[2:] == 7.0).all() and torch.equal(S[1:], before[1:])


def test_step_extreme_gates():
    """Full decay (g = -inf), no decay, no write, and raw inputs at the ends of the range."""
    q, k, v, g, beta, S, gate, cu = step_inputs([4, 4], 2, 2, 64, 64, torch.float32, False, 14, 2)
    g[0], g[1], beta[1], beta[2] = -float("inf"), 0.0, 0.0, 1.0
    o = torch.zeros(8, 2, 64, device="cuda")
    ro, rS = ref_step(q, k, v, g, beta, S, None, None, cu, None, None, 1.0, o)
    gdn.gdn_step(q, k, v, g, beta, S, cu_seqlens=cu, o=o)
    torch.cuda.synchronize()
    check("o", o, ro, 1e-4, 30.0)
    check("S", S, rS, 1e-4, 30.0)
    q, k, v, g, beta, S, gate, cu = step_inputs([4, 4], 2, 2, 64, 64, torch.float32, True, 15, 2)
    q[0], k[1] = 0.0, 0.0                 # zero rows normalise to zero
    g[2], g[3], beta[2], beta[3] = 200.0, -200.0, 200.0, -200.0
    ro, rS = ref_step(q, k, v, g, beta, S, None, None, cu, None, gate, 1.0, o)
    gdn.gdn_step(q, k, v, g, beta, S, cu_seqlens=cu, gate=gate, o=o)
    torch.cuda.synchronize()
    check("o", o, ro, 1e-4, 30.0)
    check("S", S, rS, 1e-4, 30.0)


def test_step_nan_stays_in_its_head():
    q, k, v, g, beta, S, _, cu = step_inputs([2, 2], 3, 3, 64, 64, torch.float32, False, 16, 2)
    v[0, 1] = float("nan")
    o = gdn.gdn_step(q, k, v, g, beta, S, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert torch.isnan(o[0:2, 1]).all() and torch.isnan(S[0, 1]).all()
    assert torch.isfinite(o[:, [0, 2]]).all() and torch.isfinite(o[2:]).all()
    assert torch.isfinite(S[:, [0, 2]]).all() and torch.isfinite(S[1]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,commit", [(2, 1), (8, 3), (12, 8), (20, 17)])
def test_step_nan_in_a_draft_stays_behind_the_commit(dtype, n, commit):
    """A NaN in what follows the committed tokens reaches neither the cache nor
    the outputs before it."""
    a = step_inputs([n], 2, 2, 64, 64, DT[dtype], False, n, 1)
    q, k, v, g, beta, S, _, cu = a
    S0, sound = S.clone(), [t.clone() for t in (q, k, v, g, beta)]
    want = gdn.gdn_step(*sound, S0, cu_seqlens=cu, n_commit=i32([commit]))
    for t in (q, k, v, g, beta):
        t[commit:] = float("nan")
    o = gdn.gdn_step(q, k, v, g, beta, S, cu_seqlens=cu, n_commit=i32([commit]))
    torch.cuda.synchronize()
    assert torch.equal(S, S0) and torch.equal(o[:commit], want[:commit])
    assert torch.isnan(o[commit:]).all()


@pytest.mark.parametrize("dtype,dk,dv,tol", [("f32", 64, 64, 1e-4), ("bf16", 128, 128, 2e-2),
                                             ("bf16", 128, 256, 2e-2)])
def test_step_continues_a_chunk(dtype, dk, dv, tol):
    """A prompt through gdn_chunk_fwd, then tokens one by one, against the whole
    sequence in one chunk call."""
    from chunked_linear_recurrence_gated_gb300.inputs import make_inputs
    x = make_inputs(2, 75, 4, dk, dv, dtype=DT[dtype], seed=5, device="cuda", decay="weak")
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o_all, S_all = gdn.gdn_chunk_fwd(*a)
    _, S = gdn.gdn_chunk_fwd(*[t[:, :70].contiguous() for t in a])
    outs = [gdn.gdn_step(*[t[:, 70 + i] for t in a], S) for i in range(5)]
    torch.cuda.synchronize()
    err = lambda u, w: float((u.float() - w.float()).abs().max() / w.float().abs().max())
    assert err(torch.stack(outs, 1), o_all[:, 70:]) <= tol
    assert err(S, S_all) <= tol


def test_step_drafts_then_commit_equals_one_by_one():
    """Verified drafts leave the slot alone; passing the accepted ones again,
    committed, gives the bits of having passed them first."""
    q, k, v, g, beta, S, gate, cu = step_inputs([6], 2, 2, 128, 128, torch.bfloat16, True, 21, 1)
    a = (q, k, v, g, beta)
    S0 = S.clone()
    o = gdn.gdn_step(*a, S, cu_seqlens=cu, n_commit=i32([0]), gate=gate)
    assert torch.equal(S, S0)
    o2 = gdn.gdn_step(*a, S, cu_seqlens=cu, n_commit=i32([3]), gate=gate)
    torch.cuda.synchronize()
    assert torch.equal(o, o2)
    S1 = S0.clone()
    o3 = gdn.gdn_step(*[t[:3] for t in a], S1, cu_seqlens=i32([0, 3]), gate=gate)
    torch.cuda.synchronize()
    col = float(S0.norm(dim=-2).max()) + float(v.abs().max())
    assert float((S1 - S).abs().max()) <= 2e-5 * 4 * col
    check("o", o3, np64(o[:3]), 2e-5 * 4 + 2.0 ** -8, col)


def test_step_past_32_bits():
    """Slots whose offsets pass 2^31 elements."""
    n_slots, H, dk, dv = 140, 128, 128, 1
    slots = 2 ** 31 // (64 * 128 * 256) + 3
    S = torch.zeros(slots, 64, 128, 256, device="cuda")
    r = gen(31)
    last = slots - 1
    S[last] = r(64, 128, 256)
    q, k, v = r(1, 64, 128), r(1, 64, 128), r(1, 64, 256)
    q, k = (torch.nn.functional.normalize(t, dim=-1) for t in (q, k))
    g, beta = -torch.rand(1, 64, device="cuda"), torch.rand(1, 64, device="cuda")
    S0 = S[last:].clone()
    o = gdn.gdn_step(q, k, v, g, beta, S, i32([last]), i32([last]))
    torch.cuda.synchronize()
    ro, rS = lo.step(*[np64(t) for t in (q, k, v, g, beta, S0)])
    col = float(S0.norm(dim=-2).max()) + 5.0
    check("o", o, ro, 4e-5, col)
    check("S", S[last:], rS, 4e-5, col)
    assert not S[:last].any()


# ------------------------------------------------------------- conv over a cache
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4, 8])
@pytest.mark.parametrize("act", ["silu", "none"])
def test_conv_step(dtype, W, act):
    for C, pad in ((44, 4), (512, 0), (1032, 16), (8, 8)):
        r = gen(W + C)
        lens = [1, 5, 0, 0, 9, 2, 3]
        x = r(sum(lens), C + pad, dtype=DT[dtype])[:, pad // 4 * 4:][:, :C]
        w, b, state = r(C, W, by=W ** -0.5), r(C), r(9, W - 1, C, dtype=DT[dtype])
        si, so, commit = [0, 1, 2, 3, -1, 5, 77], [0, 1, 2, 4, 7, 8, -1], [1, 2, 0, 0, 9, 0, 3]
        cu = np.concatenate([[0], np.cumsum(lens)])
        b = b if act == "silu" else None
        ry, rs = lo.conv_step(np64(x), np64(w), 0.0 if b is None else np64(b), np64(state), si, so,
                              cu, commit, act)
        y = gdn.gdn_conv_step(x, w, b, state, i32(si), i32(so), i32(cu), i32(commit), act=act)
        torch.cuda.synchronize()
        check("y", y, ry, 1e-5)
        assert np.array_equal(np64(state), rs)


def test_conv_step_one_token_each():
    r = gen(3)
    x, w, b, state = r(37, 96), r(96, 4), r(96), r(40, 3, 96)
    ry, rs = lo.conv_step(np64(x), np64(w), np64(b), np64(state))
    y = gdn.gdn_conv_step(x, w, b, state)
    torch.cuda.synchronize()
    check("y", y, ry, 1e-5)
    assert np.array_equal(np64(state), rs)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W", [5, 6, 7])
def test_conv_step_other_widths(dtype, W):
    r = gen(40 + W)
    lens = [0, 1, 3, 4, 5, 6, 7, 8, 12]
    n, C = sum(lens), 68
    x, w, b = r(n, C, dtype=DT[dtype]), r(C, W, by=W ** -0.5), r(C)
    state = r(len(lens), W - 1, C, dtype=DT[dtype])
    commit = [0, 1, 2, 4, 0, 5, 7, 3, 12]
    cu = np.concatenate([[0], np.cumsum(lens)])
    ry, rs = lo.conv_step(np64(x), np64(w), np64(b), np64(state), cu=cu, commit=commit)
    y = gdn.gdn_conv_step(x, w, b, state, cu_seqlens=i32(cu), n_commit=i32(commit))
    torch.cuda.synchronize()
    check("y", y, ry, 1e-5)
    assert np.array_equal(np64(state), rs)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_conv_step_many_sequences(dtype):
    """More sequences than threads per channel: each takes several, loads of the next in flight."""
    r, rng = gen(5), np.random.default_rng(5)
    N, C = 1300, 4096
    lens = rng.integers(0, 8, N)
    commit = np.minimum(rng.integers(0, 8, N), lens)
    x, w, b = r(int(lens.sum()), C, dtype=DT[dtype]), r(C, 4, by=0.5), r(C)
    state = r(N + 3, 3, C, dtype=DT[dtype])
    si = rng.permutation(N + 3)[:N]
    cu = np.concatenate([[0], np.cumsum(lens)])
    ry, rs = lo.conv_step(np64(x), np64(w), np64(b), np64(state), si, si, cu, commit)
    y = gdn.gdn_conv_step(x, w, b, state, i32(si), i32(si), i32(cu), i32(commit))
    torch.cuda.synchronize()
    check("y", y, ry, 1e-5)
    assert np.array_equal(np64(state), rs)


def test_conv_step_continues_a_chunk():
    r = gen(4)
    x, w, b = r(2, 20, 64), r(64, 4), r(64)
    y_all, s_all = gdn.gdn_conv_fwd(x, w, b)
    _, s = gdn.gdn_conv_fwd(x[:, :15].contiguous(), w, b)
    ys = [gdn.gdn_conv_step(x[:, 15 + i], w, b, s) for i in range(5)]
    torch.cuda.synchronize()
    assert torch.equal(s, s_all)
    check("y", torch.stack(ys, 1), np64(y_all[:, 15:]), 1e-5)


# -------------------------------------------------------- maps of the recurrence
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("B,T,H,Hk", [(1, 1, 1, 1), (2, 37, 6, 2), (1, 300, 40, 40), (3, 65, 35, 5),
                                      (1, 3001, 4, 1)])
def test_prep(dtype, dk, B, T, H, Hk):
    dt = DT[dtype]
    r = gen(T + H)
    qk = r(B, T, 2 * Hk * dk, dtype=dt)
    q, k = (qk[..., i * Hk * dk:(i + 1) * Hk * dk].unflatten(2, (Hk, dk)) for i in range(2))
    gates = r(B, T, 2 * H + 1, dtype=dt, by=2.0)
    xg, xb = gates[..., :H], gates[..., H:2 * H]
    q[0, 0] = 0.0                         # a zero row
    rate, bias = r(H, by=0.5), r(H)
    d = r(B, T, H, dk, dtype=dt), r(B, T, H, dk, dtype=dt), r(B, T, H, dtype=dt), r(B, T, H, dtype=dt)
    if dtype == "f32":
        xg[0, 0, 0], xb[0, 0, 0] = 100.0, -100.0
    a = [np64(t) for t in (q, k, xg, xb, rate, bias)]
    got = gdn.gdn_prep_fwd(q, k, xg, xb, rate, bias, q_scale=0.3)
    for name, u, ref in zip(("q", "k", "g", "beta"), got, lo.prep_fwd(*a, q_scale=0.3)):
        check(name, u, ref, 1e-5)
    got = gdn.gdn_prep_bwd(q, k, xg, xb, rate, bias, *d, q_scale=0.3)
    again = gdn.gdn_prep_bwd(q, k, xg, xb, rate, bias, *d, q_scale=0.3)
    torch.cuda.synchronize()
    ref, mags = lo.prep_bwd(*a, *[np64(t) for t in d], q_scale=0.3)
    # the zero row's gradient is of order 1 / sqrt(eps): compared by itself
    check("dq", got[0].flatten(0, 1)[1:], ref[0].reshape(B * T, Hk, dk)[1:], 5e-5)
    check("dq zero row", got[0][0, 0], ref[0][0, 0], 5e-5)
    for i, name in ((1, "dk"), (2, "dxg"), (3, "dxb")):
        check(name, got[i], ref[i], 5e-5)
    check("drate", got[4], ref[4], 2e-5, mags[0])
    check("dbias", got[5], ref[5], 2e-5, mags[1])
    for u, v in zip(got, again):
        assert torch.equal(u, v)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prep_many_tokens(dtype):
    """Several tokens of a head to a thread in the gates' backward."""
    test_prep(dtype, 64, 1, 6007, 35, 5)


# --------------------------------------------------------------------- gated norm
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("B,T,H,d,pad", [(1, 1, 1, 128, 0), (2, 33, 3, 64, 8), (1, 129, 5, 256, 64),
                                         (1, 50, 2, 8, 0), (3, 7, 2, 104, 8), (1, 40, 1, 200, 0),
                                         (2, 700, 4, 128, 0)])
def test_gate_norm(dtype, act, B, T, H, d, pad):
    dt = DT[dtype]
    r = gen(T + d)
    o, dy, w = r(B, T, H, d, dtype=dt, by=0.3), r(B, T, H, d, dtype=dt), 1.0 + r(d, by=0.2)
    z = r(B, T, H * d + pad, dtype=dt, by=2.0)[..., pad:].unflatten(2, (H, d))
    o[0, 0, 0] = 0.0                      # a row of zeros
    z[0, 0, 0, 0], z[0, 0, 0, 1] = 200.0, -200.0
    a = [np64(t) for t in (o, z, w)]
    y = gdn.gdn_gate_norm_fwd(o, z, w, act)
    got = gdn.gdn_gate_norm_bwd(o, z, w, dy, act)
    again = gdn.gdn_gate_norm_bwd(o, z, w, dy, act)
    torch.cuda.synchronize()
    check("y", y, lo.gate_norm_fwd(*a, act), 1e-5)
    ref, mag = lo.gate_norm_bwd(*a, np64(dy), act)
    rows = lambda t: t.reshape(-1, d)[1:]
    check("do", rows(got[0]), rows(ref[0]), 5e-5)
    check("do zero row", got[0][0, 0, 0], ref[0][0, 0, 0], 5e-5)
    check("dz", got[1], ref[1], 5e-5)
    check("dw", got[2], ref[2], 2e-5, mag)
    for u, v in zip(got, again):
        assert torch.equal(u, v)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,H,d", [(2, 9000, 3, 128), (1, 7001, 4, 256), (1, 9001, 8, 56)])
def test_gate_norm_many_rows(dtype, B, T, H, d):
    """More rows than the backward's blocks take at a time."""
    test_gate_norm(dtype, "silu", B, T, H, d, 8)


# ----------------------------------------------------------------- block boundary
@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("scale", [False, True])
@pytest.mark.parametrize("rows,C", [(1, 128), (5, 8), (37, 264), (700, 1000), (3, 2048), (9, 4104),
                                    (2, 5120), (3, 8192), (2, 16384)])
def test_res_norm(types, post, scale, rows, C):
    dt, rt = DT[types[0]], DT[types[1]]
    r = gen(rows + C)
    h, x, w = r(rows, C, dtype=rt), r(rows, C, dtype=dt, by=0.5), 1.0 + r(C, by=0.2)
    wp = 1.0 + r(C, by=0.2) if post else None
    sc = 0.5 + r(C, by=0.1) if scale else None
    dy, dh = r(rows, C, dtype=dt), r(rows, C, dtype=rt)
    f = lambda t: None if t is None else np64(t)
    ho, y = gdn.gdn_res_norm_fwd(h, x, w, wp, sc)
    rh, ry = lo.res_norm_fwd(f(h), f(x), f(w), f(wp), f(sc))
    check("h", ho, rh, 1e-5)
    check("y", y, ry, 1e-5)
    for up in (dh, None):
        got = gdn.gdn_res_norm_bwd(ho, x, w, dy, up, wp, sc)
        again = gdn.gdn_res_norm_bwd(ho, x, w, dy, up, wp, sc)
        torch.cuda.synchronize()
        ref, mags = lo.res_norm_bwd(f(ho), f(x), f(w), f(dy), f(up), f(wp), f(sc))
        for name, u, v in zip(("dh", "dx"), got, ref):
            check(name, u, v, 5e-5)
        for name, u, v, m in zip(("dw", "dw_post", "dscale"), got[2:], ref[2:], mags):
            assert (u is None) == (v is None)
            check(name, u, v, 2e-5, m)
        for u, v in zip(got, again):
            assert u is None or torch.equal(u, v)


@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("post,scale", [(False, False), (True, True)])
@pytest.mark.parametrize("rows,C", [(613, 4104), (501, 7000), (403, 8200), (307, 16376), (306, 16384)])
def test_res_norm_many_split_rows(types, post, scale, rows, C):
    """Rows split over CTAs of a cluster, several to each."""
    test_res_norm(types, post, scale, rows, C)


def test_res_norm_in_place_and_without_a_block():
    r = gen(8)
    h, x, w, dy, dh = r(40, 512), r(40, 512), r(512), r(40, 512), r(40, 512)
    ho, y = gdn.gdn_res_norm_fwd(h, x, w)
    h2 = h.clone()
    ho2, y2 = gdn.gdn_res_norm_fwd(h2, x, w, h_out=h2)
    assert ho2 is h2
    none, y3 = gdn.gdn_res_norm_fwd(ho, None, w)
    y4 = gdn.gdn_res_norm_fwd(ho, None, w, dtype=torch.bfloat16)[1]
    a = gdn.gdn_res_norm_bwd(ho, x, w, dy, dh)
    d2 = dh.clone()
    b = gdn.gdn_res_norm_bwd(ho, None, w, dy, d2, dh=d2)
    torch.cuda.synchronize()
    assert torch.equal(ho, h2) and torch.equal(y, y2) and none is None and torch.equal(y, y3)
    assert torch.equal(y4, y3.to(torch.bfloat16))
    assert a[1] is a[0] and b[0] is d2
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


# ------------------------------------------------------------------ common ground
def test_no_tokens():
    e = lambda *s: torch.empty(*s, device="cuda")
    one = torch.ones(64, device="cuda")
    assert gdn.gdn_step(e(0, 2, 64), e(0, 2, 64), e(0, 2, 64), e(0, 2), e(0, 2), e(1, 2, 64, 64)).shape[0] == 0
    assert gdn.gdn_conv_step(e(0, 8), torch.ones(8, 4, device="cuda"), None, e(1, 3, 8)).shape == (0, 8)
    out = gdn.gdn_prep_bwd(e(1, 0, 2, 64), e(1, 0, 2, 64), e(1, 0, 2), e(1, 0, 2), one[:2], one[:2],
                           e(1, 0, 2, 64), e(1, 0, 2, 64), e(1, 0, 2), e(1, 0, 2))
    assert gdn.gdn_prep_fwd(e(1, 0, 2, 64), e(1, 0, 2, 64), e(1, 0, 2), e(1, 0, 2), one[:2], one[:2])[0].numel() == 0
    dw = gdn.gdn_gate_norm_bwd(e(1, 0, 1, 64), e(1, 0, 1, 64), one, e(1, 0, 1, 64))[2]
    assert gdn.gdn_gate_norm_fwd(e(1, 0, 1, 64), e(1, 0, 1, 64), one).numel() == 0
    r = gdn.gdn_res_norm_bwd(e(0, 64), e(0, 64), one, e(0, 64), None, one, one)
    assert gdn.gdn_res_norm_fwd(e(0, 64), e(0, 64), one)[1].numel() == 0
    torch.cuda.synchronize()
    for t in (out[4], out[5], dw, *r[2:]):
        assert not t.any()


def test_other_stream():
    """Work on a stream of the caller's: ordered with that stream, its workspace too."""
    r = gen(9)
    o, z, w, dy = r(1, 4096, 8, 128), r(1, 4096, 8, 128), r(128), r(1, 4096, 8, 128)
    ref = gdn.gdn_gate_norm_bwd(o, z, w, dy)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    outs = [gdn.gdn_gate_norm_bwd(o, z, w, dy, stream=s) for s in (st, st.cuda_stream)]
    junk = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(4)]
    st.synchronize()
    for got in outs:
        for u, v in zip(ref, got):
            assert torch.equal(u, v)
    del junk


def test_captured_in_a_graph():
    r = gen(10)
    q, k, v, g, beta = r(3, 2, 64), r(3, 2, 64), r(3, 4, 64), r(3, 4), r(3, 4)
    gate, S = (r(4), r(4)), r(3, 4, 64, 64)
    S0 = S.clone()
    want = gdn.gdn_step(q, k, v, g, beta, S, gate=gate)
    torch.cuda.synchronize()
    S1 = S.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = gdn.gdn_step(q, k, v, g, beta, S, gate=gate)
    S.copy_(S0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(S, S1)


@pytest.mark.parametrize("N", [1, 200])
def test_dependent_calls_back_to_back(N):
    """A call may be launched before its predecessor has ended: calls that read, and
    write over, what the one before has just written or read give the same bits as
    with a synchronisation after each."""
    def run(wait):
        r = gen(11)
        wait = torch.cuda.synchronize if wait else (lambda: None)
        cw, cb, conv = r(512, 4), r(512), r(N, 3, 512)
        S, gates, gate = r(N, 4, 64, 64), (r(N, 4), r(N, 4)), (r(4), r(4))
        wn, w, wp = r(64), r(256), r(256)
        x, z, h = r(N, 512), r(1, N, 4, 64), r(N, 256)
        dy, kept = r(1, N, 4, 64), []
        for _ in range(20):
            y = gdn.gdn_conv_step(x, cw, cb, conv)
            wait()
            q, k, v = (u.unflatten(-1, (-1, 64)) for u in y.split((128, 128, 256), -1))
            o = gdn.gdn_step(q, k, v, *gates, S, gate=gate)
            wait()
            z = gdn.gdn_gate_norm_fwd(o[None], z, wn)
            wait()
            h, z = gdn.gdn_res_norm_fwd(h, z.view(N, 256), w, w_post=wp)
            wait()
            z = z.view(1, N, 4, 64)
            do, dz, dw = gdn.gdn_gate_norm_bwd(o[None], z, wn, dy)
            wait()
            dx = gdn.gdn_res_norm_bwd(h, do.view(N, 256), w, dz.view(N, 256), w_post=wp)
            wait()
            dy = dx[0].view(1, N, 4, 64)
            kept += [o, z, dw, dx[2]]
        torch.cuda.synchronize()
        return kept + [S, conv, h, dy]

    for a, b in zip(run(True), run(False)):
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))
