"""GPU parity of linear attention with a decay for each head (include/gdn_lin.h) and of
the query / key norms with the rotation (gdn_qk_norm_*) against their fp64 oracle, at
the sizes, strides and masks where they can go wrong.

Tolerances. Every result is a sum of products; A is the same sum over the terms'
magnitudes (the oracle on absolute values), so a relative error e of any factor moves
the result by at most e A. fp32: two TF32 parts hold an operand to 2^-23, the product
of the second parts that is left out is 2^-22, a decay factor is good to 2^-21, and the
at most 128 / 8 + 64 / 8 accumulating steps of a tensor-core product and the state's
multiply-adds over the chunks round by 2^-23 each: below 2^-17 A in all. bf16: the
results that stay on the tensor cores round one factor of each term to bf16 once (a
masked product, or the state as an operand): 2^-8 A; the stored value rounds by another
2^-8 of itself. fp32 results of bf16 calls (states) take operands of two bf16 parts: a
weight w is held as wh + wl to 2^-16; of y w the first part is y wh rounded, and the rest,
y wl + (y wh - first), at most 2 2^-8 |y w|, is rounded by 2^-8 of itself, 2^-15; together
3 2^-16 A. Norms: values to 1e-5 of max|ref| (statistics of at most 256 terms in short
chains), parameter sums to 2e-5 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

from chunked_linear_recurrence_gated_gb300 import gdn
from helpers import np64
from oracle import lin_ops as lo

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = 2.0 ** -8  # unit roundoff of bf16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s, dtype=torch.float32, by=1.0: (
        torch.randn(*s, generator=g, device="cuda") * by).to(dtype)


def check(name, got, ref, tol):
    ref = np.asarray(ref, dtype=np.float64)
    assert tuple(got.shape) == ref.shape, (name, got.shape, ref.shape)
    tol = tol + 1e-30 + (HALF * np.abs(ref) if got.dtype == torch.bfloat16 else 0.0)
    off = np.abs(np64(got) - ref) - tol
    assert not (off > 0).any() and not np.isnan(off).any(), (name, off.max(), np.abs(ref).max())


def state_tol(dtype):
    return 2.0 ** -17 if dtype == torch.float32 else 3 * 2.0 ** -16


def value_tol(dtype):
    return 2.0 ** -17 if dtype == torch.float32 else HALF


# ------------------------------------------------------------- whole sequences
def lin_inputs(B, T, H, dk, dv, dtype, decay="mid", seed=0, nseq=None):
    r = gen(seed)
    qkv = r(B, T, H * (2 * dk + dv) + 8, dtype=dtype)  # one strided row for each token
    q, k = (qkv[..., i * H * dk:(i + 1) * H * dk].unflatten(2, (H, dk)) for i in range(2))
    v = qkv[..., 2 * H * dk:2 * H * dk + H * dv].unflatten(2, (H, dv))
    by = {"none": 0.0, "weak": 0.01, "mid": 0.3, "strong": 20.0}
    if decay in by:
        g = (-r(B, T, H + 3).abs() * by[decay]).to(dtype)[..., 1:1 + H]
    elif decay == "mixed":  # all of these in one sequence, and the state forgotten at times
        w = torch.tensor([0.0, 0.01, 0.5, 40.0], device="cuda")
        g = -r(B, T, H).abs() * w[torch.arange(T, device="cuda") * 7 % 4][None, :, None]
        g[:, 3::29] = -float("inf")
        g = g.to(dtype)
    else:  # one for each head
        g = -torch.exp(-1.5 * torch.arange(H, device="cuda", dtype=torch.float32))
    n = nseq or B
    return dict(q=q, k=k, v=v, g=g, S=r(n, H, dk, dv), do=r(B, T, H, dv, dtype=dtype),
                dS=r(n, H, dk, dv))


def host(*ts):
    return [None if t is None else np64(t) for t in ts]


def against_oracle(x, scale=1.0, cu=None, states=True, want=("fwd", "bwd")):
    dtype = x["q"].dtype
    S, dS = (x["S"], x["dS"]) if states else (None, None)
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    n = [np64(x[i]) for i in "qkvg"]
    a = [np.abs(t) for t in n[:3]] + [n[3]]
    St, dSt, do = host(S, dS, x["do"])
    mags = [None if t is None else np.abs(t) for t in (St, dSt, do)]
    rows = np.zeros(x["q"].shape[:2], dtype=bool)  # that belong to a sequence
    for t0, t1 in lo._spans(x["q"].shape[1], x["q"].shape[0], cu):
        rows.reshape(-1)[t0:t1] = True
    with np.errstate(invalid="ignore"):
        if "fwd" in want:
            o, end = gdn.gdn_lin_fwd(x["q"], x["k"], x["v"], x["g"], S, scale=scale, cu_seqlens=cud)
            ro, rend = lo.lin_fwd(*n, St, scale, cu)
            ao, aend = lo.lin_fwd(*a, mags[0], abs(scale), cu)
            check("o", o[torch.tensor(rows, device="cuda")], ro[rows], value_tol(dtype) * ao[rows])
            check("S_out", end, rend, state_tol(dtype) * aend)
        if "bwd" in want:
            got = gdn.gdn_lin_bwd(x["q"], x["k"], x["v"], x["g"], S, x["do"], dS, scale=scale,
                                  cu_seqlens=cud)
            ref = lo.lin_bwd(*n, St, do, dSt, scale, cu)
            mag = lo.lin_bwd(*a, mags[0], mags[2], mags[1], abs(scale), cu)
            for i, name in enumerate(("dq", "dk", "dv")):
                at = torch.tensor(rows, device="cuda")
                check(name, got[i][at], ref[i][rows], value_tol(dtype) * mag[i][rows])
            if x["g"].dim() == 1:
                check("dg", got[3], ref[3].sum((0, 1)), value_tol(dtype) * mag[3].sum((0, 1)))
            else:
                check("dg", got[3][torch.tensor(rows, device="cuda")], ref[3][rows],
                      dg_tol(dtype, mag[3], cu)[rows])
            check("dS_in", got[4], ref[4], state_tol(dtype) * mag[4])
    return got if "bwd" in want else None


def dg_tol(dtype, mag, cu):
    """A token's dg is joined from sums over its chunk, whose terms' magnitudes are those
    of the pairs across some token of the chunk: at most the largest dg magnitudes near it."""
    B, T, H = mag.shape
    near = np.zeros_like(mag)
    for t in range(T):
        near[:, t] = mag[:, max(0, t - 128):t + 128].max(1)
    return value_tol(dtype) * near


DIMS = [(64, 64), (64, 128), (128, 64), (128, 128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("T", [1, 63, 130])
def test_lin_sizes(dtype, dk, dv, T):
    against_oracle(lin_inputs(2, T, 3, dk, dv, DT[dtype], seed=T + dk), scale=dk ** -0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [2, 64, 65, 127, 128, 129, 192, 257])
def test_lin_lengths(dtype, T):
    against_oracle(lin_inputs(1, T, 1, 128, 128, DT[dtype], seed=T), scale=0.3, states=T % 2 == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", ["none", "weak", "strong", "mixed", "head"])
def test_lin_decays(dtype, decay):
    against_oracle(lin_inputs(1, 300, 2, 128, 64, DT[dtype], decay, seed=5), scale=-0.2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cu", [[0, 200], [0, 0, 1, 65, 193, 193, 300, 321], [5, 6, 70, 200],
                                [0] * 9, [7, 7, 7, 135, 320]])
@pytest.mark.parametrize("decay", ["mid", "head"])
def test_lin_packed(dtype, cu, decay):
    x = lin_inputs(1, 321, 2, 64, 128, DT[dtype], decay, seed=len(cu), nseq=len(cu) - 1)
    against_oracle(x, scale=0.25, cu=cu, states=len(cu) % 2 == 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lin_packed_neighbours_do_not_leak(dtype):
    """NaN and infinities in rows of no sequence and of the next one stay there; rows of no
    sequence are left as they were."""
    cu = [3, 100, 100, 230]
    x = lin_inputs(1, 300, 2, 128, 128, DT[dtype], seed=3, nseq=3)
    for i in ("q", "k", "v", "g", "do"):
        x[i][:, :3] = float("nan")
        x[i][:, 230:] = float("inf")
    d = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o = torch.full((1, 300, 2, 128), 7.0, dtype=DT[dtype], device="cuda")
    gdn.gdn_lin_fwd(x["q"], x["k"], x["v"], x["g"], x["S"], cu_seqlens=d, o=o)
    assert (o[:, :3] == 7).all() and (o[:, 230:] == 7).all()
    against_oracle(x, cu=cu)
    x["v"][:, 100:] = float("nan")  # the last sequence: the others are as before
    a = gdn.gdn_lin_fwd(x["q"], x["k"], x["v"], x["g"], x["S"], cu_seqlens=d)
    assert torch.equal(a[0][:, 3:100], o[:, 3:100]) and not a[1][:2].isnan().any()
    assert a[1][2].isnan().any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cu", [[0, 10, 5, 20], [-1, 10, 20, 30], [0, 10, 20, 41], [0, 40, 0, 40]])
def test_lin_malformed_offsets_are_reported(dtype, cu):
    x = lin_inputs(1, 40, 2, 64, 64, DT[dtype], "head", nseq=3)
    d = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o = torch.full((1, 40, 2, 64), 7.0, dtype=DT[dtype], device="cuda")
    S = torch.full((3, 2, 64, 64), 5.0, device="cuda")
    ws = gdn.alloc_workspace(1 << 24, "cuda")
    gdn.gdn_lin_fwd(x["q"], x["k"], x["v"], x["g"], x["S"], cu_seqlens=d, o=o, S_out=S, workspace=ws)
    assert gdn.gdn_workspace_status(ws) == 1
    assert (o == 7).all() and (S == 5).all()
    r = gdn.gdn_lin_bwd(x["q"], x["k"], x["v"], x["g"], x["S"], x["do"], x["dS"], cu_seqlens=d,
                        workspace=ws)
    assert gdn.gdn_workspace_status(ws) == 1
    assert (r[3] == 0).all()
    gdn.gdn_lin_fwd(x["q"], x["k"], x["v"], x["g"], x["S"][:1], workspace=ws)
    assert gdn.gdn_workspace_status(ws) == 0


def test_lin_no_tokens():
    for dtype in DT.values():
        x = lin_inputs(2, 0, 2, 64, 128, dtype, "head")
        o, S = gdn.gdn_lin_fwd(x["q"], x["k"], x["v"], x["g"], x["S"])
        assert o.shape == (2, 0, 2, 128) and torch.equal(S, x["S"])
        r = gdn.gdn_lin_bwd(x["q"], x["k"], x["v"], x["g"], x["S"], x["do"], x["dS"])
        assert torch.equal(r[4], x["dS"]) and (r[3] == 0).all()
        assert (gdn.gdn_lin_fwd(x["q"], x["k"], x["v"], x["g"])[1] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lin_chunks_chain(dtype):
    """Chunks linked by their boundary state and its gradient against the whole sequence."""
    dt = DT[dtype]
    x = lin_inputs(1, 500, 2, 128, 128, dt, "weak", seed=9)
    cuts = [0, 128, 129, 400, 500]
    S, outs, ins = x["S"], [], []
    for a, b in zip(cuts, cuts[1:]):
        ins.append(S)
        o, S = gdn.gdn_lin_fwd(*(x[i][:, a:b] for i in "qkvg"), S, scale=0.1)
        outs.append(o)
    n = [np64(x[i]) for i in "qkvg"]
    mag = [np.abs(t) for t in n[:3]] + [n[3]]
    St, dSt, do = host(x["S"], x["dS"], x["do"])
    ro, rS = lo.lin_fwd(*n, St, 0.1)
    ao, aS = lo.lin_fwd(*mag, np.abs(St), 0.1)
    check("o", torch.cat(outs, 1), ro, value_tol(dt) * ao)
    check("S", S, rS, len(cuts) * state_tol(dt) * aS)
    dS, parts = x["dS"], []
    for (a, b), s in reversed(list(zip(zip(cuts, cuts[1:]), ins))):
        r = gdn.gdn_lin_bwd(*(x[i][:, a:b] for i in "qkvg"), s, x["do"][:, a:b].contiguous(), dS,
                            scale=0.1)
        dS = r[4]
        parts.insert(0, r[:4])
    ref = lo.lin_bwd(*n, St, do, dSt, 0.1)
    am = lo.lin_bwd(*mag, np.abs(St), np.abs(do), np.abs(dSt), 0.1)
    for i, name in enumerate(("dq", "dk", "dv")):
        check(name, torch.cat([p[i] for p in parts], 1), ref[i], 1.1 * value_tol(dt) * am[i])
    check("dg", torch.cat([p[3] for p in parts], 1), ref[3], 1.1 * dg_tol(dt, am[3], None))
    check("dS_in", dS, ref[4], len(cuts) * state_tol(dt) * am[4])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,H", [(1, 3001, 1), (3, 1500, 2), (1, 1100, 33), (70, 40, 3)])
def test_lin_long(dtype, B, T, H):
    against_oracle(lin_inputs(B, T, H, 64, 64, DT[dtype], "weak", seed=T), scale=0.125)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lin_states_in_place_and_repeatable(dtype):
    x = lin_inputs(2, 200, 2, 128, 128, DT[dtype], "head")
    a = [x[i] for i in "qkvg"]
    o, S = gdn.gdn_lin_fwd(*a, x["S"])
    S2 = x["S"].clone()
    o2, same = gdn.gdn_lin_fwd(*a, S2, S_out=S2)
    assert torch.equal(o, o2) and torch.equal(S, S2) and same.data_ptr() == S2.data_ptr()
    r = gdn.gdn_lin_bwd(*a, x["S"], x["do"], x["dS"])
    for _ in range(3):
        r2 = gdn.gdn_lin_bwd(*a, x["S"], x["do"], x["dS"])
        assert all(torch.equal(i, j) for i, j in zip(r, r2))
    assert gdn.gdn_lin_fwd(*a, x["S"], want_state=False)[1] is None
    assert gdn.gdn_lin_bwd(*a, x["S"], x["do"], x["dS"], want_state=False)[4] is None


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("packed", [False, True])
def test_lin_states_in_place_over_many_units(dtype, packed):
    """A sequence that many CTAs share, its last state written where its first one is read."""
    T, H = 9001, 20
    x = lin_inputs(1, T, H, 64, 64, DT[dtype], "weak", seed=5)
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda") if packed else None
    a = [x[i] for i in "qkvg"]
    o, S = gdn.gdn_lin_fwd(*a, x["S"], cu_seqlens=cu)
    want = gdn.gdn_lin_bwd(*a, x["S"], x["do"], x["dS"], cu_seqlens=cu)
    sh = gdn.gdn_lin_shape(1, T, H, 64, 64, 0 if dtype == "f32" else 1, 1, *(t.stride(1) for t in a), 1.0)
    lib, p = gdn.load(), lambda t: None if t is None else t.data_ptr()
    for _ in range(5):
        S2 = x["S"].clone()
        o2, _ = gdn.gdn_lin_fwd(*a, S2, S_out=S2, cu_seqlens=cu)
        assert torch.equal(o, o2) and torch.equal(S, S2)
        dS = x["dS"].clone()
        got = [torch.full_like(t, float("nan")) for t in want[:4]]
        ws = torch.empty(lib.gdn_lin_workspace_bytes(sh, 1), dtype=torch.uint8, device="cuda")
        assert lib.gdn_lin_bwd(sh, *map(p, a), None, p(x["S"]), p(cu), p(x["do"]), p(dS), *map(p, got),
                               None, p(dS), p(ws), ws.numel(),
                               torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert all(torch.equal(i, j) for i, j in zip(want, got + [dS]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lin_on_another_stream_and_in_a_graph(dtype):
    x = lin_inputs(1, 700, 2, 128, 64, DT[dtype], seed=21)
    a = [x[i] for i in "qkvg"]
    want = gdn.gdn_lin_fwd(*a, x["S"]), gdn.gdn_lin_bwd(*a, x["S"], x["do"], x["dS"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = (gdn.gdn_lin_fwd(*a, x["S"], stream=s),
           gdn.gdn_lin_bwd(*a, x["S"], x["do"], x["dS"], stream=s))
    torch.cuda.synchronize()
    for w, r in zip(want, got):
        assert all(torch.equal(i, j) for i, j in zip(w, r))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gdn.gdn_lin_fwd(*a, x["S"]), gdn.gdn_lin_bwd(*a, x["S"], x["do"], x["dS"])
    for i in range(2):
        for t in (*got[0], *got[1]):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for w, r in zip(want, got):
            assert all(torch.equal(i, j) for i, j in zip(w, r))


# -------------------------------------------------------------- token by token
def step_case(lens, H, Hk, dk, dv, dtype, const, seed, slots, most_commit=None):
    r = gen(seed)
    n = sum(lens)
    qkv = r(n, 2 * Hk * dk + H * dv + 16, dtype=dtype)
    q, k = (qkv[:, i * Hk * dk:(i + 1) * Hk * dk].unflatten(1, (Hk, dk)) for i in range(2))
    v = qkv[:, 2 * Hk * dk:2 * Hk * dk + H * dv].unflatten(1, (H, dv))
    g = -r(H).abs() if const else (-r(n, H + 1).abs()).to(dtype)[:, 1:]
    return q, k, v, g, r(slots, H, dk, dv)


def step_check(args, dtype, lens, scale=1.0, **kw):
    q, k, v, g, S = args
    up = {x: (None if y is None else torch.tensor(y, dtype=torch.int32, device="cuda"))
          for x, y in kw.items()}
    cache = S.clone()
    o = torch.full(v.shape, 7.0, dtype=dtype, device="cuda")
    names = dict(slot_in="slot_in", slot_out="slot_out", cu="cu_seqlens", commit="n_commit")
    gdn.gdn_lin_step(q, k, v, g, cache, scale=scale, o=o, **{names[x]: y for x, y in up.items()})
    n = host(q, k, v, g, S)
    old = np.full(v.shape, 7.0)
    ro, rS = lo.lin_step(*n, scale=scale, o=old, **kw)
    a = [np.abs(t) for t in n[:3]] + [n[3], np.abs(n[4])]
    ao, aS = lo.lin_step(*a, scale=abs(scale), o=old * 0, **kw)
    # a token's multiply-adds and its factor e^g round by 2^-24 and 2^-22; a dot product
    # of 128 terms in chains of at most 32 and a tree
    tol = 2.0 ** -22 * (8 + max(lens, default=0))
    check("o", o, ro, tol * ao)
    check("S", cache, rS, tol * aS)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("H,Hk,N", [(4, 4, 1), (6, 2, 5), (3, 1, 2)])
@pytest.mark.parametrize("const", [False, True])
def test_lin_step_one_token(dtype, dk, dv, H, Hk, N, const):
    a = step_case([1] * N, H, Hk, dk, dv, DT[dtype], const, N + dk, N + 2)
    step_check(a, DT[dtype], [1], scale=0.3)
    step_check(a, DT[dtype], [1], slot_in=[N + 1] + [-1] * (N - 1),
               slot_out=list(range(1, N + 1)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,commit", [
    ([3, 0, 1, 8, 9], None), ([3, 0, 1, 8, 9], [0, 0, 1, 3, 9]), ([17, 2, 33], [16, 1, 8]),
    ([0, 0], [0, 0]), ([4, 5, 6], [9, -1, 0])])
def test_lin_step_tokens(dtype, lens, commit):
    N = len(lens)
    a = step_case(lens, 4, 2, 128, 128, DT[dtype], N % 2 == 0, N, 2 * N)
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    step_check(a, DT[dtype], lens, cu=cu, commit=commit)
    step_check(a, DT[dtype], lens, cu=cu, commit=commit, slot_in=[-1] + [99] * (N - 2) + [1],
               slot_out=[2 * N - 1] + [-5] * (N - 2) + [0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lin_step_bad_offsets_and_rows_behind(dtype):
    a = step_case([12], 2, 2, 64, 64, DT[dtype], False, 8, 4)
    step_check(a, DT[dtype], [4], cu=[0, 4, 2, 13])   # decreasing, and past the end
    step_check(a, DT[dtype], [4], cu=[-3, 2, 6])
    step_check(a, DT[dtype], [4], cu=[0, 4, 7])       # rows 7.. belong to no sequence


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lin_step_rejected_tokens_leave_no_trace(dtype):
    dt = DT[dtype]
    q, k, v, g, S = step_case([12, 3], 2, 1, 128, 64, dt, False, 5, 2)
    for x in (q, k, v, g):
        x[4:12] = float("nan")
    cache = S.clone()
    cu = torch.tensor([0, 12, 15], dtype=torch.int32, device="cuda")
    c = torch.tensor([4, 3], dtype=torch.int32, device="cuda")
    o = gdn.gdn_lin_step(q, k, v, g, cache, cu_seqlens=cu, n_commit=c)
    assert not cache.isnan().any() and not o[:4].isnan().any() and not o[12:].isnan().any()
    keep = torch.cat([torch.arange(4), torch.arange(12, 15)]).cuda()
    S2 = S.clone()
    o2 = gdn.gdn_lin_step(*(x[keep] for x in (q, k, v, g)), S2,
                          cu_seqlens=torch.tensor([0, 4, 7], dtype=torch.int32, device="cuda"))
    assert torch.equal(cache, S2) and torch.equal(o[keep], o2)


def test_lin_step_tokens_one_by_one_give_the_same_bits():
    q, k, v, g, S = step_case([21], 3, 3, 128, 128, torch.bfloat16, False, 6, 1)
    all_at_once = S.clone()
    o = gdn.gdn_lin_step(q, k, v, g, all_at_once,
                         cu_seqlens=torch.tensor([0, 21], dtype=torch.int32, device="cuda"))
    for t in range(21):
        ot = gdn.gdn_lin_step(*(x[t:t + 1] for x in (q, k, v, g)), S)
        assert torch.equal(ot[0], o[t])
    assert torch.equal(S, all_at_once)


def test_lin_step_offsets_past_32_bits():
    """A cache of 9.7 GB: slots whose bytes and elements lie past 2^32 and 2^31."""
    slots, H = 4632, 32
    S = torch.empty(slots, H, 128, 128, device="cuda")
    a = step_case([1, 1], H, H, 128, 128, torch.bfloat16, False, 7, 1)
    at = torch.tensor([slots - 1, slots - 2], dtype=torch.int32, device="cuda")
    r = gen(8)
    for i in (1, 2):
        S[slots - i] = r(H, 128, 128)
    small = torch.stack([S[slots - 1], S[slots - 2]])
    o = gdn.gdn_lin_step(*a[:4], S, slot_in=at, slot_out=at)
    o2 = gdn.gdn_lin_step(*a[:4], small)
    assert torch.equal(o, o2) and torch.equal(S[slots - 1], small[0])
    assert torch.equal(S[slots - 2], small[1])


# ------------------------------------------------------------------- qk norm
def qk_inputs(B, T, Hq, Hk, d, rot, dtype, weights, seed, far=0, H=0):
    r = gen(seed)
    x = r(B, T, (Hq + Hk) * d + 8, dtype=dtype, by=2.0)
    q, k = x[..., :Hq * d].unflatten(2, (Hq, d)), x[..., Hq * d:(Hq + Hk) * d].unflatten(2, (Hk, d))
    w = [1.0 + r(d, by=0.2) if weights else None for _ in range(2)]
    f = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
         if rot else None)
    pos = far + torch.from_numpy(np.random.default_rng(seed).integers(-50, 50, (B, T)))
    pos = pos.to(torch.int32).cuda()
    d2 = [r(B, T, H or h, d, dtype=dtype) for h in (Hq, Hk)]
    return q, k, w, f, pos, d2


def qk_check(q, k, w, f, pos, d2, **kw):
    n = host(q, k, *w) + [None if f is None else f.cpu().numpy()]  # frequencies keep 64 bits
    p = None if pos is None else pos.cpu().numpy()
    got = gdn.gdn_qk_norm_fwd(q, k, *w, f, pos=pos, **kw)
    ref = lo.qk_norm_fwd(*n, p, **kw)
    for name, a, b in zip("qk", got, ref):
        check(name, a, b, 1e-5 * np.abs(b).max(initial=0.0))
    got = gdn.gdn_qk_norm_bwd(q, k, *w, f, *d2, pos=pos, **kw)
    ref, mag = lo.qk_norm_bwd(*n, *host(*d2), p, **kw)
    for name, a, b in zip(("dq", "dk"), got, ref):
        check(name, a, b, 5e-5 * np.abs(b).max(initial=0.0))
    for name, a, b, m in zip(("dwq", "dwk"), got[2:], ref[2:], mag):
        if b is None:
            assert a is None
        else:
            check(name, a, b, 2e-5 * m)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("style", ["half", "pairs"])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (128, 0), (256, 256),
                                   (256, 112)])
def test_qk_norm_widths(dtype, style, d, rot):
    x = qk_inputs(2, 7, 3, 1, d, rot, DT[dtype], True, d + rot, far=1000)
    qk_check(*x, style=style, q_scale=d ** -0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hk,H", [(1, 1, 1, 1, 0), (1, 1, 16, 4, 16), (2, 33, 6, 2, 12),
                                         (1, 300, 5, 5, 0), (3, 65, 2, 1, 2), (1, 40, 17, 17, 34)])
@pytest.mark.parametrize("weights", [True, False])
def test_qk_norm_heads(dtype, B, T, Hq, Hk, H, weights):
    x = qk_inputs(B, T, Hq, Hk, 64, 32, DT[dtype], weights, T, H=H)
    qk_check(*x, H=H or None, style="pairs" if T % 2 else "half")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_qk_norm_more_rows_than_a_wave(dtype):
    x = qk_inputs(1, 6000, 7, 3, 128, 128, DT[dtype], True, 1)
    qk_check(*x, q_scale=0.1)


@pytest.mark.parametrize("far", [0, 1 << 20, 2 ** 31 - 100, -2 ** 31 + 100])
@pytest.mark.parametrize("style", ["half", "pairs"])
def test_qk_norm_far_positions(far, style):
    """Angles of the farthest positions: fp64's own pos * f is off by 2^31 2^-53, and its
    reduction mod 2 pi by as much."""
    x = qk_inputs(1, 50, 2, 2, 128, 128, torch.float32, False, 3, far=far)
    qk_check(*x, style=style)


def test_qk_norm_frequencies():
    """Large, tiny, zero and negative frequencies, and positions from the row."""
    q, k, w, _, _, d2 = qk_inputs(2, 90, 2, 2, 64, 64, torch.float32, True, 4)
    f = torch.tensor([0.0, 1e-300, 1e-12, -0.3, 1.0, 3.14159, -100.25, 1e4] * 4, device="cuda",
                     dtype=torch.float64)
    qk_check(q, k, w, f, None, d2)
    qk_check(q, k, w, f, None, d2, style="pairs", q_scale=-2.0, eps=0.5)


def test_qk_norm_no_rows_and_zero_rows():
    for dt in DT.values():
        x = qk_inputs(2, 0, 2, 1, 64, 64, dt, True, 0)
        qk_check(*x)
        q, k, w, f, pos, d2 = qk_inputs(1, 5, 2, 1, 64, 64, dt, True, 0)
        q[:, 2], k[:, 3] = 0, 0
        qk_check(q, k, w, f, pos, d2)


def test_qk_norm_graph_and_stream():
    q, k, w, f, pos, d2 = qk_inputs(1, 300, 4, 2, 128, 64, torch.bfloat16, True, 2)
    want = gdn.gdn_qk_norm_fwd(q, k, *w, f, pos), gdn.gdn_qk_norm_bwd(q, k, *w, f, *d2, pos=pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = (gdn.gdn_qk_norm_fwd(q, k, *w, f, pos, stream=s),
           gdn.gdn_qk_norm_bwd(q, k, *w, f, *d2, pos=pos, stream=s))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = gdn.gdn_qk_norm_fwd(q, k, *w, f, pos), gdn.gdn_qk_norm_bwd(q, k, *w, f, *d2, pos=pos)
    graph.replay()
    torch.cuda.synchronize()
    for w_, g_, c_ in zip(want, got, cap):
        for a, b, c in zip(w_, g_, c_):
            assert torch.equal(a, b) and torch.equal(a, c)


# -------------------------------------------------------------- used together
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layer_over_a_prompt_and_token_by_token(dtype):
    """Norms and rotation, linear attention, gated norm: a prompt at once, continued token by
    token from its boundary state, against the plain layer over everything."""
    dt = DT[dtype]
    r = gen(31)
    T, P, Hq, H, d = 150, 141, 2, 4, 64
    x = r(1, T, (2 * Hq + H) * d, dtype=dt)
    q, k = (x[..., i * Hq * d:(i + 1) * Hq * d].unflatten(2, (Hq, d)) for i in range(2))
    v = x[..., 2 * Hq * d:].unflatten(2, (H, d))
    g = (-r(1, T, H).abs() * 0.1).to(dt)
    wq, wk, wn, z = 1 + r(d, by=0.1), 1 + r(d, by=0.1), 1 + r(d, by=0.1), r(1, T, H, d, dtype=dt)
    f = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
    kw = dict(q_scale=d ** -0.5)
    S = torch.empty(1, H, d, d, device="cuda")
    qn, kn = gdn.gdn_qk_norm_fwd(q[:, :P], k[:, :P], wq, wk, f, H=H, **kw)
    o, _ = gdn.gdn_lin_fwd(qn, kn, v[:, :P], g[:, :P], S_out=S)
    outs = [gdn.gdn_gate_norm_fwd(o, z[:, :P].contiguous(), wn)]
    for t in range(P, T):
        pos = torch.tensor([[t]], dtype=torch.int32, device="cuda")
        qn, kn = gdn.gdn_qk_norm_fwd(q[:, t:t + 1], k[:, t:t + 1], wq, wk, f, pos=pos, **kw)
        o = gdn.gdn_lin_step(qn[0], kn[0], v[0, t:t + 1], g[0, t:t + 1], S)
        outs.append(gdn.gdn_gate_norm_fwd(o[None], z[:, t:t + 1], wn))
    n = host(q, k, wq, wk) + [f.cpu().numpy()] + host(v, g, z, wn)
    rq, rk = lo.qk_norm_fwd(*n[:5], H=H, **kw)
    ro, rS = lo.lin_fwd(rq, rk, n[5], n[6])
    from oracle import layer_ops
    ref = layer_ops.gate_norm_fwd(ro, n[7], n[8])
    # bf16: q, k, o and a factor inside are rounded to 2^-8 each, and the norm of o
    # carries the errors of its row to each value; no cancellation beyond that here
    by = 1e-4 if dt == torch.float32 else 6 * HALF
    err = np.abs(np64(torch.cat(outs, 1)) - ref)
    assert err.max() <= by * np.abs(ref).max()
    assert np.abs(np64(S) - rS).max() <= by * np.abs(rS).max()


# --------------------------------------------------------- large and unusual calls
def wide_check(x, cu=None, scale=0.1):
    """A bf16 call too large for the oracle, against the fp32 kernels (held to the oracle
    above, 2^-17 A) on the same values, with A from the magnitudes by the same kernels."""
    d = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    f = {i: None if x[i] is None else x[i].float() for i in ("q", "k", "v", "g", "S", "do", "dS")}
    m = {i: t if i == "g" or t is None else t.abs() for i, t in f.items()}

    def both(a):
        b = [a[i] for i in ("q", "k", "v", "g", "S")]
        return (gdn.gdn_lin_fwd(*b, scale=scale, cu_seqlens=d),
                gdn.gdn_lin_bwd(*b, a["do"], a["dS"], scale=scale, cu_seqlens=d))

    (o, S), (dq, dk, dv, dg, dS) = both(x)
    (ro, rS), ref = both(f)
    (ao, aS), mag = both(m)
    for name, got, want, a, e in (("o", o, ro, ao, HALF), ("S", S, rS, aS, 3 * 2.0 ** -16),
                                  ("dq", dq, ref[0], mag[0], HALF), ("dk", dk, ref[1], mag[1], HALF),
                                  ("dv", dv, ref[2], mag[2], HALF),
                                  ("dS", dS, ref[4], mag[4], 3 * 2.0 ** -16)):
        tol = (e + 2.0 ** -16) * a + 1e-30 + (HALF * want.abs() if got.dtype == torch.bfloat16 else 0.0)
        off = (got.float() - want).abs() - tol
        assert not (off > 0).any() and not off.isnan().any(), (name, off.max())
    # dg sums the chunk's pairs: as dg_tol, over blocks of 128 tokens on either side
    near = torch.nn.functional.max_pool1d(mag[3].transpose(1, 2), 257, 1, 128).transpose(1, 2)
    off = (dg.float() - ref[3]).abs() - ((HALF + 2.0 ** -16) * near + HALF * ref[3].abs() + 1e-30)
    assert not (off > 0).any() and not off.isnan().any(), ("dg", off.max())


@pytest.mark.parametrize("B,T,H,dk,dv,decay", [(1, 20000, 5, 128, 128, "weak"), (2, 3333, 40, 64, 128, "mid"),
                                               (9, 1025, 17, 128, 64, "mixed"), (160, 129, 2, 64, 64, "weak")])
def test_lin_large(B, T, H, dk, dv, decay):
    wide_check(lin_inputs(B, T, H, dk, dv, torch.bfloat16, decay, seed=T))


@pytest.mark.parametrize("case", ["many short", "one long", "units of the most chunks"])
def test_lin_packed_large(case):
    rng = np.random.default_rng(3)
    if case == "many short":  # more sequences than the planning block has threads, empty ones too
        lens, H = np.concatenate([rng.integers(0, 9, 2500), [700, 0, 1]]), 2
        rng.shuffle(lens)
    elif case == "one long":
        lens, H = np.array([0, 5, 9000, 128, 0]), 3
    else:
        lens, H = np.array([8300, 300, 40]), 170
    cu = [2] + (2 + np.cumsum(lens)).tolist()
    x = lin_inputs(1, cu[-1] + 3, H, 64, 64, torch.bfloat16, "weak", seed=4, nseq=len(lens))
    for i in "qkvg":  # rows of no sequence: the fp32 call leaves them unwritten too
        x[i] = x[i].contiguous()
    d = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o = torch.zeros_like(x["v"])
    a = [x[i] for i in "qkvg"]
    _, S = gdn.gdn_lin_fwd(*a, x["S"], cu_seqlens=d, o=o)
    f = [t.float() for t in a]
    ro, ao = (torch.zeros_like(f[2]) for _ in range(2))
    _, rS = gdn.gdn_lin_fwd(*f, x["S"], cu_seqlens=d, o=ro)
    _, aS = gdn.gdn_lin_fwd(*(t.abs() for t in f[:3]), f[3], x["S"].abs(), cu_seqlens=d, o=ao)
    assert ((o.float() - ro).abs() <= (HALF + 2.0 ** -16) * ao + HALF * ro.abs()).all()
    assert ((S - rS).abs() <= 2.0 ** -14 * aS + 1e-30).all()
    s = slice(cu[0], cu[-1])
    got = gdn.gdn_lin_bwd(*a, x["S"], x["do"], x["dS"], cu_seqlens=d)
    ref = gdn.gdn_lin_bwd(*f, x["S"], x["do"].float(), x["dS"], cu_seqlens=d)
    mag = gdn.gdn_lin_bwd(*(t.abs() for t in f[:3]), f[3], x["S"].abs(), x["do"].float().abs(),
                          x["dS"].abs(), cu_seqlens=d)
    for i in range(3):
        off = (got[i][:, s].float() - ref[i][:, s]).abs()
        assert (off <= (HALF + 2.0 ** -16) * mag[i][:, s] + HALF * ref[i][:, s].abs() + 1e-30).all(), i
    assert ((got[4] - ref[4]).abs() <= 2.0 ** -14 * mag[4] + 1e-30).all()
    near = torch.nn.functional.max_pool1d(mag[3][:, s].float().transpose(1, 2), 257, 1, 128)
    off = (got[3][:, s].float() - ref[3][:, s]).abs()
    assert (off <= (HALF + 2.0 ** -16) * near.transpose(1, 2) + HALF * ref[3][:, s].abs() + 1e-30).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lin_rows_past_32_bits(dtype):
    """Token rows so far apart that the last ones' offsets pass 2^32 elements."""
    T, H = 300, 2
    ld = (1 << 32) // 256 + 64
    x = lin_inputs(1, T, H, 64, 128, DT[dtype], seed=6)
    wide = torch.empty(T * ld, dtype=DT[dtype], device="cuda")
    far = {}
    at = 0
    for i in "qkvg":
        w = x[i].shape[2] * (x[i].shape[3] if i != "g" else 1)
        far[i] = wide.as_strided(x[i].shape, (T * ld, ld) + x[i].stride()[2:] if i == "g" else
                                 (T * ld, ld, x[i].shape[3], 1), at)
        far[i].copy_(x[i])
        at += -(-w // 8) * 8
    a, b = [x[i] for i in "qkvg"], [far[i] for i in "qkvg"]
    for r, w in zip(gdn.gdn_lin_fwd(*b, x["S"]), gdn.gdn_lin_fwd(*a, x["S"])):
        assert torch.equal(r, w)
    for r, w in zip(gdn.gdn_lin_bwd(*b, x["S"], x["do"], x["dS"]),
                    gdn.gdn_lin_bwd(*a, x["S"], x["do"], x["dS"])):
        assert torch.equal(r, w)


def test_lin_broadcast_rows():
    """One row for all tokens (a stride of zero), which the tiles' copies cannot describe."""
    x = lin_inputs(1, 200, 2, 64, 64, torch.bfloat16, seed=8)
    k = x["k"][:, 5:6].expand(-1, 200, -1, -1)
    assert k.stride(1) == 0
    x["k"] = k
    against_oracle(x, scale=0.2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lin_graph_reads_its_offsets_at_replay(dtype):
    x = lin_inputs(1, 900, 2, 64, 64, DT[dtype], seed=10, nseq=3)
    a = [x[i] for i in "qkvg"]
    cu = torch.tensor([0, 100, 300, 900], dtype=torch.int32, device="cuda")
    run = lambda: (gdn.gdn_lin_fwd(*a, x["S"], cu_seqlens=cu)
                   + gdn.gdn_lin_bwd(*a, x["S"], x["do"], x["dS"], cu_seqlens=cu))
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for at in ([0, 900, 900, 900], [0, 0, 450, 900], [0, 100, 300, 900]):
        cu.copy_(torch.tensor(at, dtype=torch.int32))
        want = run()
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(i, j) for i, j in zip(want, got))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lin_calls_on_two_streams_at_once(dtype):
    xs = [lin_inputs(1, 3000, 6, 128, 128, DT[dtype], seed=s) for s in (1, 2)]
    call = lambda x, **kw: (gdn.gdn_lin_fwd(*(x[i] for i in "qkvg"), x["S"], **kw)
                            + gdn.gdn_lin_bwd(*(x[i] for i in "qkvg"), x["S"], x["do"], x["dS"], **kw))
    want = [call(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [call(x, stream=s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert all(torch.equal(i, j) for i, j in zip(w, g))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lin_graphs_that_share_a_workspace(dtype):
    """Two graphs captured with one workspace, replayed in turn on one stream."""
    xs = [lin_inputs(1, T, 3, 64, 128, DT[dtype], seed=T) for T in (1500, 400)]
    args = [[x[i] for i in "qkvg"] + [x["S"]] for x in xs]
    ws = gdn.alloc_workspace(1 << 27, "cuda")
    want = [gdn.gdn_lin_fwd(*a) + gdn.gdn_lin_bwd(*a, x["do"], x["dS"]) for a, x in zip(args, xs)]
    graphs, got = [], []
    for a, x in zip(args, xs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(gdn.gdn_lin_fwd(*a, workspace=ws)
                       + gdn.gdn_lin_bwd(*a, x["do"], x["dS"], workspace=ws))
        graphs.append(g)
    for n in (0, 1, 1, 0):
        for t in got[n]:
            t.fill_(float("nan"))
        graphs[n].replay()
        graphs[1 - n].replay()
    torch.cuda.synchronize()
    assert gdn.gdn_workspace_status(ws) == 0
    for w, r in zip(want, got):
        assert all(torch.equal(i, j) for i, j in zip(w, r))
