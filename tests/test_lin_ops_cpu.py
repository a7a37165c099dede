"""Linear attention and the query / key norms without a GPU: header and binding agree,
every bad argument is refused on the host, and the fp64 oracle of the GPU tests is
pinned (against the quadratic form, the chunk oracle's recurrence and differences)."""
import ctypes

import numpy as np
import pytest
import torch

from chunked_linear_recurrence_gated_gb300 import build, gdn
from oracle import layer_ops, lin_ops
from test_abi_cpu import header_functions

P = ctypes.c_void_p
FAKE = 1 << 20  # aligned, never dereferenced: every call below fails its checks


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load()


def test_header_and_binding_agree(lib):
    names = header_functions("gdn_lin.h")
    assert names == sorted(gdn.LIN_EXPORTS)
    for n in names:
        assert hasattr(lib, n)


def call(f, s, ptrs, ws=None):
    a = [P(x) if x else None for x in ptrs]
    return f(s, *a, *([P(ws[0]) if ws[0] else None, ws[1]] if ws else []), None)


def shape(cls, base, kw):
    d = base | kw
    return cls(*[d[f[0]] for f in cls._fields_])


STEP = dict(N=3, n_tok=3, n_slots=4, H=4, Hk=2, dk=128, dv=128, dtype=1, ldq=256, ldk=256, ldv=512,
            ldg=4, scale=1.0)
STEP_PTRS = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, decay=None, S=FAKE, slot_in=None, slot_out=None,
                 cu=None, commit=None, o=FAKE)


@pytest.mark.parametrize("kw,ptrs,status", [
    (dict(N=-1), {}, 1), (dict(n_tok=5), {}, 1), (dict(n_slots=2), {}, 1), (dict(H=0), {}, 1),
    (dict(H=5), {}, 1), (dict(Hk=0), {}, 1), (dict(dk=96), {}, 2), (dict(dv=256), {}, 2),
    (dict(dtype=2), {}, 2), (dict(ldq=260), {}, 1), (dict(ldv=-512), {}, 1), (dict(ldg=-1), {}, 1),
    (dict(N=1 << 28, n_tok=1 << 28, n_slots=1 << 28), {}, 2), ({}, dict(q=None), 1),
    ({}, dict(S=None), 1), ({}, dict(o=None), 1), ({}, dict(g=None), 1), ({}, dict(decay=FAKE), 1),
    ({}, dict(g=None, decay=FAKE + 2), 1), ({}, dict(q=FAKE + 8), 1), ({}, dict(S=FAKE + 8), 1),
    ({}, dict(g=FAKE + 1), 1), ({}, dict(cu=FAKE + 2), 1), ({}, dict(o=FAKE + 2), 1)])
def test_lin_step_refusals(lib, kw, ptrs, status):
    s = shape(gdn.gdn_lin_step_shape, STEP, kw)
    assert call(lib.gdn_lin_step, s, (STEP_PTRS | ptrs).values()) == status


LIN = dict(B=2, T=70, H=4, dk=128, dv=64, dtype=1, nseq=2, ldq=512, ldk=512, ldv=256, ldg=4,
           scale=1.0)
FWD = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, decay=None, S_in=None, cu=None, o=FAKE, S_out=FAKE)
BWD = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, decay=None, S_in=None, cu=None, dout=FAKE, dS_out=None,
           dq=FAKE, dk=FAKE, dv=FAKE, dg=FAKE, ddecay=None, dS_in=FAKE)


@pytest.mark.parametrize("kw,ptrs,status", [
    (dict(B=0, nseq=0), {}, 1), (dict(T=-1), {}, 1), (dict(H=0), {}, 1), (dict(nseq=3), {}, 1),
    (dict(nseq=0), {}, 1), (dict(dk=32), {}, 2), (dict(dv=256), {}, 2), (dict(dtype=2), {}, 2),
    (dict(ldq=508), {}, 1), (dict(ldv=-256), {}, 1), (dict(ldg=-4), {}, 1),
    (dict(B=1 << 16, T=1 << 15, nseq=1 << 16), {}, 2), (dict(B=20000, nseq=20000), {}, 2),
    ({}, dict(q=None), 1), ({}, dict(g=None), 1), ({}, dict(decay=FAKE), 1),
    ({}, dict(v=FAKE + 8), 1), ({}, dict(g=FAKE + 1), 1), ({}, dict(S_in=FAKE + 8), 1),
    ({}, dict(cu=FAKE), 1), (dict(B=1), dict(cu=FAKE + 1), 1)])
def test_lin_refusals(lib, kw, ptrs, status):
    s = shape(gdn.gdn_lin_shape, LIN, kw)
    both = {k: v for k, v in ptrs.items() if k in FWD}
    assert call(lib.gdn_lin_fwd, s, (FWD | both).values(), (FAKE, 1 << 50)) == status
    assert call(lib.gdn_lin_bwd, s, (BWD | both).values(), (FAKE, 1 << 50)) == status
    if status == 2:
        assert lib.gdn_lin_workspace_bytes(s, 0) == 0


@pytest.mark.parametrize("f,ptrs", [
    (0, dict(o=None)), (0, dict(o=FAKE + 8)), (0, dict(S_out=FAKE + 4)),
    (1, dict(dout=None)), (1, dict(dq=None)), (1, dict(dv=FAKE + 2)), (1, dict(dg=None)),
    (1, dict(ddecay=FAKE)), (1, dict(g=None, decay=FAKE)), (1, dict(dS_in=FAKE + 8)),
    (1, dict(dS_out=FAKE + 4))])
def test_lin_refusals_of_results(lib, f, ptrs):
    s = shape(gdn.gdn_lin_shape, LIN, {})
    fn, base = ((lib.gdn_lin_fwd, FWD), (lib.gdn_lin_bwd, BWD))[f]
    assert call(fn, s, (base | ptrs).values(), (FAKE, 1 << 50)) == 1


def test_lin_workspace(lib):
    s = shape(gdn.gdn_lin_shape, LIN, {})
    for back, f, p in ((0, lib.gdn_lin_fwd, FWD), (1, lib.gdn_lin_bwd, BWD)):
        need = lib.gdn_lin_workspace_bytes(s, back)
        assert need > 0
        for ws in ((None, need), (FAKE + 16, need), (FAKE, need - 1)):
            assert call(f, s, p.values(), ws) == 3
    assert lib.gdn_lin_workspace_bytes(s, 2) == 0
    assert lib.gdn_lin_fwd(None, *[None] * 9, None, 0, None) == 1


@pytest.mark.parametrize("dtype", [0, 1])
def test_lin_workspace_of_packed_calls(lib, dtype):
    """Sized by the tokens and the sequences, not by their product: at most a state, a row of
    factors and some words for each 64 tokens and each sequence."""
    s = shape(gdn.gdn_lin_shape, LIN, dict(B=1, T=20001, H=32, nseq=13, dtype=dtype, ldq=4096, ldk=4096,
                                           ldv=2048, ldg=32))
    unit = 32 * (128 * 64 * 4 + 1024)
    for back in (0, 1):
        assert lib.gdn_lin_workspace_bytes(s, back) <= (1 + back) * (20001 // 64 + 2 * 13 + 1) * unit
    s = shape(gdn.gdn_lin_shape, LIN, dict(B=2, nseq=3))
    assert lib.gdn_lin_workspace_bytes(s, 0) == 0  # neither packed nor one for each of the batch


QK = dict(rows=7, T=7, Hq=4, Hk=2, H=0, d=128, rot=64, style=0, dtype=1, ldq=512, ldk=256,
          q_scale=1.0, eps=1e-6)


@pytest.mark.parametrize("kw,ptr,status", [
    (dict(rows=-1), None, 1), (dict(T=0), None, 1), (dict(Hq=0), None, 1), (dict(H=6), None, 1),
    (dict(H=-4), None, 1), (dict(d=96), None, 2), (dict(rot=136), None, 2), (dict(rot=24), None, 2),
    (dict(rot=-16), None, 2), (dict(style=2), None, 1), (dict(dtype=2), None, 2),
    (dict(eps=0.0), None, 1), (dict(eps=float("nan")), None, 1), (dict(ldq=508), None, 1),
    (dict(ldk=-256), None, 1), (dict(rows=1 << 29), None, 2), ({}, (0, None), 1),
    ({}, (1, FAKE + 8), 1), ({}, (2, FAKE + 4), 1), ({}, (4, None), 1), ({}, (4, FAKE + 4), 1),
    ({}, (5, FAKE + 2), 1), ({}, (6, None), 1), ({}, (7, FAKE + 8), 1)])
def test_qk_norm_refusals(lib, kw, ptr, status):
    s = shape(gdn.gdn_qk_norm_shape, QK, kw)
    for f, n, ws in ((lib.gdn_qk_norm_fwd, 8, None), (lib.gdn_qk_norm_bwd, 12, (FAKE, 1 << 40))):
        p = [FAKE] * n
        if ptr:
            p[ptr[0]] = ptr[1]
        assert call(f, s, p, ws) == status
    if status == 2:
        assert lib.gdn_qk_norm_workspace_bytes(s) == 0


def test_qk_norm_backward_refusals(lib):
    s = shape(gdn.gdn_qk_norm_shape, QK, {})
    need = lib.gdn_qk_norm_workspace_bytes(s)
    p = [FAKE] * 12
    for ws in ((None, need), (FAKE + 64, need), (FAKE, need - 1)):
        assert call(lib.gdn_qk_norm_bwd, s, p, ws) == 3
    for i, x in ((10, None), (2, None), (11, FAKE + 2), (8, None)):  # a weight and its gradient
        assert call(lib.gdn_qk_norm_bwd, s, p[:i] + [x] + p[i + 1:], (FAKE, need)) == 1


@pytest.mark.parametrize("f,args", [
    ("gdn_lin_fwd", 4), ("gdn_lin_bwd", 6), ("gdn_qk_norm_fwd", 2), ("gdn_lin_step", 5)])
def test_python_entry_refuses_cpu_tensors(lib, f, args):
    x = torch.zeros(1, 3, 2, 64)
    x = x[0] if f == "gdn_lin_step" else x
    with pytest.raises(ValueError):
        getattr(gdn, f)(*[x] * args)
    with pytest.raises(TypeError):
        getattr(gdn, f)(*[None] * args)


# ---------------------------------------------------------------- the oracle
def inputs(seed, B=2, T=9, H=2, dk=4, dv=3, n=None):
    r = np.random.default_rng(seed).standard_normal
    n = n or B
    return (r((B, T, H, dk)), r((B, T, H, dk)), r((B, T, H, dv)), -np.abs(r((B, T, H))),
            r((n, H, dk, dv)), r((B, T, H, dv)), r((n, H, dk, dv)))


def test_oracle_is_the_quadratic_form():
    q, k, v, g, S, _, _ = inputs(1)
    c = np.cumsum(g, 1)
    L = np.exp(c[:, :, None] - c[:, None]) * np.tril(np.ones((9, 9)))[None, :, :, None]
    A = np.einsum("bthi,bshi->btsh", q, k) * L
    o = np.einsum("btsh,bshj->bthj", A, v) + np.einsum("bthi,bhij,bth->bthj", q, S, np.exp(c))
    got, end = lin_ops.lin_fwd(q, k, v, g, S, scale=0.5)
    assert np.abs(got - 0.5 * o).max() < 1e-12
    w = np.exp(c[:, -1:] - c)
    assert np.abs(end - np.exp(c[:, -1])[..., None, None] * S
                  - np.einsum("bshi,bshj,bsh->bhij", k, v, w)).max() < 1e-12


def test_oracle_packed_and_step_agree_with_the_whole_sequences():
    q, k, v, g, S, _, _ = inputs(2, B=1, T=9, n=3)
    cu = [0, 4, 4, 9]
    o, end = lin_ops.lin_fwd(q, k, v, g, S, 0.7, cu)
    for s in range(3):
        sl = slice(cu[s], cu[s + 1])
        a, b = lin_ops.lin_fwd(q[:, sl], k[:, sl], v[:, sl], g[:, sl], S[s:s + 1], 0.7)
        assert np.abs(a - o[:, sl]).max(initial=0.0) < 1e-13 and np.abs(b - end[s]).max() < 1e-13
    o2, cache = lin_ops.lin_step(q[0], k[0], v[0], g[0], S, cu=cu, scale=0.7)
    assert np.abs(o2 - o[0]).max() < 1e-13 and np.abs(cache - end).max() < 1e-13


def test_oracle_step_without_the_delta_correction():
    """The gated delta rule with orthogonal keys in an empty state has nothing to correct."""
    r = np.random.default_rng(3)
    q, v, g = r.standard_normal((4, 1, 4)), r.standard_normal((4, 1, 3)), -r.random((4, 1))
    k = np.linalg.qr(r.standard_normal((4, 4)))[0][:, None]
    S = np.zeros((1, 1, 4, 3))
    a = layer_ops.step(q, k, v, g, np.ones((4, 1)), S, cu=[0, 4])
    b = lin_ops.lin_step(q, k, v, g, S, cu=[0, 4])
    assert all(np.abs(x - y).max() < 1e-13 for x, y in zip(a, b))


def differences(f, x, d, h=1e-6):
    """Directional derivative of f at x along d."""
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("cu", [None, [0, 4, 4, 9]])
@pytest.mark.parametrize("i", range(5))
def test_oracle_gradients_by_differences(cu, i):
    B = 2 if cu is None else 1
    q, k, v, g, S, do, dS = inputs(4 + i, B=B, n=None if cu is None else 3)
    args = [q, k, v, g, S]

    def loss(x):
        a = args[:i] + [x] + args[i + 1:]
        o, end = lin_ops.lin_fwd(*a, 0.8, cu)
        return (o * do).sum() + (end * dS).sum()

    d = np.random.default_rng(9).standard_normal(args[i].shape)
    got = lin_ops.lin_bwd(q, k, v, g, S, do, dS, 0.8, cu)[i]
    assert abs(differences(loss, args[i], d) - (got * d).sum()) < 1e-6 * np.abs(got * d).sum()


@pytest.mark.parametrize("style", ["half", "pairs"])
@pytest.mark.parametrize("i", range(4))
def test_oracle_qk_norm_gradients_by_differences(style, i):
    r = np.random.default_rng(11)
    q, k = r.standard_normal((2, 3, 4, 8)), r.standard_normal((2, 3, 2, 8))
    args = [q, k, r.standard_normal(8), r.standard_normal(8)]
    freq, pos = r.random(2), r.integers(0, 1000, (2, 3))
    dq, dk = r.standard_normal((2, 3, 4, 8)), r.standard_normal((2, 3, 4, 8))
    kw = dict(pos=pos, H=4, style=style, q_scale=0.3, eps=0.1)

    def loss(x):
        a, b = lin_ops.qk_norm_fwd(*(args[:i] + [x] + args[i + 1:]), freq, **kw)
        return (a * dq).sum() + (b * dk).sum()

    d = r.standard_normal(args[i].shape)
    got = lin_ops.qk_norm_bwd(*args, freq, dq, dk, **kw)[0][i]
    assert abs(differences(loss, args[i], d) - (got * d).sum()) < 1e-6 * np.abs(got * d).sum()


@pytest.mark.parametrize("style", ["half", "pairs"])
def test_oracle_rotation_keeps_products_of_relative_positions(style):
    r = np.random.default_rng(12)
    x, y, freq = r.standard_normal((1, 1, 1, 8)), r.standard_normal((1, 1, 1, 8)), r.random(4)

    def dot(i, j):
        a = lin_ops.qk_norm_fwd(x, y, None, None, freq, np.array([[i]]), style=style)[0]
        b = lin_ops.qk_norm_fwd(x, y, None, None, freq, np.array([[j]]), style=style)[1]
        return (a * b).sum()

    assert abs(dot(5, 3) - dot(105, 103)) < 1e-9 and abs(dot(5, 3) - dot(5, 4)) > 1e-3
