"""The layer operators without a GPU: the header and the binding agree, every
bad argument is refused on the host, and the fp64 oracle of the GPU tests is
pinned (against the chunk oracle, the short-convolution oracle and differences)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from chunked_linear_recurrence_gated_gb300 import build, gdn
from oracle import layer_ops as lo
from oracle import short_conv
from test_abi_cpu import header_functions

P = ctypes.c_void_p
FAKE = 1 << 20  # aligned, never dereferenced: every call below fails its checks


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load()


def test_header_and_binding_agree(lib):
    names = header_functions("gdn_layer.h")
    assert names == sorted(gdn.LAYER_EXPORTS)
    for n in names:
        assert hasattr(lib, n)


def call(f, s, ptrs, ws=None):
    a = [P(x) if x else None for x in ptrs]
    return f(s, *a, *([P(ws[0]) if ws[0] else None, ws[1]] if ws else []), None)


def step_shape(**kw):
    d = dict(N=3, n_tok=3, n_slots=4, H=4, Hk=2, dk=128, dv=128, dtype=1, ldq=256, ldk=256,
             ldv=512, ldg=4, ldb=4, q_scale=1.0, eps=1e-6)
    d.update(kw)
    return gdn.gdn_step_shape(*[d[f[0]] for f in gdn.gdn_step_shape._fields_])


STEP_PTRS = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, rate=FAKE, bias=FAKE, S=FAKE,
                 slot_in=None, slot_out=None, cu=None, commit=None, o=FAKE)


@pytest.mark.parametrize("shape,ptrs,status", [
    (dict(N=-1), {}, 1), (dict(n_tok=5), {}, 1), (dict(n_slots=2), {}, 1), (dict(H=0), {}, 1),
    (dict(H=5), {}, 1), (dict(Hk=0), {}, 1), (dict(dk=96), {}, 2), (dict(dv=32), {}, 2),
    (dict(dtype=2), {}, 2), (dict(eps=0.0), {}, 1), (dict(eps=float("nan")), {}, 1),
    (dict(ldq=260), {}, 1), (dict(ldv=-512), {}, 1), (dict(ldg=-1), {}, 1),
    ({}, dict(q=None), 1), ({}, dict(S=None), 1), ({}, dict(o=None), 1), ({}, dict(rate=None), 1),
    ({}, dict(q=FAKE + 8), 1), ({}, dict(S=FAKE + 8), 1), ({}, dict(g=FAKE + 1), 1),
    ({}, dict(cu=FAKE + 2), 1), ({}, dict(o=FAKE + 2), 1)])
def test_step_refusals(lib, shape, ptrs, status):
    assert call(lib.gdn_step, step_shape(**shape), (STEP_PTRS | ptrs).values()) == status


def test_step_nothing_to_do(lib):
    s = step_shape(N=0, n_tok=0)
    assert call(lib.gdn_step, s, [None] * 13) == 1          # slots but no cache
    assert call(lib.gdn_step, step_shape(N=0, n_tok=0, n_slots=0), [None] * 13) == 0
    assert lib.gdn_step(None, *[None] * 13, None) == 1


@pytest.mark.parametrize("shape,ptrs,status", [
    (dict(N=-1), {}, 1), (dict(n_tok=9), {}, 1), (dict(C=0), {}, 1), (dict(C=66), {}, 2),
    (dict(W=1), {}, 2), (dict(W=9), {}, 2), (dict(dtype=3), {}, 2), (dict(act=2), {}, 1),
    (dict(ldx=66), {}, 1), ({}, dict(x=FAKE + 4), 1), ({}, dict(w=None), 1),
    ({}, dict(state=None), 1), ({}, dict(y=FAKE + 8), 1)])
def test_conv_step_refusals(lib, shape, ptrs, status):
    d = dict(N=3, n_tok=3, n_slots=4, C=64, W=4, dtype=1, act=1, ldx=64) | shape
    p = dict(x=FAKE, w=FAKE, b=None, state=FAKE, slot_in=None, slot_out=None, cu=None,
             commit=None, y=FAKE) | ptrs
    assert call(lib.gdn_conv_step, gdn.gdn_conv_step_shape(*d.values()), p.values()) == status


@pytest.mark.parametrize("shape,ptr,status", [
    (dict(rows=-1), None, 1), (dict(H=3), None, 1), (dict(dk=32), None, 2), (dict(dtype=4), None, 2),
    (dict(eps=0.0), None, 1), (dict(ldq=252), None, 1), (dict(ldb=-4), None, 1),
    ({}, (0, None), 1), ({}, (1, FAKE + 8), 1), ({}, (4, None), 1), ({}, (6, FAKE + 8), 1),
    ({}, (8, FAKE + 2), 1)])
def test_prep_refusals(lib, shape, ptr, status):
    d = dict(rows=7, H=4, Hk=2, dk=128, dtype=1, ldq=256, ldk=256, ldg=4, ldb=4, q_scale=1.0,
             eps=1e-6) | shape
    s = gdn.gdn_prep_shape(*d.values())
    for f, n, ws in ((lib.gdn_prep_fwd, 10, None), (lib.gdn_prep_bwd, 16, (FAKE, 1 << 40))):
        p = [FAKE] * n
        if ptr:
            p[ptr[0]] = ptr[1]
        assert call(f, s, p, ws) == status
    if not ptr and not shape.keys() & {"ldq"}:
        assert lib.gdn_prep_workspace_bytes(s) == 0


@pytest.mark.parametrize("shape,ptr,status", [
    (dict(rows=-1), None, 1), (dict(d=0), None, 1), (dict(d=12), None, 2), (dict(d=264), None, 2),
    (dict(act=0), None, 1), (dict(dtype=2), None, 2), (dict(eps=-1.0), None, 1),
    (dict(ldz=251), None, 1), ({}, (0, None), 1), ({}, (1, FAKE + 8), 1), ({}, (2, FAKE + 4), 1)])
def test_gate_norm_refusals(lib, shape, ptr, status):
    d = dict(rows=7, H=2, d=128, dtype=1, act=1, ldz=256, eps=1e-6) | shape
    s = gdn.gdn_gate_norm_shape(*d.values())
    for f, n, ws in ((lib.gdn_gate_norm_fwd, 4, None), (lib.gdn_gate_norm_bwd, 7, (FAKE, 1 << 40))):
        p = [FAKE] * n
        if ptr:
            p[ptr[0]] = ptr[1]
        assert call(f, s, p, ws) == status


@pytest.mark.parametrize("shape,ptr,status", [
    (dict(rows=-1), None, 1), (dict(C=0), None, 1), (dict(C=12), None, 2), (dict(C=16392), None, 2),
    (dict(dtype=0), None, 2), (dict(res_dtype=2), None, 2), (dict(eps=0.0), None, 1),
    ({}, (0, None), 1), ({}, (1, None), 1), ({}, (1, FAKE + 8), 1), ({}, (2, None), 1),
    ({}, (3, FAKE + 8), 1)])
def test_res_norm_refusals(lib, shape, ptr, status):
    d = dict(rows=7, C=128, dtype=1, res_dtype=1, eps=1e-6) | shape
    s = gdn.gdn_res_norm_shape(*d.values())
    for f, n, ws in ((lib.gdn_res_norm_fwd, 7, None), (lib.gdn_res_norm_bwd, 12, (FAKE, 1 << 40))):
        p = [FAKE] * n
        if ptr:
            p[ptr[0]] = ptr[1]
        assert call(f, s, p, ws) == status
    if not shape and ptr is None:
        p = [FAKE] * 12
        p[10] = None                                     # a scale without its gradient
        assert call(lib.gdn_res_norm_bwd, s, p, (FAKE, 1 << 40)) == 1


def test_workspace_refusals(lib):
    shapes = (("prep", gdn.gdn_prep_shape(700, 4, 2, 128, 1, 256, 256, 4, 4, 1.0, 1e-6), 16),
              ("gate_norm", gdn.gdn_gate_norm_shape(700, 2, 128, 1, 1, 256, 1e-6), 7),
              ("res_norm", gdn.gdn_res_norm_shape(700, 128, 1, 1, 1e-6), 12))
    for name, s, n in shapes:
        need = getattr(lib, f"gdn_{name}_workspace_bytes")(s)
        assert need > 0 and need % 256 == 0
        f = getattr(lib, f"gdn_{name}_bwd")
        for ws in ((None, need), (FAKE + 16, need), (FAKE, need - 1)):
            assert call(f, s, [FAKE] * n, ws) == 3


def test_binding_refuses_host_tensors_and_wrong_shapes():
    z = torch.zeros
    with pytest.raises(ValueError):
        gdn.gdn_step(z(1, 1, 64), z(1, 1, 64), z(1, 1, 64), z(1, 1), z(1, 1), z(1, 1, 64, 64))
    with pytest.raises(ValueError):
        gdn.gdn_conv_step(z(1, 8), z(8, 4), None, z(1, 3, 8))
    with pytest.raises(ValueError):
        gdn.gdn_gate_norm_fwd(z(1, 1, 1, 64), z(1, 1, 1, 64), z(64))
    with pytest.raises(ValueError):
        gdn.gdn_res_norm_fwd(z(1, 64), None, z(64))
    with pytest.raises(ValueError):
        gdn.gdn_prep_fwd(z(1, 1, 1, 64), z(1, 1, 1, 64), z(1, 1, 1), z(1, 1, 1), z(1), z(1))
    with pytest.raises(ValueError):                      # rows of two strides
        gdn._rows("x", z(2, 3, 8)[:, :2], 1)
    with pytest.raises(ValueError):                      # not dense inside a row
        gdn._rows("x", z(3, 8)[:, ::2], 1)
    assert gdn._rows("x", z(4, 16)[:, 8:], 1) == 16
    assert gdn._rows("x", z(2, 3, 4, 8)[..., :2, :], 2) == 32


# ------------------------------------------------------------------ oracle pins
def rng_of(seed):
    r = np.random.default_rng(seed)
    return lambda *s: r.standard_normal(s)


def test_oracle_step_is_the_chunk_oracle():
    """The packed token loop equals the chunk oracle (token by token, fp64), sequence by sequence."""
    n = rng_of(1)
    lens, H, dk, dv = [5, 0, 3], 2, 64, 64
    q, k, v = n(8, H, dk) * 0.1, n(8, H, dk) * 0.1, n(8, H, dv)
    g, beta = -np.abs(n(8, H)), lo.sigmoid(n(8, H))
    S = n(4, H, dk, dv)
    cu = np.concatenate([[0], np.cumsum(lens)])
    o, out = lo.step(q, k, v, g, beta, S, cu=cu, slot_in=[2, 0, -1], slot_out=[2, 0, 3])
    for s, (i, w) in enumerate(((2, 2), (None, None), (None, 3))):
        a, b = cu[s], cu[s + 1]
        if a == b:
            continue
        t = lambda x: torch.from_numpy(x[None, a:b].astype(np.float32))
        S0 = None if i is None else torch.from_numpy(S[i:i + 1].astype(np.float32))
        ro, rS = oracle.fwd(t(q), t(k), t(v), t(g), t(beta), S0)
        assert np.abs(o[a:b] - np.asarray(ro)[0]).max() < 1e-5
        assert np.abs(out[w] - np.asarray(rS)[0]).max() < 1e-5
    assert np.array_equal(out[0], S[0]) and np.array_equal(out[1], S[1])


def test_oracle_step_commit_and_shared_heads():
    n = rng_of(2)
    H, Hk, dk, dv, T = 4, 2, 8, 4, 5
    a = n(T, Hk, dk), n(T, Hk, dk), n(T, H, dv), n(T, H), n(T, H)
    gate = (n(H) * 0.1, n(H))
    S = n(3, H, dk, dv)
    o, out = lo.step(*a, S, cu=[0, T], commit=[2], slot_in=[1], slot_out=[2], gate=gate)
    o2, out2 = lo.step(*[x[:2] for x in a], S, cu=[0, 2], slot_in=[1], slot_out=[2], gate=gate)
    assert np.allclose(out, out2) and np.allclose(o[:2], o2)
    assert np.array_equal(out[1], S[1])
    # the maps of the raw form are those of prep_fwd, per value head
    p = lo.prep_fwd(*[x[None] for x in (a[0], a[1], a[3], a[4])], *gate)
    o3, _ = lo.step(p[0][0], p[1][0], a[2], p[2][0], p[3][0], S, cu=[0, T], slot_in=[1])
    assert np.allclose(o, o3)


def test_oracle_conv_step_is_the_short_conv_oracle():
    n = rng_of(3)
    x, w, b, st = n(7, 8), n(8, 4), n(8), n(3, 3, 8)
    y, out = lo.conv_step(x, w, b, st, cu=[0, 5, 7], commit=[5, 1], slot_in=[1, 2], slot_out=[1, 0])
    for s, (a, e, i) in enumerate(((0, 5, 1), (5, 7, 2))):
        ry, rs = short_conv.conv_fwd(x[None, a:e], w, b, st[i:i + 1], "silu")
        assert np.allclose(y[a:e], ry[0])
        if s == 0:
            assert np.allclose(out[1], rs[0])
    assert np.allclose(out[0], np.concatenate([st[2], x[5:7]])[1:4])


def differences(f, args, which, gouts, eps=1e-6):
    """Central differences of sum <f(args), gouts> in args[which]."""
    base = args[which]
    out = np.zeros_like(base)
    for i in np.ndindex(*base.shape):
        val = []
        for sgn in (1, -1):
            a = list(args)
            a[which] = base.copy()
            a[which][i] += sgn * eps
            r = f(*a)
            val.append(sum((u * d).sum() for u, d in zip(r, gouts)))
        out[i] = (val[0] - val[1]) / (2 * eps)
    return out


def close(got, ref):
    # central differences: truncation ~eps^2, cancellation ~1e-16 / eps of values of order 10
    assert np.abs(got - ref).max() <= 1e-7 * max(1.0, np.abs(ref).max()) + 2e-8


def test_oracle_prep_gradient():
    n = rng_of(4)
    B, T, H, Hk, dk = 1, 3, 4, 2, 8
    args = (n(B, T, Hk, dk), n(B, T, Hk, dk), n(B, T, H), n(B, T, H), n(H) * 0.3, n(H))
    d = (n(B, T, H, dk), n(B, T, H, dk), n(B, T, H), n(B, T, H))
    got, _ = lo.prep_bwd(*args, *d, q_scale=0.7)
    f = lambda *a: lo.prep_fwd(*a, q_scale=0.7)
    for i in range(6):
        close(got[i], differences(f, args, i, d))


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_oracle_gate_norm_gradient(act):
    n = rng_of(5)
    args = (n(1, 2, 3, 8), n(1, 2, 3, 8), n(8))
    dy = n(1, 2, 3, 8)
    got, _ = lo.gate_norm_bwd(*args, dy, act)
    for i in range(3):
        close(got[i], differences(lambda *a: [lo.gate_norm_fwd(*a, act)], args, i, [dy]))


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("scale", [False, True])
def test_oracle_res_norm_gradient(post, scale):
    n = rng_of(6)
    h, x, w, dy, dh = n(3, 8), n(3, 8), n(8), n(3, 8), n(3, 8)
    wp, sc = n(8) if post else None, n(8) if scale else None
    args = [h, x, w] + [t for t in (wp, sc) if t is not None]

    def f(h, x, w, *rest):
        rest = list(rest)
        return lo.res_norm_fwd(h, x, w, rest.pop(0) if post else None, rest.pop(0) if scale else None)

    got, _ = lo.res_norm_bwd(f(*args)[0], x, w, dy, dh, wp, sc)
    have = [g for g in got if g is not None]
    for i in range(len(args)):
        close(have[i], differences(f, args, i, (dh, dy)))
