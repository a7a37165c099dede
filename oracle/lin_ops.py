"""fp64 restatement of linear attention with a decay for each head (include/gdn_lin.h)
and of the query and key norms with the rotation (gdn_qk_norm_*, include/gdn_layer.h)
for the tests: token loops and formulas written out in numpy, gradients by hand, no
code shared with the GPU path. On the absolute values of its inputs the recurrence
returns the sum of the magnitudes of every result's terms, which bounds what
roundings of its factors can do to it."""
import numpy as np

from .layer_ops import _calls


def _spans(T, B, cu):
    return [(b * T, (b + 1) * T) for b in range(B)] if cu is None else list(zip(cu[:-1], cu[1:]))


def lin_fwd(q, k, v, g, S_in=None, scale=1.0, cu=None):
    """(o, S_out); rows of no sequence of o are zero. g [B, T, H] or [H]."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    q, k, v = (x.reshape(B * T, H, x.shape[-1]) for x in (q, k, v))
    a = np.exp(np.broadcast_to(g, (B, T, H)).reshape(B * T, H))
    spans = _spans(T, B, cu)
    S = np.zeros((len(spans), H, dk, dv)) if S_in is None else S_in.copy()
    o = np.zeros((B * T, H, dv))
    for s, (t0, t1) in enumerate(spans):
        for t in range(t0, t1):
            S[s] = a[t][:, None, None] * S[s] + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * np.einsum("hi,hij->hj", q[t], S[s])
    return o.reshape(B, T, H, dv), S


def lin_bwd(q, k, v, g, S_in, dout, dS_out=None, scale=1.0, cu=None):
    """(dq, dk, dv, dg, dS_in), with dg [B, T, H] in any case."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    q, k, v, do = (x.reshape(B * T, H, x.shape[-1]) for x in (q, k, v, dout))
    a = np.exp(np.broadcast_to(g, (B, T, H)).reshape(B * T, H))
    spans = _spans(T, B, cu)
    dq, dk_, dv_ = np.zeros((B * T, H, dk)), np.zeros((B * T, H, dk)), np.zeros((B * T, H, dv))
    dg = np.zeros((B * T, H))
    dS = np.zeros((len(spans), H, dk, dv))
    for s, (t0, t1) in enumerate(spans):
        S = [np.zeros((H, dk, dv)) if S_in is None else S_in[s]]
        for t in range(t0, t1):
            S.append(a[t][:, None, None] * S[-1] + k[t][:, :, None] * v[t][:, None, :])
        R = np.zeros((H, dk, dv)) if dS_out is None else dS_out[s].copy()
        for t in reversed(range(t0, t1)):
            dq[t] = scale * np.einsum("hij,hj->hi", S[t - t0 + 1], do[t])
            R = R + scale * q[t][:, :, None] * do[t][:, None, :]
            dk_[t] = np.einsum("hij,hj->hi", R, v[t])
            dv_[t] = np.einsum("hij,hi->hj", R, k[t])
            dg[t] = a[t] * (R * S[t - t0]).sum((1, 2))
            R = a[t][:, None, None] * R
        dS[s] = R
    return tuple(x.reshape(B, T, *x.shape[1:]) for x in (dq, dk_, dv_, dg)) + (dS,)


def lin_step(q, k, v, g, S, slot_in=None, slot_out=None, cu=None, commit=None, scale=1.0, o=None):
    """(o, S after the call); rows of no sequence keep `o`."""
    n, H, _ = v.shape
    q, k = (np.repeat(x, H // x.shape[1], axis=1) for x in (q, k))
    a = np.exp(np.broadcast_to(g, (n, H)))
    out = S.copy()
    o = np.zeros(v.shape) if o is None else o.copy()
    for t0, T, c, i, w in _calls(n if cu is None else len(cu) - 1, n, len(S), slot_in, slot_out,
                                 cu, commit):
        M = S[i].copy() if i >= 0 else np.zeros(S.shape[1:])
        kept = M.copy()
        for t in range(t0, t0 + T):
            M = a[t][:, None, None] * M + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * np.einsum("hi,hij->hj", q[t], M)
            if t - t0 + 1 == c:
                kept = M.copy()
        if w >= 0:
            out[w] = kept
    return o, out


def _turn(x, inv_freq, pos, style, back=False, magnitude=False):
    """The first 2 len(inv_freq) values of x [B, T, H, d] turned by pos * inv_freq, or the
    sum of the two terms' magnitudes that each turned value is made of."""
    n = 0 if inv_freq is None else len(inv_freq)
    if n == 0:
        return np.abs(x) if magnitude else x
    ang = pos.astype(np.float64)[..., None] * inv_freq
    c, s = np.cos(ang)[:, :, None], np.sin(ang)[:, :, None] * (-1.0 if back else 1.0)
    if magnitude:
        a, b = (slice(0, n), slice(n, 2 * n)) if style == "half" else (slice(0, 2 * n, 2),
                                                                      slice(1, 2 * n, 2))
        y = np.abs(x)
        u, v = y[..., a].copy(), y[..., b].copy()
        y[..., a] = u * np.abs(c) + v * np.abs(s)
        y[..., b] = v * np.abs(c) + u * np.abs(s)
        return y
    y = x.copy()
    a, b = (slice(0, n), slice(n, 2 * n)) if style == "half" else (slice(0, 2 * n, 2),
                                                                  slice(1, 2 * n, 2))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def qk_norm_fwd(q, k, wq, wk, inv_freq, pos=None, H=None, style="half", q_scale=1.0, eps=1e-6):
    if pos is None:
        pos = np.broadcast_to(np.arange(q.shape[1]), q.shape[:2])
    out = []
    for x, w, by in ((q, wq, q_scale), (k, wk, 1.0)):
        n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if w is None else w)
        y = by * _turn(n, inv_freq, pos, style)
        out.append(np.repeat(y, H // x.shape[2], axis=2) if H else y)
    return tuple(out)


def qk_norm_bwd(q, k, wq, wk, inv_freq, dqn, dkn, pos=None, H=None, style="half", q_scale=1.0,
                eps=1e-6):
    """(dq, dk, dwq, dwk), (sum |terms| of dwq, of dwk)."""
    if pos is None:
        pos = np.broadcast_to(np.arange(q.shape[1]), q.shape[:2])
    dx, dw, mag = [], [], []
    for x, w, by, d in ((q, wq, q_scale, dqn), (k, wk, 1.0, dkn)):
        B, T, h, D = x.shape
        d = d.reshape(B, T, h, d.shape[2] // h, D).sum(3)
        big = abs(by) * _turn(d, inv_freq, pos, style, back=True, magnitude=True)
        d = by * _turn(d, inv_freq, pos, style, back=True)
        r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        e = d if w is None else d * w
        dx.append(r * (e - x * r * (e * x * r).mean(-1, keepdims=True)))
        dw.append(None if w is None else (d * x * r).sum((0, 1, 2)))
        mag.append(None if w is None else (big * np.abs(x) * r).sum((0, 1, 2)))
    return (*dx, *dw), tuple(mag)
