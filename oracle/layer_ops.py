"""fp64 restatement of the layer operators (include/gdn_layer.h) for the tests:
formulas written out in numpy, gradients by hand, no code shared with the GPU
path. Parameter gradients come with the sum of their terms' magnitudes, which
bounds the rounding error of summing them in fp32."""
import numpy as np


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def softplus(x):
    return np.maximum(x, 0.0) + np.log1p(np.exp(-np.abs(x)))


def _calls(N, n_tok, n_slots, slot_in, slot_out, cu, commit):
    """(first row, tokens, committed, slot read or -1, slot written or -1) per sequence."""
    for s in range(N):
        a, b = (s, s + 1) if cu is None else (int(cu[s]), int(cu[s + 1]))
        if a < 0 or b < a or b > n_tok:
            a = b = 0
        c = b - a if commit is None else min(max(int(commit[s]), 0), b - a)
        i = s if slot_in is None else int(slot_in[s])
        o = s if slot_out is None else int(slot_out[s])
        yield (a, b - a, c, i if 0 <= i < n_slots else -1, o if 0 <= o < n_slots else -1)


def step(q, k, v, g, beta, S, slot_in=None, slot_out=None, cu=None, commit=None, gate=None,
         q_scale=1.0, eps=1e-6, o=None):
    """Token loop. Returns (o, S after the call); rows of no sequence keep `o`."""
    n, H, _ = v.shape
    G = H // q.shape[1]
    if gate is not None:
        rate, bias = gate
        q = q_scale * q / np.sqrt((q * q).sum(-1, keepdims=True) + eps)
        k = k / np.sqrt((k * k).sum(-1, keepdims=True) + eps)
        g = -np.exp(rate) * softplus(g + bias)
        beta = sigmoid(beta)
    q, k = np.repeat(q, G, axis=1), np.repeat(k, G, axis=1)
    out = S.copy()
    o = np.zeros(v.shape) if o is None else o.copy()
    N = n if cu is None else len(cu) - 1
    for t0, T, c, i, w in _calls(N, n, len(S), slot_in, slot_out, cu, commit):
        M = S[i].copy() if i >= 0 else np.zeros(S.shape[1:])
        kept = M.copy()
        for t in range(t0, t0 + T):
            for h in range(H):
                A = np.exp(g[t, h]) * M[h]
                M[h] = A + beta[t, h] * np.outer(k[t, h], v[t, h] - k[t, h] @ A)
                o[t, h] = q[t, h] @ M[h]
            if t - t0 + 1 == c:
                kept = M.copy()
        if w >= 0:
            out[w] = kept
    return o, out


def conv_step(x, w, b, state, slot_in=None, slot_out=None, cu=None, commit=None, act="silu",
              y=None):
    n, C = x.shape
    W = w.shape[1]
    out = state.copy()
    y = np.zeros((n, C)) if y is None else y.copy()
    N = n if cu is None else len(cu) - 1
    for t0, T, c, i, o in _calls(N, n, len(state), slot_in, slot_out, cu, commit):
        old = state[i] if i >= 0 else np.zeros((W - 1, C))
        ext = np.concatenate([old, x[t0:t0 + T]])
        for t in range(T):
            z = (ext[t:t + W] * w.T).sum(0) + (0.0 if b is None else b)
            y[t0 + t] = z * sigmoid(z) if act == "silu" else z
        if o >= 0:
            out[o] = ext[c:c + W - 1]
    return y, out


def prep_fwd(q, k, xg, xb, rate, bias, q_scale=1.0, eps=1e-6):
    G = xg.shape[2] // q.shape[2]
    unit = lambda x, s: np.repeat(s * x / np.sqrt((x * x).sum(-1, keepdims=True) + eps), G, axis=2)
    return unit(q, q_scale), unit(k, 1.0), -np.exp(rate) * softplus(xg + bias), sigmoid(xb)


def prep_bwd(q, k, xg, xb, rate, bias, dqn, dkn, dg, dbeta, q_scale=1.0, eps=1e-6):
    """(dq, dk, dxg, dxb, drate, dbias), (sum |terms| of drate, of dbias)."""
    B, T, Hk, D = q.shape

    def back(x, d, s):
        d = d.reshape(B, T, Hk, -1, D).sum(3)
        n2 = (x * x).sum(-1, keepdims=True) + eps
        return s * (d / np.sqrt(n2) - x * (x * d).sum(-1, keepdims=True) / n2 ** 1.5)

    g = -np.exp(rate) * softplus(xg + bias)
    dxg = -dg * np.exp(rate) * sigmoid(xg + bias)
    b = sigmoid(xb)
    out = (back(q, dqn, q_scale), back(k, dkn, 1.0), dxg, dbeta * b * (1.0 - b),
           (dg * g).sum((0, 1)), dxg.sum((0, 1)))
    return out, (np.abs(dg * g).sum((0, 1)), np.abs(dxg).sum((0, 1)))


def _act(z, act):
    s = sigmoid(z)
    return (z * s, s + z * s * (1.0 - s)) if act == "silu" else (s, s * (1.0 - s))


def gate_norm_fwd(o, z, w, act="silu", eps=1e-6):
    return o / np.sqrt((o * o).mean(-1, keepdims=True) + eps) * w * _act(z, act)[0]


def gate_norm_bwd(o, z, w, dy, act="silu", eps=1e-6):
    """(do, dz, dw), sum |terms| of dw."""
    a, da = _act(z, act)
    m = (o * o).mean(-1, keepdims=True) + eps
    n, e = o / np.sqrt(m), dy * a * w
    do = e / np.sqrt(m) - o * (e * o).mean(-1, keepdims=True) / m ** 1.5
    term = (dy * a * n).reshape(-1, o.shape[-1])
    return (do, dy * n * w * da, term.sum(0)), np.abs(term).sum(0)


def res_norm_fwd(h, x, w, w_post=None, scale=None, eps=1e-6):
    if x is not None:
        p = x if w_post is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w_post
        h = h + (p if scale is None else scale * p)
    return h, h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * w


def res_norm_bwd(h, x, w, dy, dh_out=None, w_post=None, scale=None, eps=1e-6):
    """(dh, dx, dw, dw_post, dscale), the sums of |terms| of the last three. dh is
    itself a sum of three terms that can cancel, so its parts are counted apart."""
    def norm_back(u, e):  # gradient of u / sqrt(mean u^2 + eps) for the upstream e
        m = (u * u).mean(-1, keepdims=True) + eps
        return e / np.sqrt(m) - u * (e * u).mean(-1, keepdims=True) / m ** 1.5

    rows = lambda t: t.reshape(-1, t.shape[-1])
    n = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    dh = norm_back(h, dy * w) + (0.0 if dh_out is None else dh_out)
    parts = (0.0 if dh_out is None else np.abs(dh_out)) + (np.abs(dy * w) + np.abs(
        n * (dy * w * n).mean(-1, keepdims=True))) / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    terms, mags = [dy * n, None, None], [np.abs(dy * n), None, None]
    dx = dh
    mx = None if w_post is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if scale is not None:
        p = x if w_post is None else mx * w_post
        terms[2], mags[2] = dh * p, parts * np.abs(p)
        dx, parts = dh * scale, parts * np.abs(scale)
    if w_post is not None:
        terms[1], mags[1] = dx * mx, parts * np.abs(mx)
        dx = norm_back(x, dx * w_post)
    sums = [None if t is None else rows(t).sum(0) for t in terms]
    return (dh, dx, *sums), [None if t is None else rows(t).sum(0) for t in mags]
