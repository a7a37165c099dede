"""How exact a call of gdn_step with several tokens per sequence is: the error measure
and bound of its tests, and a numpy restatement of its tiles of 8 tokens with a chosen
number of TF32 parts per fp32 operand.

The bound, per head in relative 2-norm. With two parts an operand is held to 2^-23 of
itself and the product of the second parts (2^-24) is dropped: a product is good to
2^-21.6. A dot product of 128 terms is a chain of 16 accumulations of 8 products,
each cut off below 2^-23 of the larger of its addends with up to two such cuts: at
most 16 * 2^-22 = 3.8e-6, together 4.1e-6. A tile has three such sums in a row (c,
then u, then the state or the output): 1.2e-5 for each tile."""
import numpy as np

PER_TILE = 1.2e-5
TILE = 8


def bound(lens):
    return PER_TILE * max(1, max(-(-n // TILE) for n in lens))


def error(got, ref):
    """Largest relative 2-norm error over the leading index of got and ref [heads, ...]."""
    d = (got - ref).reshape(len(ref), -1)
    n = np.linalg.norm(ref.reshape(len(ref), -1), axis=1)
    return float((np.linalg.norm(d, axis=1) / np.maximum(n, 1e-30)).max())


def by_head(o, cu):
    """o [tokens, H, dv] as the heads of its sequences, one array each."""
    return [o[a:b, h][None] for a, b in zip(cu, cu[1:]) if b > a for h in range(o.shape[1])]


def _cut(x):
    """fp64 to fp32, towards zero."""
    r = x.astype(np.float32)
    return np.where(np.abs(r.astype(np.float64)) > np.abs(x),
                    np.nextafter(r, np.float32(0)), r).astype(np.float32)


def _split(x, parts, exact):
    if exact:
        return x, np.zeros_like(x)
    mask = np.uint32(0xffffe000)
    hi = ((x.view(np.uint32) + np.uint32(0x1000)) & mask).view(np.float32)
    lo = ((x - hi).view(np.uint32) & mask).view(np.float32)
    return hi, lo if parts == 2 else np.zeros_like(lo)


def _chain(acc, a, b):
    """acc + a @ b over the second axis of a, 8 at a time."""
    for s in range(0, a.shape[1], 8):
        acc = _cut(acc.astype(np.float64) + a[:, s:s + 8].astype(np.float64)
                   @ b[s:s + 8].astype(np.float64))
    return acc


def _dot(a, b, parts, exact_a, exact_b):
    a, b = np.ascontiguousarray(a), np.ascontiguousarray(b)
    (ah, al), (bh, bl) = _split(a, parts, exact_a), _split(b, parts, exact_b)
    zero = np.zeros((a.shape[0], b.shape[1]), np.float32)
    return _chain(zero, ah, bh) + _chain(_chain(zero, al, bh), ah, bl)


def tiles(q, k, v, g, beta, S, parts, bf16):
    """One head of one sequence, gates and norms given: q, k [T, dk], v [T, dv], g, beta
    [T], S [dk, dv], all fp32 (of bf16 values where bf16). Returns (o, S)."""
    S, o = S.copy(), np.zeros_like(v)
    for t0 in range(0, len(q), TILE):
        s = slice(t0, t0 + TILE)
        qt, kt, vt, bt = q[s], k[s], v[s], beta[s]
        n = len(qt)
        a = np.exp(g[s]).astype(np.float32)
        c = _dot(S.T, kt.T, parts, False, bf16)
        p = _dot(S.T, qt.T, parts, False, bf16)
        kk = _dot(kt, kt.T, parts, bf16, bf16)
        qk = _dot(qt, kt.T, parts, bf16, bf16)
        D = np.ones((n, n), np.float32)          # D[t, j] = a[j + 1] .. a[t]
        for t in range(n):
            for j in range(t - 1, -1, -1):
                D[t, j] = D[t, j + 1] * a[j + 1]
        gam = np.cumprod(a, dtype=np.float32)
        u = np.zeros_like(vt)
        for t in range(n):
            x = vt[t] - gam[t] * c[:, t]
            for j in range(t):
                x = x - D[t, j] * kk[t, j] * u[j]
            u[t] = bt[t] * x
            y = gam[t] * p[:, t]
            for j in range(t + 1):
                y = y + D[t, j] * qk[t, j] * u[j]
            o[t0 + t] = y
        S = gam[n - 1] * S + _dot(kt.T, D[n - 1][:, None] * u, parts, bf16, False)
    return o, S
