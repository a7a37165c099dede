"""Performance cases of the layer operators around the chunk transition.

Five operators: the recurrent gated delta rule over a cache of states, the short
convolution over a cache of its last inputs, the maps that feed the recurrence
(forward and backward), the gated norm of its output and the norm around a
block's residual addition (forward and backward each). With ``own`` false,
``run`` computes them in elementary torch operations in fp32; with ``own`` true
it calls the library's kernels. ``exact`` evaluates the definitions in fp64.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one sequence being generated: latency
        dict(name="step one sequence", op="step", dtype="bf16", N=1, most=1, H=16, Hk=16, dk=128,
             dv=128, raw=True),
        # a serving batch, one token each
        dict(name="step batch", op="step", dtype="bf16", N=256, most=1, H=32, Hk=32, dk=128,
             dv=128, raw=True),
        # drafted tokens verified: ragged, part of them committed, shared key heads, wide values
        dict(name="step drafts", op="step", dtype="bf16", N=45, most=8, H=16, Hk=8, dk=128,
             dv=256, raw=True),
        # full-precision model with maps of its own
        dict(name="step f32", op="step", dtype="f32", N=93, most=3, H=6, Hk=6, dk=64, dv=64,
             raw=False),
        # the q / k / v convolution of one sequence being generated
        dict(name="conv step one sequence", op="conv", dtype="bf16", N=1, most=1, C=6144, W=4),
        # and of a batch with drafted tokens
        dict(name="conv step drafts", op="conv", dtype="bf16", N=301, most=6, C=6144, W=4),
        # one 32768-token chunk of the long-context training workload
        dict(name="prep forward", op="prep", dir="fwd", dtype="bf16", T=32768, H=16, Hk=16, dk=128),
        # gradients of shared key heads, odd token count
        dict(name="prep backward shared", op="prep", dir="bwd", dtype="bf16", T=8193, H=24, Hk=8,
             dk=128),
        # the largest forward: 128K tokens of the output norm
        dict(name="gate norm forward", op="gate_norm", dir="fwd", dtype="bf16", T=131072, H=16,
             d=128, act="silu"),
        # wide values, odd token count
        dict(name="gate norm backward", op="gate_norm", dir="bwd", dtype="bf16", T=16411, H=16,
             d=256, act="silu"),
        # block boundary with a norm on both sides, fp32 residual stream
        dict(name="res norm forward", op="res_norm", dir="fwd", dtype="bf16", res="f32", rows=20011,
             C=4096, post=True, scale=True),
        # the same boundary in training, bf16 residual stream
        dict(name="res norm backward", op="res_norm", dir="bwd", dtype="bf16", res="bf16",
             rows=32768, C=2048, post=True, scale=True),
    ]


CAP = 1.5e9  # bytes of the largest drawn case (the largest listed one has 1.6e9)


def log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["step", "step", "conv", "prep", "gate_norm", "res_norm"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op in ("step", "prep"):
        c["Hk"] = log_int(rng, 1, 32)
        c["H"] = c["Hk"] * rng.choice([g for g in (1, 1, 2, 3, 4) if g * c["Hk"] <= 64])
        c["dk"] = rng.choice([64, 128])
    if op == "step":
        c |= dict(N=log_int(rng, 1, 512), most=rng.choice([1, 1, 2, 3, 4, 6, 8, 16]),
                  dv=rng.choice([64, 128, 256]), raw=rng.random() < 0.7)
        size = "N"
    elif op == "conv":
        c |= dict(N=log_int(rng, 1, 1024), most=rng.choice([1, 1, 2, 4, 7, 16]),
                  C=8 * log_int(rng, 8, 1500), W=rng.choice([2, 3, 4, 4, 4, 5, 8]))
        size = "N"
    else:
        c["dir"] = rng.choice(["fwd", "bwd"])
        size = "T"
        if op == "prep":
            c["T"] = log_int(rng, 1, 131072)
        elif op == "gate_norm":
            c |= dict(T=log_int(rng, 1, 131072), H=log_int(rng, 1, 64),
                      d=rng.choice([64, 128, 128, 256]), act=rng.choice(["silu", "sigmoid"]))
        else:
            size = "rows"
            c |= dict(rows=log_int(rng, 1, 131072), C=8 * log_int(rng, 16, 2048),
                      post=rng.random() < 0.5, scale=rng.random() < 0.5,
                      res="f32" if c["dtype"] == "f32" else rng.choice(["bf16", "f32"]))
    if c.get("C") == 3072:
        c["C"] = 3080
    while work(c)["bytes"] > CAP:
        c[size] = c[size] * 2 // 3
    return c


def ragged(case):
    """Tokens, committed tokens, and whether it starts from a zero state, of each sequence."""
    N, most = case["N"], case["most"]
    if most == 1:
        lens = [1] * N
    else:  # zero-length ones (nothing to do for them this time) among them
        lens = [(5 * i + most) % (most + 1) for i in range(N)]
    commit = [n if most == 1 or i % 3 == 0 else n // 2 if i % 3 == 1 else 0
              for i, n in enumerate(lens)]
    fresh = [i % 11 == 10 for i in range(N)]
    return lens, commit, fresh


def pool_slots(case):
    """Cache size and the number of sequences that branch off into a new slot."""
    forks = case["N"] // 7
    return case["N"] + forks + 1, forks


def work(case):
    e, op = SIZE[case["dtype"]], case["op"]
    if op in ("step", "conv"):
        lens, commit, fresh = ragged(case)
        forks = pool_slots(case)[1]
        n = sum(lens)
        # a branch without committed tokens is a copy; without tokens and branch nothing moves
        reads = sum(not f and (m > 0 or i < forks) for i, (m, f) in enumerate(zip(lens, fresh)))
        writes = sum(c > 0 or f or i < forks for i, (c, f) in enumerate(zip(commit, fresh)))
        if op == "step":
            H, Hk, dk, dv = (case[k] for k in ("H", "Hk", "dk", "dv"))
            tok = (2 * Hk * dk + 2 * H * dv + 2 * H) * e
            return {"bytes": (reads + writes) * H * dk * dv * 4 + n * tok,
                    "flops": n * H * dk * dv * 8}
        C, W = case["C"], case["W"]
        return {"bytes": (reads + writes) * (W - 1) * C * e + 2 * n * C * e + C * (W + 1) * 4,
                "flops": n * C * (2 * W + 4)}
    if op == "prep":
        T, H, Hk, dk = (case[k] for k in ("T", "H", "Hk", "dk"))
        heads = Hk + H if case["dir"] == "fwd" else 2 * Hk + H
        gates = 4 if case["dir"] == "fwd" else 6
        return {"bytes": T * (2 * heads * dk + gates * H) * e, "flops": T * 2 * heads * dk * 3}
    if op == "gate_norm":
        n = case["T"] * case["H"] * case["d"]
        k = 3 if case["dir"] == "fwd" else 5
        return {"bytes": n * k * e + case["d"] * 4, "flops": n * 5 * k}
    n, r = case["rows"] * case["C"], SIZE[case["res"]]
    if case["dir"] == "fwd":  # x, y; h in and out
        per = 2 * e + 2 * r
    else:  # dy; h, dh in, dh out; x where its norm or scale needs it, dx where it is not dh
        plain = not case["post"] and not case["scale"]
        per = e + 3 * r + (0 if plain else e) + (0 if plain and e == r else e)
    return {"bytes": n * per + case["C"] * 4 * (1 + case["post"] + case["scale"]), "flops": n * 12}


# ---------------------------------------------------------------- the inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DT[case["dtype"]]

    def randn(*shape, dtype=dt, by=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * by).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=gen, device="cuda") * (hi - lo) + lo

    def rates(H):
        """Log decay rates and the bias that puts softplus(bias) into [0.001, 0.1]."""
        first = torch.exp(uniform(H, lo=math.log(0.001), hi=math.log(0.1)))
        return torch.log(uniform(H, lo=1.0, hi=16.0)), first + torch.log(-torch.expm1(-first))

    op = case["op"]
    s = dict(case)
    if op in ("step", "conv"):
        lens, commit, fresh = ragged(case)
        N, n = case["N"], sum(lens)
        slots, forks = pool_slots(case)
        perm = torch.randperm(slots, generator=gen, device="cuda").to(torch.int32)
        zero = torch.tensor(fresh, device="cuda")
        s["slot_in"] = torch.where(zero, -1, perm[:N]).to(torch.int32)
        s["slot_out"] = torch.cat([perm[N:N + forks], perm[forks:N]])
        cu = [0]
        for m in lens:
            cu.append(cu[-1] + m)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda") if case["most"] > 1 else None
        s["commit"] = (torch.tensor(commit, dtype=torch.int32, device="cuda")
                       if case["most"] > 1 else None)
    if op == "step":
        H, Hk, dk, dv = (case[k] for k in ("H", "Hk", "dk", "dv"))
        qkv = randn(n, 2 * Hk * dk + H * dv)  # one row for each token, as the convolution leaves it
        qkv = torch.nn.functional.silu(qkv) if case["raw"] else qkv
        gates = randn(n, 2 * H)
        s["q"], s["k"] = (qkv[:, i * Hk * dk:(i + 1) * Hk * dk].unflatten(1, (Hk, dk))
                          for i in range(2))
        s["v"] = qkv[:, 2 * Hk * dk:].unflatten(1, (H, dv))
        s["g"], s["beta"] = gates[:, :H], gates[:, H:]
        s["rate"], s["bias"] = rates(H)
        if not case["raw"]:
            for x in ("q", "k"):
                s[x].copy_(torch.nn.functional.normalize(s[x].float(), dim=-1))
            s["g"].copy_(-torch.nn.functional.softplus(s["g"].float() + 2.0))
            s["beta"].copy_(torch.sigmoid(s["beta"].float()))
        s["S"] = randn(slots, H, dk, dv, dtype=torch.float32, by=0.1)
    elif op == "conv":
        C, W = case["C"], case["W"]
        s["x"], s["state"] = randn(n, C), randn(slots, W - 1, C)
        s["w"] = randn(C, W, dtype=torch.float32, by=W ** -0.5)
        s["b"] = randn(C, dtype=torch.float32, by=0.1)
    elif op == "prep":
        T, H, Hk, dk = (case[k] for k in ("T", "H", "Hk", "dk"))
        qk = torch.nn.functional.silu(randn(1, T, 2 * Hk * dk))
        s["q"], s["k"] = (qk[..., i * Hk * dk:(i + 1) * Hk * dk].unflatten(2, (Hk, dk))
                          for i in range(2))
        gates = randn(1, T, 2 * H)
        s["xg"], s["xb"] = gates[..., :H], gates[..., H:]
        s["rate"], s["bias"] = rates(H)
        if case["dir"] == "bwd":
            s["dq"], s["dk_"] = randn(1, T, H, dk, by=0.02), randn(1, T, H, dk, by=0.02)
            s["dg"], s["dbeta"] = randn(1, T, H, by=0.02), randn(1, T, H, by=0.02)
    elif op == "gate_norm":
        T, H, d = (case[k] for k in ("T", "H", "d"))
        s["o"] = randn(1, T, H, d, by=0.3)
        s["z"] = randn(1, T, H, d)
        s["w"] = 1.0 + randn(d, dtype=torch.float32, by=0.1)
        if case["dir"] == "bwd":
            s["dy"] = randn(1, T, H, d, by=0.02)
    else:
        rows, C, rt = case["rows"], case["C"], DT[case["res"]]
        s["h"], s["x"] = randn(rows, C, dtype=rt), randn(rows, C, by=0.5)
        s["w"] = 1.0 + randn(C, dtype=torch.float32, by=0.1)
        s["w_post"] = 1.0 + randn(C, dtype=torch.float32, by=0.1) if case["post"] else None
        s["s"] = 0.5 + randn(C, dtype=torch.float32, by=0.1) if case["scale"] else None
        if case["dir"] == "bwd":
            s["dy"], s["dh"] = randn(rows, C, by=0.02), randn(rows, C, dtype=rt, by=0.02)
    return s


# ----------------------------------------------------------- the framework's
def run_own(s):
    from chunked_linear_recurrence_gated_gb300 import gdn

    op = s["op"]
    if op == "step":
        gate = (s["rate"], s["bias"]) if s["raw"] else None
        o = gdn.gdn_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["S"], s["slot_in"],
                         s["slot_out"], s["cu"], s["commit"], gate=gate,
                         q_scale=s["dk"] ** -0.5 if s["raw"] else 1.0, eps=EPS)
        return o, s["S"]
    if op == "conv":
        y = gdn.gdn_conv_step(s["x"], s["w"], s["b"], s["state"], s["slot_in"], s["slot_out"],
                              s["cu"], s["commit"], act="silu")
        return y, s["state"]
    if op == "prep":
        a = (s["q"], s["k"], s["xg"], s["xb"], s["rate"], s["bias"])
        if s["dir"] == "fwd":
            return gdn.gdn_prep_fwd(*a, q_scale=s["dk"] ** -0.5, eps=EPS)
        return gdn.gdn_prep_bwd(*a, s["dq"], s["dk_"], s["dg"], s["dbeta"],
                                q_scale=s["dk"] ** -0.5, eps=EPS)
    if op == "gate_norm":
        if s["dir"] == "fwd":
            return gdn.gdn_gate_norm_fwd(s["o"], s["z"], s["w"], act=s["act"], eps=EPS)
        return gdn.gdn_gate_norm_bwd(s["o"], s["z"], s["w"], s["dy"], act=s["act"], eps=EPS)
    kw = dict(w_post=s["w_post"], scale=s["s"], eps=EPS)
    if s["dir"] == "fwd":
        return gdn.gdn_res_norm_fwd(s["h"], s["x"], s["w"], **kw)
    return gdn.gdn_res_norm_bwd(s["h"], s["x"], s["w"], s["dy"], s["dh"], **kw)


# ----------------------------------------------------------- the plain forms
def unit(x, scale=1.0):
    return x * (scale * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS))


def rms(x):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def softplus(x):
    return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-x.abs()))


def gate_of(z, act):
    sg = torch.sigmoid(z)
    return (z * sg, sg * (1.0 + z * (1.0 - sg))) if act == "silu" else (sg, sg * (1.0 - sg))


def start_states(s, pool):
    """The cached states of the call's sequences (zeros for a fresh one), in fp32."""
    known = (s["slot_in"] >= 0).view(-1, *[1] * (pool.dim() - 1))
    return pool[s["slot_in"].clamp(min=0).long()].float() * known


def plain_step(s):
    f = lambda x: x.float()  # noqa: E731
    q, k, v, g, beta = (f(s[x]) for x in ("q", "k", "v", "g", "beta"))
    if s["raw"]:
        q, k = unit(q, s["dk"] ** -0.5), unit(k)
        g = -torch.exp(s["rate"]) * softplus(g + s["bias"])
        beta = torch.sigmoid(beta)
    q, k = (x.repeat_interleave(s["H"] // s["Hk"], dim=1) for x in (q, k))
    a = torch.exp(g)
    S = start_states(s, s["S"])
    o = torch.empty_like(v)
    if s["cu"] is None:
        S = a[..., None, None] * S
        u = beta[..., None] * (v - (k[..., None] * S).sum(2))
        S = S + k[..., None] * u[:, :, None, :]
        o = (q[..., None] * S).sum(2)
        s["S"][s["slot_out"].long()] = S
        return o.to(s["v"].dtype), s["S"]
    at, end, kept = s["cu"][:-1].long(), s["cu"][1:].long(), S
    o = torch.zeros(o.shape[0] + 1, *o.shape[1:], device=o.device)  # the last row takes what is masked
    for t in range(s["most"]):  # the recurrence over the drafted tokens
        live = at + t < end
        i = torch.where(live, at + t, 0)
        S1 = a[i][..., None, None] * S
        u = beta[i][..., None] * (v[i] - (k[i][..., None] * S1).sum(2))
        S1 = S1 + k[i][..., None] * u[:, :, None, :]
        o[torch.where(live, i, o.shape[0] - 1)] = (q[i][..., None] * S1).sum(2)
        S = torch.where(live[:, None, None, None], S1, S)
        kept = torch.where((s["commit"] > t)[:, None, None, None], S, kept)
    s["S"][s["slot_out"].long()] = kept
    return o[:-1].to(s["v"].dtype), s["S"]


def plain_conv(s):
    W, x = s["W"], s["x"].float()
    state = start_states(s, s["state"])
    N, n = state.shape[0], x.shape[0]
    if s["cu"] is None:
        cu = torch.arange(N + 1, device=x.device)
        commit = torch.ones(N, dtype=torch.long, device=x.device)
    else:
        cu, commit = s["cu"].long(), s["commit"].long()
    # every sequence's cached inputs, then its new ones, as rows of one table
    rows = torch.cat([state.flatten(0, 1), x])
    taps = torch.arange(W - 1, device=x.device)

    def ext(seq, i):  # row of the table that holds input i of x_ext of a sequence
        return torch.where(i < W - 1, seq * (W - 1) + i, N * (W - 1) + cu[seq] + i - (W - 1))

    tok = torch.arange(n, device=x.device)
    seq = torch.searchsorted(cu, tok, right=True) - 1
    window = rows[ext(seq[:, None], (tok - cu[seq])[:, None] + torch.arange(W, device=x.device))]
    z = (window * s["w"].t()).sum(1) + s["b"]
    y = (z * torch.sigmoid(z)).to(s["x"].dtype)
    last = rows[ext(torch.arange(N, device=x.device)[:, None], commit[:, None] + taps)]
    s["state"][s["slot_out"].long()] = last.to(s["state"].dtype)
    return y, s["state"]


def plain_prep(s):
    q, k, xg, xb = (s[x].float() for x in ("q", "k", "xg", "xb"))
    G, dt, scale = s["H"] // s["Hk"], s["q"].dtype, s["dk"] ** -0.5
    sp, rate = xg + s["bias"], torch.exp(s["rate"])
    beta = torch.sigmoid(xb)
    g = -rate * softplus(sp)
    if s["dir"] == "fwd":
        qn, kn = (x.repeat_interleave(G, dim=2) for x in (unit(q, scale), unit(k)))
        return qn.to(dt), kn.to(dt), g.to(dt), beta.to(dt)

    def back(x, d, c):
        d = d.float().unflatten(2, (s["Hk"], G)).sum(3)
        r = torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS)
        return (c * r * (d - x * (r * r * (x * d).sum(-1, keepdim=True)))).to(dt)

    dg, dbeta = s["dg"].float(), s["dbeta"].float()
    dxg = -dg * rate * torch.sigmoid(sp)
    dxb = dbeta * beta * (1.0 - beta)
    return (back(q, s["dq"], scale), back(k, s["dk_"], 1.0), dxg.to(dt), dxb.to(dt),
            (dg * g).sum((0, 1)), dxg.sum((0, 1)))


def plain_gate_norm(s):
    o, z, w, dt = s["o"].float(), s["z"].float(), s["w"], s["o"].dtype
    r = torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS)
    n = o * r
    a, da = gate_of(z, s["act"])
    if s["dir"] == "fwd":
        return (n * w * a).to(dt)
    dy = s["dy"].float()
    D = dy * a * w
    do = r * (D - n * (D * n).mean(-1, keepdim=True))
    return do.to(dt), (dy * n * w * da).to(dt), (dy * a * n).sum((0, 1, 2))


def plain_res_norm(s):
    h, x, dt, rt = s["h"].float(), s["x"].float(), s["x"].dtype, s["h"].dtype
    post, sc = s["w_post"], s["s"]
    p = x if post is None else rms(x) * post
    if s["dir"] == "fwd":
        h = h + (p if sc is None else sc * p)
        return h.to(rt), (rms(h) * s["w"]).to(dt)
    dy = s["dy"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    n, D = h * r, dy * s["w"]
    dh = s["dh"].float() + r * (D - n * (D * n).mean(-1, keepdim=True))
    dp = dh if sc is None else sc * dh
    dx, dpost = dp, None
    if post is not None:
        rx = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        m, E = x * rx, dp * post
        dx, dpost = rx * (E - m * (E * m).mean(-1, keepdim=True)), (dp * m).sum(0)
    dsc = None if sc is None else (dh * p).sum(0)
    return dh.to(rt), dx.to(dt), (dy * n).sum(0), dpost, dsc


PLAIN = dict(step=plain_step, conv=plain_conv, prep=plain_prep, gate_norm=plain_gate_norm,
             res_norm=plain_res_norm)


def run(state):
    return run_own(state) if own else PLAIN[state["op"]](state)


# --------------------------------------------------- the definitions in fp64
def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    op = case["op"]
    if op in ("step", "conv"):
        N = case["N"]
        lens, commit, fresh = ragged(case)
        start = [0]
        for m in lens:
            start.append(start[-1] + m)
        src, dst = s["slot_in"].tolist(), s["slot_out"].tolist()
    if op == "step":
        G = case["H"] // case["Hk"]
        q, k, v, g, beta = (d[x] for x in ("q", "k", "v", "g", "beta"))
        if case["raw"]:
            q = q / torch.sqrt(q.pow(2).sum(-1, keepdim=True) + EPS) / math.sqrt(case["dk"])
            k = k / torch.sqrt(k.pow(2).sum(-1, keepdim=True) + EPS)
            g = -d["rate"].exp() * torch.nn.functional.softplus(g + d["bias"], threshold=100.0)
            beta = beta.sigmoid()
        q, k = q.repeat_interleave(G, 1), k.repeat_interleave(G, 1)
        out, o = d["S"].clone(), torch.zeros_like(v)
        eye = torch.eye(case["dk"], device=v.device, dtype=torch.float64)
        order = sorted(range(N), key=lambda i: -lens[i])
        ids = torch.tensor(order, device=v.device)
        S = torch.stack([d["S"][i] if i >= 0 else torch.zeros_like(d["S"][0]) for i in src])[ids]
        first = torch.tensor(start[:-1], device=v.device)[ids]
        kept, want = S.clone(), torch.tensor(commit, device=v.device)[ids]
        for t in range(max(lens, default=0)):
            m = sum(n > t for n in lens)  # the sequences that have a token t, longest first
            i = first[:m] + t
            kk, al = k[i], g[i].exp()[..., None, None]
            b = beta[i][..., None, None]
            erase = eye - b * kk[..., :, None] * kk[..., None, :]
            S[:m] = al * (erase @ S[:m]) + b * kk[..., :, None] * v[i][..., None, :]
            o[i] = torch.matmul(q[i][..., None, :], S[:m]).squeeze(-2)
            now = want[:m] == t + 1
            kept[:m][now] = S[:m][now]
        out[torch.tensor(dst, device=v.device)[ids]] = kept
        return o, out
    if op == "conv":
        W, out, ys = case["W"], d["state"].clone(), []
        w = d["w"]
        for i in range(N):
            old = d["state"][src[i]] if src[i] >= 0 else torch.zeros_like(d["state"][0])
            x = torch.cat([old, d["x"][start[i]:start[i + 1]]])
            out[dst[i]] = x[commit[i]:commit[i] + W - 1]
            if lens[i]:
                z = torch.einsum("tcw,cw->tc", x.unfold(0, W, 1), w) + d["b"]
                ys.append(z / (1.0 + torch.exp(-z)))
        return torch.cat(ys) if ys else torch.zeros_like(d["x"]), out
    back = case["dir"] == "bwd"

    def leaf(*names):
        return [None if d[n] is None else d[n].detach().clone().requires_grad_(back) for n in names]

    def grads(outs, gouts, of):
        some = [t for t in of if t is not None]
        got = iter(torch.autograd.grad(outs, some, gouts))
        return tuple(None if t is None else next(got) for t in of)

    def norm(x):
        return x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS)

    if op == "prep":
        q, k, xg, xb, rate, bias = of = leaf("q", "k", "xg", "xb", "rate", "bias")
        G = case["H"] // case["Hk"]
        unit64 = [x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) + EPS) for x in (q, k)]
        outs = (unit64[0].repeat_interleave(G, 2) / math.sqrt(case["dk"]),
                unit64[1].repeat_interleave(G, 2),
                -rate.exp() * torch.nn.functional.softplus(xg + bias, threshold=100.0),
                xb.sigmoid())
        return grads(outs, [d[x] for x in ("dq", "dk_", "dg", "dbeta")], of) if back else outs
    if op == "gate_norm":
        o, z, w = of = leaf("o", "z", "w")
        y = norm(o) * w * (z.sigmoid() * z if case["act"] == "silu" else z.sigmoid())
        return grads([y], [d["dy"]], of) if back else y
    h, x, w, post, sc = of = leaf("h", "x", "w", "w_post", "s")
    p = x if post is None else norm(x) * post
    if not back:
        h = h + (p if sc is None else sc * p)
        return h, norm(h) * w
    # the gradient is taken at the residual that the forward stored: h here is its output
    step = p if sc is None else sc * p
    out = h + (step - step.detach())
    return grads([out, norm(out) * w], [d["dh"], d["dy"]], of)
