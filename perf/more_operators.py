"""Performance cases of linear attention with a decay for each head and of the maps
before it.

Three operators: the recurrence S <- e^g S + k v^T, o = scale S^T q over whole
prompts and training chunks (forward and backward, batches and packed sequences),
the same recurrence token by token over a cache of states, and the norm of each
query and key head with the rotation by its position (forward and backward). With
``own`` false, ``run`` computes them in elementary torch operations in fp32; with
``own`` true it calls the library's kernels. ``exact`` evaluates the definitions in
fp64, token by token.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6
CH = 64  # tokens that the plain form takes together


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one sequence being generated: latency
        dict(name="lin step one sequence", op="lin_step", dtype="bf16", N=1, most=1, H=16, Hk=16,
             dk=128, dv=128, const=False),
        # a serving batch, one token each
        dict(name="lin step batch", op="lin_step", dtype="bf16", N=256, most=1, H=32, Hk=32,
             dk=128, dv=128, const=False),
        # drafted tokens verified: ragged, part of them committed, one fixed decay for each head
        dict(name="lin step drafts", op="lin_step", dtype="bf16", N=45, most=8, H=24, Hk=8, dk=128,
             dv=128, const=True),
        # a short prompt: latency of the whole chain of launches
        dict(name="lin forward prompt", op="lin", dir="fwd", dtype="bf16", B=1, T=777, seqs=0, H=16,
             dk=128, dv=128, const=False, state=False),
        # one 32768-token chunk of the long-context training workload, forward
        dict(name="lin forward chunk", op="lin", dir="fwd", dtype="bf16", B=1, T=32768, seqs=0,
             H=16, dk=128, dv=128, const=False, state=True),
        # prompts of a serving batch, packed, fixed decays, narrow values
        dict(name="lin forward packed", op="lin", dir="fwd", dtype="bf16", B=1, T=20001, seqs=13,
             H=32, dk=128, dv=64, const=True, state=True),
        # the training chunk's backward
        dict(name="lin backward chunk", op="lin", dir="bwd", dtype="bf16", B=1, T=32768, seqs=0,
             H=16, dk=128, dv=128, const=False, state=True),
        # full-precision model in training, small heads, odd length
        dict(name="lin backward f32", op="lin", dir="bwd", dtype="f32", B=2, T=2049, seqs=0, H=6,
             dk=64, dv=64, const=False, state=True),
        # documents packed into one training row
        dict(name="lin backward packed", op="lin", dir="bwd", dtype="bf16", B=1, T=8191, seqs=9,
             H=24, dk=64, dv=128, const=False, state=False),
        # one token of one sequence, far into its context
        dict(name="qk norm one token", op="qk_norm", dir="fwd", dtype="bf16", B=1, T=1, Hq=16, Hk=4,
             H=0, d=128, rot=128, style="half", far=1000000, weights=True),
        # the long-context chunk
        dict(name="qk norm forward", op="qk_norm", dir="fwd", dtype="bf16", B=1, T=32768, Hq=16,
             Hk=16, H=0, d=128, rot=128, style="half", far=229376, weights=True),
        # training with shared heads written out, part of each head rotated, odd token count
        dict(name="qk norm backward shared", op="qk_norm", dir="bwd", dtype="bf16", B=1, T=8193,
             Hq=24, Hk=8, H=24, d=128, rot=64, style="pairs", far=0, weights=True),
    ]


CAP = 0.9e9  # bytes of the largest drawn case (the largest listed one has 1.1e9)


def log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["lin_step", "lin", "lin", "lin", "qk_norm", "qk_norm"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "lin_step":
        c["Hk"] = log_int(rng, 1, 32)
        c["H"] = c["Hk"] * rng.choice([g for g in (1, 1, 2, 3, 4) if g * c["Hk"] <= 64])
        c |= dict(N=log_int(rng, 1, 512), most=rng.choice([1, 1, 2, 3, 4, 6, 8, 16]),
                  dk=rng.choice([64, 128]), dv=rng.choice([64, 128]), const=rng.random() < 0.3)
        size = "N"
    elif op == "lin":
        c |= dict(dir=rng.choice(["fwd", "bwd"]), B=1, T=log_int(rng, 1, 49152), seqs=0,
                  H=log_int(rng, 1, 64), dk=rng.choice([64, 128, 128]), dv=rng.choice([64, 128, 128]),
                  const=rng.random() < 0.3, state=rng.random() < 0.5)
        if rng.random() < 0.4:
            c["seqs"] = log_int(rng, 1, 64)
        elif rng.random() < 0.4:
            c["B"] = log_int(rng, 2, 16)
        size = "T"
    else:
        c |= dict(dir=rng.choice(["fwd", "bwd"]), B=rng.choice([1, 1, 2, 5]),
                  T=log_int(rng, 1, 65536), Hq=log_int(rng, 1, 32), H=0,
                  d=rng.choice([64, 128, 128, 256]), style=rng.choice(["half", "pairs"]),
                  far=rng.choice([0, 0, 12345, 1000000]), weights=rng.random() < 0.8)
        c["Hk"] = rng.choice([h for h in range(1, c["Hq"] + 1) if c["Hq"] % h == 0])
        c["H"] = rng.choice([0, c["Hq"]])
        c["rot"] = rng.choice([c["d"], c["d"], c["d"] // 2, c["d"] // 4])
        size = "T"
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


def packed(case):
    """First rows of the sequences of a chunk call, and the end of the last one."""
    if not case["seqs"]:
        return [b * case["T"] for b in range(case["B"] + 1)]
    part = [(1 + (5 * i + 2) % 7) ** 2 for i in range(case["seqs"])]
    cuts = [0]
    for p in part:
        cuts.append(cuts[-1] + p)
    return [round(case["T"] * c / cuts[-1]) for c in cuts]


def work(case):
    e, op = SIZE[case["dtype"]], case["op"]
    if op == "lin_step":
        H, Hk, dk, dv = (case[k] for k in ("H", "Hk", "dk", "dv"))
        lens, commit, fresh = ragged(case)
        forks = pool_slots(case)[1]
        n = sum(lens)
        # a branch without committed tokens is a copy; without tokens and branch nothing moves
        reads = sum(not f and (m > 0 or i < forks) for i, (m, f) in enumerate(zip(lens, fresh)))
        writes = sum(c > 0 or f or i < forks for i, (c, f) in enumerate(zip(commit, fresh)))
        tok = (2 * Hk * dk + 2 * H * dv) * e + (0 if case["const"] else H * e)
        return {"bytes": (reads + writes) * H * dk * dv * 4 + n * tok,
                "flops": n * H * dk * dv * 5}
    if op == "lin":
        H, dk, dv = (case[k] for k in ("H", "dk", "dv"))
        n, back = case["B"] * case["T"], case["dir"] == "bwd"
        nseq = len(packed(case)) - 1
        rows = 4 * dk + 3 * dv if back else 2 * dk + 2 * dv
        gates = 0 if case["const"] else 2 if back else 1
        states = nseq * H * dk * dv * 4 * ((3 if back else 2) if case["state"] else 1)
        # the state's update and its product with q for each token; backward 3 times that
        return {"bytes": n * H * (rows + gates) * e + states,
                "flops": n * H * dk * dv * (12 if back else 4)}
    n, back = case["B"] * case["T"], case["dir"] == "bwd"
    Hq, Hk, d = (case[k] for k in ("Hq", "Hk", "d"))
    out = 2 * case["H"] if case["H"] else Hq + Hk
    heads = 2 * (Hq + Hk) + out if back else Hq + Hk + out
    return {"bytes": n * (heads * d * e + 4), "flops": n * heads * d * 5}


# ---------------------------------------------------------------- the inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DT[case["dtype"]]

    def randn(*shape, dtype=dt, by=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * by).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=gen, device="cuda") * (hi - lo) + lo

    def log_decay(*shape):
        """Log-decays of each token (rate times softplus of a projection), or one for each head."""
        H = shape[-1]
        if case["const"]:  # from next to none to strong, another set for each seed
            return -torch.exp2(-8.0 * (torch.arange(H, device="cuda") + uniform(H)) / H)
        first = torch.exp(uniform(H, lo=math.log(0.001), hi=math.log(0.1)))
        bias = first + torch.log(-torch.expm1(-first))
        x = randn(*shape, dtype=torch.float32)
        return (-uniform(H, lo=1.0, hi=16.0) * torch.nn.functional.softplus(x + bias)).to(dt)

    def unit(x):
        return torch.nn.functional.normalize(x.float(), dim=-1).to(dt)

    op, s = case["op"], dict(case)
    if op == "lin_step":
        H, Hk, dk, dv = (case[k] for k in ("H", "Hk", "dk", "dv"))
        lens, commit, fresh = ragged(case)
        N, n = case["N"], sum(lens)
        slots, forks = pool_slots(case)
        perm = torch.randperm(slots, generator=gen, device="cuda").to(torch.int32)
        s["slot_in"] = torch.where(torch.tensor(fresh, device="cuda"), -1, perm[:N]).to(torch.int32)
        s["slot_out"] = torch.cat([perm[N:N + forks], perm[forks:N]])
        s["cu"] = s["commit"] = None
        if case["most"] > 1:
            cu = [0]
            for m in lens:
                cu.append(cu[-1] + m)
            s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
            s["commit"] = torch.tensor(commit, dtype=torch.int32, device="cuda")
        qkv = randn(n, 2 * Hk * dk + H * dv)  # one row for each token, as the projection leaves it
        s["q"], s["k"] = (qkv[:, i * Hk * dk:(i + 1) * Hk * dk].unflatten(1, (Hk, dk))
                          for i in range(2))
        s["k"].copy_(unit(s["k"]))
        s["v"] = qkv[:, 2 * Hk * dk:].unflatten(1, (H, dv))
        s["g"] = log_decay(n, H)
        s["S"] = randn(slots, H, dk, dv, dtype=torch.float32, by=0.1)
    elif op == "lin":
        B, T, H, dk, dv = (case[k] for k in ("B", "T", "H", "dk", "dv"))
        s["q"], s["k"] = randn(B, T, H, dk), unit(randn(B, T, H, dk))
        s["v"] = randn(B, T, H, dv)
        s["g"] = log_decay(B, T, H)
        first = packed(case)
        n = len(first) - 1
        s["cu"] = (torch.tensor(first, dtype=torch.int32, device="cuda") if case["seqs"] else None)
        back = case["dir"] == "bwd"
        s["S_in"] = randn(n, H, dk, dv, dtype=torch.float32, by=0.1) if case["state"] else None
        s["dS"] = (randn(n, H, dk, dv, dtype=torch.float32, by=0.02) if back and case["state"]
                   else None)
        s["do"] = randn(B, T, H, dv, by=0.1) if back else None
    else:
        B, T, Hq, Hk, d = (case[k] for k in ("B", "T", "Hq", "Hk", "d"))
        qk = randn(B, T, (Hq + Hk) * d, by=2.0)
        s["q"] = qk[..., :Hq * d].unflatten(2, (Hq, d))
        s["k"] = qk[..., Hq * d:].unflatten(2, (Hk, d))
        for w in ("wq", "wk"):
            s[w] = 1.0 + randn(d, dtype=torch.float32, by=0.1) if case["weights"] else None
        r = case["rot"]
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
        start = torch.randint(0, 1000, (B, 1), generator=gen, device="cuda", dtype=torch.int32)
        s["pos"] = case["far"] + start + torch.arange(T, device="cuda", dtype=torch.int32)
        if case["dir"] == "bwd":
            s["dqn"] = randn(B, T, case["H"] or Hq, d, by=0.02)
            s["dkn"] = randn(B, T, case["H"] or Hk, d, by=0.02)
    return s


# ----------------------------------------------------------- the framework's
def run_own(s):
    from chunked_linear_recurrence_gated_gb300 import gdn

    op = s["op"]
    if op == "lin_step":
        o = gdn.gdn_lin_step(s["q"], s["k"], s["v"], s["g"], s["S"], s["slot_in"], s["slot_out"],
                             s["cu"], s["commit"], scale=s["dk"] ** -0.5)
        return o, s["S"]
    if op == "lin":
        kw = dict(scale=s["dk"] ** -0.5, cu_seqlens=s["cu"])
        if s["dir"] == "fwd":
            return gdn.gdn_lin_fwd(s["q"], s["k"], s["v"], s["g"], s["S_in"], **kw)
        return gdn.gdn_lin_bwd(s["q"], s["k"], s["v"], s["g"], s["S_in"], s["do"], s["dS"], **kw)
    kw = dict(pos=s["pos"], H=s["H"] or None, style=s["style"], q_scale=s["d"] ** -0.5, eps=EPS)
    a = (s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"])
    if s["dir"] == "fwd":
        return gdn.gdn_qk_norm_fwd(*a, **kw)
    return gdn.gdn_qk_norm_bwd(*a, s["dqn"], s["dkn"], **kw)


# ----------------------------------------------------------- the plain forms
def plain_step(s):
    q, k, v = (s[x].float() for x in ("q", "k", "v"))
    q, k = (x.repeat_interleave(s["H"] // s["Hk"], dim=1) for x in (q, k))
    q, a = q * s["dk"] ** -0.5, torch.exp(s["g"].float())
    a = a.expand(v.shape[0], s["H"])
    known = (s["slot_in"] >= 0).view(-1, 1, 1, 1)
    S = s["S"][s["slot_in"].clamp(min=0).long()] * known
    if s["cu"] is None:
        S = a[..., None, None] * S + k[..., None] * v[:, :, None, :]
        o = (q[..., None] * S).sum(2)
        s["S"][s["slot_out"].long()] = S
        return o.to(s["v"].dtype), s["S"]
    at, end, kept = s["cu"][:-1].long(), s["cu"][1:].long(), S
    n = v.shape[0]
    o = torch.zeros(n + 1, *v.shape[1:], device=v.device)  # the last row takes what is masked
    for t in range(s["most"] if n else 0):
        live = at + t < end
        i = torch.where(live, at + t, 0)
        S1 = a[i][..., None, None] * S + k[i][..., None] * v[i][:, :, None, :]
        o[torch.where(live, i, n)] = (q[i][..., None] * S1).sum(2)
        S = torch.where(live[:, None, None, None], S1, S)
        kept = torch.where((s["commit"] > t)[:, None, None, None], S, kept)
    s["S"][s["slot_out"].long()] = kept
    return o[:n].to(s["v"].dtype), s["S"]


def chunk_rows(s):
    """The rows of every sequence in whole chunks; the row behind the last stands for no token."""
    n, first = s["B"] * s["T"], packed(s)
    longest = max(b - a for a, b in zip(first, first[1:]))
    at = torch.arange(-(-longest // CH) * CH, device="cuda")
    cu = torch.arange(s["B"] + 1, device="cuda") * s["T"] if s["cu"] is None else s["cu"].long()
    row = cu[:-1, None] + at
    return torch.where(row < cu[1:, None], row, n)


def chunked(x, rows):
    """x [B, T, H, ..] as [sequence, H, chunk, CH, ..] in fp32, zeros behind a sequence's end."""
    x = x.flatten(0, 1).float()
    x = torch.cat([x, torch.zeros_like(x[:1])])
    return x[rows].unflatten(1, (-1, CH)).movedim(3, 1)


def unchunked(x, rows, like, dt):
    """The inverse of chunked."""
    x = x.movedim(1, 3).flatten(1, 2)
    n = like.shape[0] * like.shape[1]
    out = torch.empty(n + 1, *x.shape[2:], device=x.device)
    out[rows] = x
    return out[:n].unflatten(0, like.shape[:2]).to(dt)


def plain_lin(s):
    dt, scale, H = s["q"].dtype, s["dk"] ** -0.5, s["H"]
    rows = chunk_rows(s)
    q, k, v = (chunked(s[x], rows) for x in ("q", "k", "v"))
    c = chunked(s["g"].expand(*s["q"].shape[:3]), rows).cumsum(-1)  # [sequence, H, chunk, CH]
    n, nc = q.shape[0], q.shape[2]
    end = c[..., -1:]
    low = torch.tril(torch.ones(CH, CH, dtype=torch.bool, device=q.device))
    L = torch.where(low, torch.exp(torch.where(low, c[..., :, None] - c[..., None, :], 0.0)), 0.0)
    up, down, whole = torch.exp(c)[..., None], torch.exp(end - c)[..., None], torch.exp(end)[..., None]
    D = (k * down).transpose(-1, -2) @ v
    S = s["S_in"] if s["S_in"] is not None else torch.zeros(n, H, s["dk"], s["dv"], device=q.device)
    states = []
    for j in range(nc):
        states.append(S)
        S = whole[:, :, j] * S + D[:, :, j]
    P, before = (q @ k.transpose(-1, -2)) * L, torch.stack(states, 2)
    if s["dir"] == "fwd":
        o = scale * (P @ v + up * (q @ before))
        return unchunked(o, rows, s["v"], dt), S
    do = chunked(s["do"], rows) * scale
    E = (q * up).transpose(-1, -2) @ do
    R = s["dS"] if s["dS"] is not None else torch.zeros_like(S)
    states = []
    for j in reversed(range(nc)):
        states.append(R)
        R = whole[:, :, j] * R + E[:, :, j]
    after = torch.stack(states[::-1], 2)
    dP = (do @ v.transpose(-1, -2)) * L
    dq_far, dk_far = up * (do @ before.transpose(-1, -2)), down * (v @ after.transpose(-1, -2))
    dq = dP @ k + dq_far
    dk = dP.transpose(-1, -2) @ q + dk_far
    dv = P.transpose(-1, -2) @ do + down * (k @ after)
    # dg_u: every pair (s, t) with s < u <= t, inside the chunk, from before it, to behind it
    A = torch.tril((q @ k.transpose(-1, -2)) * dP, -1)
    a, b = (q * dq_far).sum(-1), (k * dk_far).sum(-1)
    late = (A.sum(-1) + a - A.sum(-2)).flip(-1).cumsum(-1).flip(-1)
    dg = late + b.cumsum(-1) - b + (whole * before * after).sum((-1, -2))[..., None]
    dg = unchunked(dg, rows, s["q"], torch.float32)
    dg = dg.sum((0, 1)) if s["const"] else dg.to(dt)
    return (*(unchunked(x, rows, s["q"], dt) for x in (dq, dk, dv)), dg, R)


def rotated(s, x, back=False):
    """The first `rot` values of each head turned by their angle (or back)."""
    r = s["rot"]
    ang = s["pos"].double()[..., None] * s["inv_freq"]
    cos, sin = torch.cos(ang).float()[:, :, None], torch.sin(ang).float()[:, :, None]
    if back:
        sin = -sin
    t, rest = x[..., :r], x[..., r:]
    if s["style"] == "half":
        a, b = t[..., :r // 2], t[..., r // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = t[..., 0::2], t[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def plain_qk_norm(s):
    dt, out = s["q"].dtype, []
    for x, w, by, d in (("q", "wq", s["d"] ** -0.5, "dqn"), ("k", "wk", 1.0, "dkn")):
        x, w = s[x].float(), s[w]
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        n = x * r
        rep = s["H"] // x.shape[2] if s["H"] else 1
        if s["dir"] == "fwd":
            y = rotated(s, n if w is None else n * w) * by
            out.append(y.repeat_interleave(rep, dim=2).to(dt))
            continue
        d = rotated(s, s[d].float().unflatten(2, (-1, rep)).sum(3), back=True) * by
        e = d if w is None else d * w
        out.append(((r * (e - n * (e * n).mean(-1, keepdim=True))).to(dt),
                    None if w is None else (d * n).sum((0, 1, 2))))
    if s["dir"] == "fwd":
        return tuple(out)
    return out[0][0], out[1][0], out[0][1], out[1][1]


PLAIN = dict(lin_step=plain_step, lin=plain_lin, qk_norm=plain_qk_norm)


def run(state):
    return run_own(state) if own else PLAIN[state["op"]](state)


# --------------------------------------------------- the definitions in fp64
def exact(case, seed):
    if case["op"] == "lin":
        longest = max(b - a for a, b in zip(packed(case), packed(case)[1:]))
        if longest > 33000:  # the loop over tokens takes too long
            return None
    s = prepare(case, seed)
    d = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    return {"lin_step": exact_step, "lin": exact_lin, "qk_norm": exact_qk_norm}[case["op"]](case, s, d)


def exact_step(case, s, d):
    N, G = case["N"], case["H"] // case["Hk"]
    lens, commit, _ = ragged(case)
    start = [0]
    for m in lens:
        start.append(start[-1] + m)
    q, k = (d[x].repeat_interleave(G, 1) for x in ("q", "k"))
    v, g = d["v"], d["g"].expand(d["v"].shape[0], case["H"])
    out, o = d["S"].clone(), torch.zeros_like(v)
    src, dst = s["slot_in"].tolist(), s["slot_out"].tolist()
    order = sorted(range(N), key=lambda i: -lens[i])  # longest first
    dev = v.device
    S = torch.stack([d["S"][src[i]] if src[i] >= 0 else torch.zeros_like(d["S"][0]) for i in order])
    first, want = (torch.tensor([x[i] for i in order], device=dev) for x in (start, commit))
    kept = S.clone()
    for t in range(max(lens)):
        m = sum(n > t for n in lens)
        i = first[:m] + t
        S[:m] = g[i].exp()[..., None, None] * S[:m] + torch.einsum("nhi,nhj->nhij", k[i], v[i])
        o[i] = torch.einsum("nhi,nhij->nhj", q[i], S[:m]) / math.sqrt(case["dk"])
        now = want[:m] == t + 1
        kept[:m][now] = S[:m][now]
    out[torch.tensor([dst[i] for i in order], device=dev)] = kept
    return o, out


def exact_lin(case, s, d):
    first = packed(case)
    lens = [b - a for a, b in zip(first, first[1:])]
    H, dk, dv = (case[x] for x in ("H", "dk", "dv"))
    B, T = case["B"], case["T"]
    dev, scale = s["q"].device, 1.0 / math.sqrt(dk)
    order = sorted(range(len(lens)), key=lambda i: -lens[i])  # longest first
    ids = torch.tensor(order, device=dev)
    at = torch.tensor(first[:-1], device=dev)[ids]
    n, longest = len(lens), max(lens)
    live = [sum(m > t for m in lens) for t in range(longest)]
    q, k, v = (d[x].flatten(0, 1) for x in ("q", "k", "v"))
    a = d["g"].expand(B, T, H).flatten(0, 1).exp()

    def state(x):
        return (torch.zeros(n, H, dk, dv, dtype=torch.float64, device=dev) if x is None
                else d[x][ids].clone())

    def unsorted(x):
        out = torch.empty_like(x)
        out[ids] = x
        return out

    def step(S, t):
        m, i = live[t], at[:live[t]] + t
        S[:m].mul_(a[i][..., None, None]).addcmul_(k[i][..., None], v[i][..., None, :])
        return m, i

    S = state("S_in" if case["state"] else None)
    if case["dir"] == "fwd":
        o = torch.empty_like(v)
        for t in range(longest):
            m, i = step(S, t)
            o[i] = torch.matmul(q[i][..., None, :], S[:m]).squeeze(-2)
        return (o * scale).unflatten(0, (B, T)), unsorted(S)
    do = d["do"].flatten(0, 1) * scale
    block = math.isqrt(longest) + 1  # states are kept for one block, recomputed from its first
    saved = []
    for t in range(longest):
        if t % block == 0:
            saved.append(S.clone())
        step(S, t)
    R = state("dS" if case["state"] else None)
    dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    da = torch.empty_like(a)
    for j in reversed(range(len(saved))):
        S = saved[j]
        inside = [S.clone()]
        for t in range(j * block, min(longest, (j + 1) * block)):
            step(S, t)
            inside.append(S.clone())
        for t in reversed(range(j * block, min(longest, (j + 1) * block))):
            m, i = live[t], at[:live[t]] + t
            now, last, r = inside[t - j * block + 1][:m], inside[t - j * block][:m], R[:m]
            dq[i] = torch.matmul(now, do[i][..., None]).squeeze(-1)
            r.addcmul_(q[i][..., None], do[i][..., None, :])
            dk_[i] = torch.matmul(r, v[i][..., None]).squeeze(-1)
            dv_[i] = torch.matmul(k[i][..., None, :], r).squeeze(-2)
            da[i] = (r * last).sum((-1, -2))
            r.mul_(a[i][..., None, None])
    dg = (da * a).unflatten(0, (B, T))
    dg = dg.sum((0, 1)) if case["const"] else dg
    return (*(x.unflatten(0, (B, T)) for x in (dq, dk_, dv_)), dg, unsorted(R))


def exact_qk_norm(case, s, d):
    back = case["dir"] == "bwd"
    r = case["rot"]
    turn = torch.polar(torch.ones_like(d["pos"], dtype=torch.float64)[..., None].expand(
        *d["pos"].shape, r // 2), d["pos"].double()[..., None] * d["inv_freq"])[:, :, None]
    outs, leaves, gouts = [], [], []
    for x, w, by, dy in (("q", "wq", case["d"] ** -0.5, "dqn"), ("k", "wk", 1.0, "dkn")):
        x = d[x].detach().clone().requires_grad_(back)
        w = None if d[w] is None else d[w].detach().clone().requires_grad_(back)
        y = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS)
        y = y if w is None else y * w
        head = y[..., :r]
        z = (torch.complex(head[..., :r // 2], head[..., r // 2:]) if case["style"] == "half"
             else torch.view_as_complex(head.unflatten(-1, (-1, 2)).contiguous())) * turn
        head = (torch.cat([z.real, z.imag], -1) if case["style"] == "half"
                else torch.view_as_real(z).flatten(-2))
        y = torch.cat([head, y[..., r:]], -1) * by
        if case["H"]:
            y = y.repeat_interleave(case["H"] // y.shape[2], 2)
        outs.append(y)
        leaves += [x, w]
        gouts.append(d.get(dy))
    if not back:
        return tuple(outs)
    some = [t for t in leaves if t is not None]
    got = iter(torch.autograd.grad(outs, some, gouts))
    dq, dwq, dk_, dwk = (None if t is None else next(got) for t in leaves)
    return dq, dk_, dwq, dwk
