"""The operators of a gated-delta-rule layer as it is served, as cases that can be measured.

Three operators: the gated delta rule over whole sequences (a prompt, a packed
batch of prompts, a long context), the same rule for one new token of each
sequence on a pool of states, and the norms before and after a block joined
with its gate, its residual scale and the residual sum.

``listed`` gives fixed cases, ``draw`` one more of the same ranges, ``prepare``
the inputs of a case on the GPU, ``run`` one pass (``own``: the library's
kernels; otherwise elementary torch operations in 32 bits), ``exact`` the same
outputs from the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
CHUNK = 64


def listed():
    return [
        # the shape of this repository's linear-attention workload, as one prompt batch
        dict(name="rule_batch", op="rule", dtype="bf16", B=4, Hk=4, Hv=4, N=8192, dk=128, dv=128,
             packed=0, state=False, token_major=False),
        # one short question: a prompt of odd length, where latency counts
        dict(name="rule_short", op="rule", dtype="bf16", B=1, Hk=4, Hv=4, N=37, dk=128, dv=128,
             packed=0, state=False, token_major=False),
        # a serving batch: prompts of different lengths (empty and one-token ones among them)
        # packed behind one another, value heads that share key heads, projections' token-major
        # layout, and states carried over from earlier turns
        dict(name="rule_packed", op="rule", dtype="bf16", B=1, Hk=4, Hv=8, N=20011, dk=128, dv=128,
             packed=24, state=True, token_major=True),
        # one document as long as an eighth of the million-token workload, its four heads
        dict(name="rule_long", op="rule", dtype="bf16", B=1, Hk=4, Hv=4, N=131072, dk=128, dv=128,
             packed=0, state=True, token_major=False),
        # a wide layer whose heads fill the card
        dict(name="rule_wide", op="rule", dtype="bf16", B=2, Hk=16, Hv=32, N=4096, dk=128, dv=128,
             packed=0, state=False, token_major=True),
        # the tiny fp32 layer of the tests
        dict(name="rule_tiny_f32", op="rule", dtype="f32", B=1, Hk=1, Hv=1, N=256, dk=32, dv=32,
             packed=0, state=True, token_major=False),
        # one user's next token
        dict(name="step_one", op="step", dtype="bf16", B=1, Hk=4, Hv=4, dk=128, dv=128, pool=1,
             idle=0),
        # a decoding batch with free slots in the pool and idle rows of a fixed-size batch
        dict(name="step_batch", op="step", dtype="bf16", B=61, Hk=8, Hv=16, dk=128, dv=128, pool=96,
             idle=5),
        # a large decoding batch of a wide layer
        dict(name="step_large", op="step", dtype="bf16", B=256, Hk=16, Hv=32, dk=128, dv=128,
             pool=256, idle=0),
        # the norms around a block for one decoded token of a 1536-wide layer
        dict(name="norm_one", op="norm", dtype="bf16", stream="bf16", rows=1, D=1536, group=1536,
             gate=0, residual=True, scale=True, next=True),
        # the same layer over its workload's 2 x 32768 tokens: each head's output normed and gated
        # on the way to the output projection
        dict(name="norm_heads", op="norm", dtype="bf16", stream="bf16", rows=65536, D=1536,
             group=384, gate=1, residual=False, scale=False, next=False),
        # a prompt through the norm after a block, gate, scale and residual in fp32, and the norm
        # before the next block
        dict(name="norm_block", op="norm", dtype="bf16", stream="f32", rows=20011, D=1536,
             group=1536, gate=2, residual=True, scale=True, next=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rule", "rule", "step", "norm"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    Hk = rng.choice((1, 2, 3, 4, 8, 16))
    Hv = Hk * rng.choice((1, 1, 2, 4))
    dk, dv = rng.choice(((128, 128), (128, 128), (64, 64), (128, 256), (96, 72), (32, 32)))
    if op == "rule":
        # 2^27 token-head-state elements at most: the listed cases' work
        most = max(1, min(65536 if dtype == "bf16" else 4096, (1 << 25) // (Hv * max(64, dv))))
        packed = rng.choice((0, 0, 1, 5, 24, 64))
        N = _log_int(rng, 1, most)
        B = 1 if packed else rng.choice((1, 1, 2, 3))
        return dict(op="rule", dtype=dtype, B=B, Hk=Hk, Hv=Hv, N=max(1, N // B), dk=dk, dv=dv,
                    packed=packed, state=rng.random() < 0.5, token_major=rng.random() < 0.5)
    if op == "step":
        B = _log_int(rng, 1, max(1, min(512, 8192 // Hv)))
        return dict(op="step", dtype=dtype, B=B, Hk=Hk, Hv=Hv, dk=dk, dv=dv,
                    pool=B + rng.randrange(0, 1 + B // 2), idle=rng.randrange(0, 1 + B // 4))
    group = rng.choice((32, 64, 96, 128, 384, 1000))
    heads = rng.choice((1, 2, 4, 5, 8))
    D = group * heads
    residual = rng.random() < 0.6
    return dict(op="norm", dtype=dtype, stream=rng.choice((dtype, "f32")),
                rows=_log_int(rng, 1, max(1, min(65536, (1 << 26) // D))), D=D, group=group,
                gate=rng.choice((0, 1, 2)), residual=residual, scale=rng.random() < 0.5,
                next=rng.random() < 0.6)


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _lengths(total, n, gen):
    """n lengths with the given sum: skewed, and from four sequences on one empty and one of a
    single token among them."""
    w = torch.empty(n, dtype=torch.float64).exponential_(generator=gen) + 0.05
    if n >= 4:
        w[1] = 0.0
        w[2] = 0.0
    rest = total - (1 if n >= 4 and total > 1 else 0)
    lens = torch.floor(w / w.sum() * rest).to(torch.int64)
    if n >= 4 and total > 1:
        lens[2] += 1
    lens[0] += total - int(lens.sum())
    return lens.tolist()


def _unit(x):
    """Queries and keys as a layer makes them: SiLU, then unit length."""
    x = x * torch.sigmoid(x)
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6)


def _rule_values(case, shape_k, shape_v, shape_s, r):
    """q, k, v, g, beta; g = -A softplus(a + bias) with A in [1, 16] for each head and time steps
    from 0.001 to 0.1, beta a sigmoid."""
    dt = _dt(case["dtype"])
    q = _unit(r(shape_k)).to(dt)
    k = _unit(r(shape_k)).to(dt)
    v = r(shape_v).to(dt)
    Hv = case["Hv"]
    A = 1.0 + 15.0 * torch.sigmoid(r((Hv,)) * 2)
    step = 0.001 * torch.exp(torch.sigmoid(r((Hv,)) * 2) * math.log(100.0))
    bias = step + torch.log(-torch.expm1(-step))
    view = [1] * len(shape_s)
    view[1] = Hv
    g = -A.view(view) * torch.nn.functional.softplus(r(shape_s) + bias.view(view))
    beta = torch.sigmoid(r(shape_s))
    return q, k, v, g.contiguous(), beta


def _token_major(x):
    """The same [B, H, N, d] values stored as [B, N, H, d]."""
    return x.transpose(1, 2).contiguous().transpose(1, 2)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def r(shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)

    s = dict(case)
    if case["op"] == "norm":
        dt, st = _dt(case["dtype"]), _dt(case["stream"])
        rows, D = case["rows"], case["D"]
        s["y"] = r((rows, D)).to(dt)
        s["w"] = 1.0 + 0.1 * r((case["group"],))
        s["z"] = r((rows, D)).to(dt) if case["gate"] else None
        s["x"] = (2.0 * r((rows, D))).to(st) if case["residual"] else None
        s["a"] = 0.3 * torch.exp(0.2 * r((D,))) if case["scale"] else None
        s["w_next"] = 1.0 + 0.1 * r((D,)) if case["next"] else None
        return s
    B, Hk, Hv, dk, dv = (case[n] for n in ("B", "Hk", "Hv", "dk", "dv"))
    s["factor"] = dk ** -0.5
    if case["op"] == "step":
        q, k, v, g, beta = _rule_values(case, (B, Hk, dk), (B, Hv, dv), (B, Hv), r)
        s.update(q=q, k=k, v=v, g=g, beta=beta)
        s["S"] = 0.3 * r((case["pool"], Hv, dv, dk))
        order = torch.randperm(case["pool"], generator=gen, device=DEV)[:B]
        idle = torch.zeros(B, dtype=torch.bool, device=DEV)
        idle[torch.randperm(B, generator=gen, device=DEV)[:min(case["idle"], B - 1)]] = True
        s["slots"] = torch.where(idle, torch.full_like(order, -1), order).to(torch.int32)
        s["active"] = torch.nonzero(~idle).flatten()
        return s
    N = case["N"]
    q, k, v, g, beta = _rule_values(case, (B, Hk, N, dk), (B, Hv, N, dv), (B, Hv, N), r)
    if case["token_major"]:
        q, k, v = _token_major(q), _token_major(k), _token_major(v)
        g, beta = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (g, beta))
    s.update(q=q, k=k, v=v, g=g, beta=beta)
    n_seq = case["packed"] or B
    s["lengths"] = s["starts"] = None
    if case["packed"]:
        cpu = torch.Generator()
        cpu.manual_seed(seed)
        s["lengths"] = _lengths(N, n_seq, cpu)
        s["starts"] = torch.tensor([0] + s["lengths"]).cumsum(0).to(torch.int32).to(DEV)
    s["S0"] = 0.3 * r((n_seq, Hv, dv, dk)) if case["state"] else None
    return s


# ---------------------------------------------------------------- plain forms


def _rows_of(s):
    """For a packed batch: the token of each place of a [sequences, longest] array, and which
    places hold one."""
    longest = max(1, max(s["lengths"]))
    at = torch.arange(longest, device=DEV)
    starts = s["starts"].long()
    held = at[None] < (starts[1:] - starts[:-1])[:, None]
    return torch.where(held, starts[:-1, None] + at[None], 0), held


def _plain_rule(s):
    f = torch.float32
    group = s["Hv"] // s["Hk"]
    q, k, v, g, beta = (s[n].to(f) for n in ("q", "k", "v", "g", "beta"))
    q, k = (x.repeat_interleave(group, 1) for x in (q, k))
    if s["lengths"] is not None:
        idx, held = _rows_of(s)
        q, k, v = ((x[0][:, idx] * held[None, :, :, None]).transpose(0, 1) for x in (q, k, v))
        g, beta = ((x[0][:, idx] * held[None]).transpose(0, 1) for x in (g, beta))
    n, H, L, dk = q.shape
    dv = v.shape[-1]
    pad = -L % CHUNK
    if pad:
        q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, pad)) for x in (q, k, v))
        g, beta = (torch.nn.functional.pad(x, (0, pad)) for x in (g, beta))
    nc = (L + pad) // CHUNK
    q, k, v = (x.reshape(n, H, nc, CHUNK, x.shape[-1]) for x in (q, k, v))
    beta = beta.reshape(n, H, nc, CHUNK, 1)
    G = g.reshape(n, H, nc, CHUNK).cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, device=DEV, dtype=torch.bool).tril()
    decay = torch.where(low, torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], 0.0)), 0.0)
    kt = k.transpose(-1, -2)
    A = (beta * (k @ kt) * decay).tril(-1)
    P = (q @ kt) * decay
    T = torch.eye(CHUNK, device=DEV, dtype=f).expand(A.shape).clone()
    for i in range(1, CHUNK):  # (1 + A)^-1, row by row for all chunks at once
        T[..., i, :i] = -(A[..., i:i + 1, :i] @ T[..., :i, :i])[..., 0, :]
    e = torch.exp(G)[..., None]
    W, U = T @ (beta * e * k), T @ (beta * v)
    Q = q * e
    last = G[..., -1:]
    K = k * torch.exp(last - G)[..., None]
    end = torch.exp(last)[..., None]
    S = torch.zeros(n, H, dk, dv, device=DEV, dtype=f)
    if s["S0"] is not None:
        S = s["S0"].transpose(-1, -2).clone()
    o = torch.empty(n, H, nc, CHUNK, dv, device=DEV, dtype=f)
    for c in range(nc):  # the state runs from chunk to chunk
        X = U[:, :, c] - W[:, :, c] @ S
        o[:, :, c] = Q[:, :, c] @ S + P[:, :, c] @ X
        S = end[:, :, c] * S + K[:, :, c].transpose(-1, -2) @ X
    o = o.reshape(n, H, nc * CHUNK, dv)[:, :, :L] * s["factor"]
    if s["lengths"] is not None:
        out = torch.zeros(H, s["N"] + 1, dv, device=DEV, dtype=f)
        at = torch.where(held, idx, s["N"]).flatten()
        out[:, at] = o.transpose(0, 1).reshape(H, -1, dv)
        o = out[None, :, :s["N"]]
    return o.to(s["v"].dtype), S.transpose(-1, -2).contiguous()


def _plain_step(s):
    f = torch.float32
    at = s["active"]
    group = s["Hv"] // s["Hk"]
    q, k = (s[n][at].to(f).repeat_interleave(group, 1) for n in ("q", "k"))
    v, g, beta = (s[n][at].to(f) for n in ("v", "g", "beta"))
    slots = s["slots"][at].long()
    S = s["S"][slots] * torch.exp(g)[..., None, None]
    u = beta[..., None] * (v - (S * k[:, :, None, :]).sum(-1))
    S = S + u[..., :, None] * k[:, :, None, :]
    o = (S * q[:, :, None, :]).sum(-1) * s["factor"]
    s["S"][slots] = S
    out = torch.zeros_like(s["v"])
    out[at] = o.to(out.dtype)
    return out, s["S"]


EPS = 1e-6


def _plain_norm(s):
    f = torch.float32
    rows, D = s["rows"], s["D"]
    y = s["y"].to(f).reshape(rows, D // s["group"], s["group"])
    m = (y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * s["w"]).reshape(rows, D)
    if s["gate"]:
        z = s["z"].to(f)
        m = m * (z * torch.sigmoid(z) if s["gate"] == 1 else torch.sigmoid(z))
    if s["a"] is not None:
        m = m * s["a"]
    if s["x"] is not None:
        m = m + s["x"].to(f)
    out = m.to(_dt(s["stream"]))
    if s["w_next"] is None:
        return (out,)
    h = m * torch.rsqrt((m * m).mean(-1, keepdim=True) + EPS) * s["w_next"]
    return out, h.to(_dt(s["dtype"]))


# ---------------------------------------------------------------- the library's calls


def _own_rule(s):
    import chunked_linear_attention_gb300 as cla
    return cla.delta_rule_chunked_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], S0=s["S0"],
                                          seq_starts=s["starts"], scale=s["factor"])


def _own_step(s):
    import chunked_linear_attention_gb300 as cla
    out = cla.delta_rule_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["S"], slots=s["slots"],
                              scale=s["factor"])
    return out, s["S"]


def _own_norm(s):
    import chunked_linear_attention_gb300 as cla
    out, h = cla.block_norm_forward(s["y"], w=s["w"], gate=s["z"],
                                    gate_act=(cla.GATE_NONE, cla.GATE_SILU, cla.GATE_SIGMOID)[s["gate"]],
                                    residual=s["x"], scale=s["a"], w_next=s["w_next"], eps=EPS,
                                    out_dtype=_dt(s["stream"]))
    return (out,) if h is None else (out, h)


def run(state):
    if own:
        return {"rule": _own_rule, "step": _own_step, "norm": _own_norm}[state["op"]](state)
    return {"rule": _plain_rule, "step": _plain_step, "norm": _plain_norm}[state["op"]](state)


# ---------------------------------------------------------------- work and the definition


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        n = case["rows"] * case["D"]
        stream = 2 if case["stream"] == "bf16" else 4
        moved = n * (size * (1 + bool(case["gate"]) + case["next"]) + stream * (1 + case["residual"]))
        return {"bytes": moved + 4 * (case["group"] + case["D"] * (case["scale"] + case["next"])),
                "flops": 12 * n}
    Hk, Hv, dk, dv = (case[n] for n in ("Hk", "Hv", "dk", "dv"))
    if case["op"] == "step":
        tokens, states = case["B"] - min(case["idle"], case["B"] - 1), 2
        states *= tokens
    else:
        tokens = case["B"] * case["N"]
        states = (case["packed"] or case["B"]) * (1 + case["state"])
    # S k, the rank-one update with its decay, S q
    return {"bytes": tokens * (size * 2 * (Hk * dk + Hv * dv) + 8 * Hv) + states * Hv * dv * dk * 4,
            "flops": tokens * Hv * 7 * dk * dv}


def _exact_rule(s):
    d = torch.float64
    group = s["Hv"] // s["Hk"]
    q, k, v, g, beta = (s[n].to(d) for n in ("q", "k", "v", "g", "beta"))
    a = torch.exp(g)
    starts = [0] + torch.tensor(s["lengths"]).cumsum(0).tolist() if s["lengths"] is not None else None
    n = len(s["lengths"]) if starts else s["B"]
    lens = s["lengths"] if starts else [s["N"]] * n
    Hv, dk, dv = s["Hv"], s["dk"], s["dv"]
    S = s["S0"].to(d).clone() if s["S0"] is not None else torch.zeros(n, Hv, dv, dk, device=DEV, dtype=d)
    o = torch.zeros(s["B"], Hv, s["N"], dv, device=DEV, dtype=d)
    by = sorted(range(n), key=lambda i: -lens[i])  # longest first: the live ones are a prefix
    live, first = S[by], torch.tensor([starts[i] if starts else 0 for i in by], device=DEV)
    batch = torch.tensor([0 if starts else i for i in by], device=DEV)
    for t in range(max(lens)):
        m = sum(x > t for x in lens)
        b, at = batch[:m], first[:m] + t
        kt, qt = (x[b, :, at].repeat_interleave(group, 1) for x in (k, q))
        St = live[:m] * a[b, :, at][..., None, None]
        u = beta[b, :, at][..., None] * (v[b, :, at] - (St @ kt[..., None])[..., 0])
        St = St + u[..., None] * kt[..., None, :]
        live[:m] = St
        o[b, :, at] = (St @ qt[..., None])[..., 0] * s["factor"]
    S[by] = live
    return o, S


def _exact_step(s):
    d = torch.float64
    out, S = torch.zeros(s["v"].shape, device=DEV, dtype=d), s["S"].to(d)
    group = s["Hv"] // s["Hk"]
    for h in range(s["Hv"]):  # S <- a S (1 - beta k k^T) + beta v k^T; o = S q
        at = s["active"]
        i = s["slots"][at].long()
        k, q, v = s["k"][at, h // group].to(d), s["q"][at, h // group].to(d), s["v"][at, h].to(d)
        b = s["beta"][at, h].to(d)[:, None, None]
        T = S[i, h] * torch.exp(s["g"][at, h].to(d))[:, None, None]
        T = T - b * torch.einsum("bvk,bk,bl->bvl", T, k, k) + b * torch.einsum("bv,bk->bvk", v, k)
        S[i, h] = T
        out[at, h] = torch.einsum("bvk,bk->bv", T, q) * s["factor"]
    return out, S


def _exact_norm(s):
    d = torch.float64
    y = s["y"].to(d).unflatten(1, (-1, s["group"]))
    m = (y / torch.sqrt(y.square().mean(-1, keepdim=True) + EPS) * s["w"].to(d)).flatten(1)
    if s["gate"]:
        m = m / (1 + torch.exp(-s["z"].to(d))) * (s["z"].to(d) if s["gate"] == 1 else 1.0)
    m = m * s["a"].to(d) if s["a"] is not None else m
    m = m + s["x"].to(d) if s["x"] is not None else m
    if s["w_next"] is None:
        return (m,)
    return m, m / torch.sqrt(m.square().mean(-1, keepdim=True) + EPS) * s["w_next"].to(d)


def exact(case, seed):
    s = prepare(case, seed)
    return {"rule": _exact_rule, "step": _exact_step, "norm": _exact_norm}[case["op"]](s)
