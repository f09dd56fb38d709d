"""Sequence mixers with a state of fixed size, as they are served, as cases that can be measured.

Three operators, each over whole prompts and for one new token of each sequence
on a pool: attention with a sliding window and a few first tokens that stay
visible (a ring of keys and values for each sequence), the selective state space
scan, and the short causal convolution in front of such a recurrence.

``listed`` gives fixed cases, ``draw`` one more of the same ranges, ``prepare``
the inputs of a case on the GPU, ``run`` one pass (``own``: the library's
kernels; otherwise elementary torch operations in 32 bits), ``exact`` the same
outputs from the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # the window attention beside the TTT layer of the LM workload: 2 x 32768 tokens of a
        # 1536-wide layer, window as long as the chunk
        dict(name="attn_layer", op="attn", dtype="bf16", B=2, Hq=12, Hk=4, N=32768, d=128,
             window=2048, sinks=4, packed=0, past=False, cache=True, token_major=True),
        # a serving batch: prompts of different lengths (empty and one-token ones among them)
        # packed behind one another, most of them later turns on a cache
        dict(name="attn_packed", op="attn", dtype="bf16", B=1, Hq=16, Hk=4, N=20011, d=64,
             window=1000, sinks=4, packed=24, past=True, cache=True, token_major=True),
        # one short question in fp32, the type of the tests, where latency counts
        dict(name="attn_short_f32", op="attn", dtype="f32", B=1, Hq=4, Hk=2, N=37, d=64,
             window=16, sinks=2, packed=0, past=False, cache=True, token_major=False),
        # one user's next token, far into a long document
        dict(name="attn_step_one", op="attn_step", dtype="bf16", B=1, Hq=12, Hk=4, d=128,
             window=2048, sinks=4, pool=1, idle=0),
        # a large decoding batch with free slots in the pool and idle rows
        dict(name="attn_step_large", op="attn_step", dtype="bf16", B=250, Hq=32, Hk=8, d=128,
             window=2048, sinks=4, pool=256, idle=5),
        # a selective scan of the LM workload's tokens and width, gated
        dict(name="scan_layer", op="scan", dtype="bf16", B=2, N=32768, D=1536, S=16, G=1,
             packed=0, state=False, gate=True, wide=True),
        # a packed batch of prompts with carried states
        dict(name="scan_packed", op="scan", dtype="bf16", B=1, N=20011, D=1000, S=16, G=2,
             packed=24, state=True, gate=True, wide=False),
        # one short question in fp32
        dict(name="scan_short_f32", op="scan", dtype="f32", B=1, N=37, D=512, S=16, G=1,
             packed=0, state=True, gate=False, wide=False),
        # a decoding batch of a wide layer
        dict(name="scan_step_large", op="scan_step", dtype="bf16", B=250, D=4096, S=16, G=1,
             pool=256, idle=5, gate=True),
        # the convolution in front of the scan, x as a part of the input projection
        dict(name="conv_layer", op="conv", dtype="bf16", B=2, N=32768, D=1536, W=4, act=True,
             packed=0, state=False, wide=True),
        # a packed batch in fp32 with an odd width
        dict(name="conv_packed_f32", op="conv", dtype="f32", B=1, N=20011, D=1001, W=4, act=True,
             packed=24, state=True, wide=False),
        # a decoding batch: q, k and v of a delta-rule layer together
        dict(name="conv_step_batch", op="conv_step", dtype="bf16", B=61, D=4096, W=4, act=True,
             pool=96, idle=5, wide=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attn", "attn", "attn_step", "scan", "scan", "scan_step", "conv", "conv_step"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op.startswith("attn"):
        Hk = rng.choice((1, 2, 3, 4, 8))
        Hq = Hk * rng.choice((1, 2, 3, 4, 8))
        d = rng.choice((128, 128, 64, 64, 96, 80, 32))
        window, sinks = _log_int(rng, 1, 4096), rng.choice((0, 0, 1, 4, 4, 130))
        if op == "attn_step":
            # 2^28 elements of keys at most
            B = _log_int(rng, 1, max(1, min(256, (1 << 28) // (Hk * (window + sinks) * 128))))
            return dict(op=op, dtype=dtype, B=B, Hq=Hq, Hk=Hk, d=d, window=window, sinks=sinks,
                        pool=B + rng.randrange(0, 1 + B // 4), idle=rng.randrange(0, 1 + B // 4))
        # 2^38 multiplications at most, 2^35 in fp32
        most = (1 << (38 if dtype == "bf16" else 35)) // (2 * Hq * d * (window + sinks))
        N = _log_int(rng, 1, max(1, min(65536, (1 << 24) // (Hq * 64), most)))
        packed = rng.choice((0, 0, 1, 5, 24))
        B = 1 if packed else rng.choice((1, 1, 2, 3))
        cache = rng.random() < 0.7
        return dict(op=op, dtype=dtype, B=B, Hq=Hq, Hk=Hk, N=max(1, N // B), d=d, window=window,
                    sinks=sinks, packed=packed, past=cache and rng.random() < 0.6, cache=cache,
                    token_major=rng.random() < 0.6)
    D = rng.choice((64, 100, 256, 768, 1000, 1001, 1536, 2048, 4096))
    if op == "conv" or op == "conv_step":
        W, act = rng.choice((2, 3, 4, 4, 4, 5)), rng.random() < 0.7
        if op == "conv_step":
            B = _log_int(rng, 1, 512)
            return dict(op=op, dtype=dtype, B=B, D=D, W=W, act=act,
                        pool=B + rng.randrange(0, 1 + B // 4), idle=rng.randrange(0, 1 + B // 4),
                        wide=rng.random() < 0.5)
        N = _log_int(rng, 1, max(1, min(65536, (1 << 26) // D)))
    else:
        S, G = rng.choice((16, 16, 16, 8, 32, 64)), rng.choice((1, 1, 1, 2))
        D += D % G
        if op == "scan_step":
            B = _log_int(rng, 1, max(1, min(512, (1 << 24) // (D * S))))
            return dict(op=op, dtype=dtype, B=B, D=D, S=S, G=G,
                        pool=B + rng.randrange(0, 1 + B // 4), idle=rng.randrange(0, 1 + B // 4),
                        gate=rng.random() < 0.6)
        N = _log_int(rng, 1, max(1, min(65536, (1 << 29) // (D * S))))
    packed = rng.choice((0, 0, 1, 5, 24, 64))
    B = 1 if packed else rng.choice((1, 1, 2, 3))
    case = dict(op=op, dtype=dtype, B=B, N=max(1, N // B), D=D, packed=packed,
                state=rng.random() < 0.5, wide=rng.random() < 0.5)
    case.update(dict(W=W, act=act) if op == "conv" else dict(S=S, G=G, gate=rng.random() < 0.6))
    return case


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


def _part(x, wide):
    """The values as the first half of a projection's output, or on their own."""
    if not wide:
        return x
    room = torch.empty(x.shape[:-1] + (2 * x.shape[-1],), device=x.device, dtype=x.dtype)
    room[..., :x.shape[-1]] = x
    return room[..., :x.shape[-1]]


def _slots(case, gen):
    """A slot of the pool for each row of a fixed-size batch, -1 for the idle rows."""
    B = case["B"]
    order = torch.randperm(case["pool"], generator=gen, device=DEV)[:B]
    idle = torch.zeros(B, dtype=torch.bool, device=DEV)
    idle[torch.randperm(B, generator=gen, device=DEV)[:min(case["idle"], B - 1)]] = True
    slots = torch.where(idle, torch.full_like(order, -1), order).to(torch.int32)
    return slots, torch.nonzero(~idle).flatten()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def r(*shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)

    s, dt, op = dict(case), _dt(case["dtype"]), case["op"]
    step = op.endswith("_step")
    B = case["B"]
    if step:
        s["slots"], s["active"] = _slots(case, gen)
    else:
        N, n_seq = case["N"], case["packed"] or B
        s["lengths"] = [N] * B
        s["starts"] = None
        if case["packed"]:
            cpu = torch.Generator()
            cpu.manual_seed(seed)
            s["lengths"] = _lengths(N, n_seq, cpu)
            s["starts"] = torch.tensor([0] + s["lengths"]).cumsum(0).to(torch.int32).to(DEV)
    if op.startswith("attn"):
        Hq, Hk, d, window, sinks = (case[n] for n in ("Hq", "Hk", "d", "window", "sinks"))
        # queries share a direction and the first keys lie along it, so that these draw weight
        u = torch.nn.functional.normalize(r(d), dim=0)
        lift = 2.0 * math.sqrt(d) * u
        places = sinks + window
        if step:
            s["q"] = (r(B, Hq, d) + 2 * u).to(dt)
            s["k"], s["v"] = r(B, Hk, d).to(dt), r(B, Hk, d).to(dt)
            ck, cv = r(case["pool"], Hk, places, d), r(case["pool"], Hk, places, d).to(dt)
            ck[:, :, :sinks] += lift
            s["cache_k"], s["cache_v"] = ck.to(dt), cv
            # half of the rows far into their text, the others anywhere in their first windows
            near = torch.randint(0, 2 * places, (B,), generator=gen, device=DEV)
            far = torch.randint(places, 1 << 20, (B,), generator=gen, device=DEV)
            half = torch.rand(B, generator=gen, device=DEV) < 0.5
            pos = torch.where(half, near, far) if B > 1 else far
            s["positions"] = pos.to(torch.int32)
            return s
        shape = (lambda H: (B, N, H, d)) if case["token_major"] else (lambda H: (B, H, N, d))
        view = (lambda x: x.transpose(1, 2)) if case["token_major"] else (lambda x: x)
        s["q"] = view((r(*shape(Hq)) + 2 * u).to(dt))
        s["k"], s["v"] = view(r(*shape(Hk)).to(dt)), view(r(*shape(Hk)).to(dt))
        s["past"] = s["cache_k"] = s["cache_v"] = s["slots"] = None
        if case["cache"]:
            pool = n_seq + 3
            ck, cv = r(pool, Hk, places, d), r(pool, Hk, places, d).to(dt)
            ck[:, :, :sinks] += lift
            s["cache_k"], s["cache_v"] = ck.to(dt), cv
            s["slots"] = torch.randperm(pool, generator=gen, device=DEV)[:n_seq].to(torch.int32)
        if case["past"]:
            past = torch.randint(0, 3 * places, (n_seq,), generator=gen, device=DEV)
            s["past"] = (past * (torch.rand(n_seq, generator=gen, device=DEV) < 0.75)).to(torch.int32)
        elif case["packed"] == 0 and sinks:
            s["k"][:, :, :sinks] += lift.to(dt)
        return s
    D = case["D"]
    wide = case.get("wide", False)
    if op.startswith("conv"):
        W = case["W"]
        s["w"], s["bias"] = r(D, W) / math.sqrt(W), 0.1 * r(D)
        s["x"] = _part(r(*((B, D) if step else (B, N, D))).to(dt), wide)
        if step:
            s["state"] = r(case["pool"], W - 1, D).to(dt)
        else:
            s["state"] = r(n_seq, W - 1, D).to(dt) if case["state"] else None
        return s
    S, G = case["S"], case["G"]
    rows = (B,) if step else (B, N)
    x = r(*rows, D)
    s["x"] = _part((x * torch.sigmoid(x)).to(dt), wide)  # what leaves the convolution
    s["z"] = _part(r(*rows, D).to(dt), wide) if case["gate"] else None
    s["B_"], s["C_"] = r(*rows, G, S).to(dt), r(*rows, G, S).to(dt)
    # time steps from 0.001 to 0.1 around the bias, A = -(1 .. S)
    mid = 0.001 * torch.exp(torch.rand(D, generator=gen, device=DEV) * math.log(100.0))
    s["dt_bias"] = mid + torch.log(-torch.expm1(-mid))
    s["dt"] = (0.5 * r(*rows, D)).to(dt)
    s["A"] = -torch.arange(1, S + 1, device=DEV, dtype=torch.float32) * torch.exp(0.1 * r(D, S))
    s["Dx"] = 1.0 + 0.1 * r(D)
    if step:
        s["state"] = 0.3 * r(case["pool"], D, S)
    else:
        s["state"] = 0.3 * r(n_seq, D, S) if case["state"] else None
    return s


# ---------------------------------------------------------------- plain forms


def _held(s):
    """For a packed batch: the token of each place of a [sequences, longest] array, and which
    places hold one."""
    longest = max(1, max(s["lengths"]))
    at = torch.arange(longest, device=DEV)
    starts = s["starts"].long()
    held = at[None] < (starts[1:] - starts[:-1])[:, None]
    return torch.where(held, starts[:-1, None] + at[None], 0), held


def _apart(s, *xs):
    """[B, N, ...] token rows as [sequences, longest, ...], zeros where a sequence has ended."""
    if s["starts"] is None:
        return xs
    idx, held = _held(s)
    return tuple(torch.where(held.view(held.shape + (1,) * (x.dim() - 2)), x[0][idx], 0) for x in xs)


def _back(s, y):
    """[sequences, longest, ...] as the token rows they came from."""
    if s["starts"] is None:
        return y
    idx, held = _held(s)
    out = torch.zeros((1, s["N"]) + y.shape[2:], device=DEV, dtype=y.dtype)
    out[0, idx[held]] = y[held]
    return out


def _ring(p, sinks, window):
    """The place of position p in a cache."""
    return torch.where(p < sinks, p, sinks + (p - sinks) % window)


def _plain_attn(s):
    f = torch.float32
    Hq, Hk, d, window, sinks = (s[n] for n in ("Hq", "Hk", "d", "window", "sinks"))
    group = Hq // Hk
    q, k, v = _apart(s, *(s[n].transpose(1, 2) for n in ("q", "k", "v")))  # [n, L, H, d]
    n, L = q.shape[:2]
    lens = torch.tensor(s["lengths"], device=DEV)
    past = s["past"].long() if s["past"] is not None else torch.zeros(n, device=DEV, dtype=torch.long)
    q, k32, v32 = q.to(f), k.to(f), v.to(f)
    block = min(256, L)
    pad = -L % block
    nb = (L + pad) // block
    # the keys before the first new one, in the order of their positions, then the new ones
    before = past[:, None] - window + torch.arange(window, device=DEV)[None]
    first = torch.arange(sinks, device=DEV)[None].expand(n, sinks)
    if s["past"] is not None:
        slot = s["slots"].long()[:, None]
        at = _ring(before.clamp(min=0), sinks, window)
        kb, vb = (c[slot, :, at].to(f) for c in (s["cache_k"], s["cache_v"]))
        kf, vf = (c[slot, :, first].to(f) for c in (s["cache_k"], s["cache_v"]))
    else:
        kb = torch.zeros(n, window, Hk, d, device=DEV, dtype=f)
        vb = kb
        kf = vf = torch.zeros(n, sinks, Hk, d, device=DEV, dtype=f)
    new = (first - past[:, None]).clamp(min=0, max=L - 1)
    seq = torch.arange(n, device=DEV)[:, None]
    late = (first >= past[:, None])[..., None, None]
    kf, vf = torch.where(late, k32[seq, new], kf), torch.where(late, v32[seq, new], vf)
    ke, ve = (torch.nn.functional.pad(torch.cat(x, 1), (0, 0, 0, 0, 0, pad))
              for x in ((kb, k32), (vb, v32)))
    q = torch.nn.functional.pad(q, (0, 0, 0, 0, 0, pad)) * d ** -0.5
    # block b's queries see the keys b * block .. (b + 1) * block + window of that order
    see = torch.arange(nb, device=DEV)[:, None] * block + torch.arange(block + window, device=DEV)
    pos_q = past[:, None, None] + (torch.arange(nb * block, device=DEV)).view(nb, block)[None]
    pos_k = past[:, None, None] - window + see[None]
    dist = pos_q[..., :, None] - pos_k[..., None, :]
    ok = (dist >= 0) & (dist < window) & (pos_k >= sinks)[..., None, :]
    ok = torch.cat((first[:, None, None, :] <= pos_q[..., None], ok), -1)  # [n, nb, block, keys]
    qh = q.view(n, nb, block, Hk, group, d).permute(0, 3, 4, 1, 2, 5)      # [n, Hk, group, nb, block, d]
    kh, vh = (x.permute(0, 2, 1, 3)[:, :, see].unsqueeze(2) for x in (ke, ve))  # [n, Hk, 1, nb, keys, d]
    kf, vf = (x.permute(0, 2, 1, 3)[:, :, None, None] for x in (kf, vf))
    w = torch.cat((qh @ kf.transpose(-1, -2), qh @ kh.transpose(-1, -2)), -1)
    w.masked_fill_(~ok[:, None, None], -math.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    o = w[..., :sinks] @ vf + w[..., sinks:] @ vh
    o = o.permute(0, 3, 4, 1, 2, 5).reshape(n, nb * block, Hq, d)[:, :L]
    out = _back(s, o).transpose(1, 2).to(s["q"].dtype)
    if s["cache_k"] is None:
        return (out,)
    t = torch.arange(L, device=DEV)[None]
    end = past[:, None] + lens[:, None]
    keep = (t < lens[:, None]) & ((past[:, None] + t < sinks) | (past[:, None] + t >= end - window))
    i, j = torch.nonzero(keep, as_tuple=True)
    place = _ring(past[i] + j, sinks, window)
    s["cache_k"][s["slots"].long()[i], :, place] = k[i, j]
    s["cache_v"][s["slots"].long()[i], :, place] = v[i, j]
    return out, s["cache_k"], s["cache_v"]


def _plain_attn_step(s):
    f = torch.float32
    at, window, sinks = s["active"], s["window"], s["sinks"]
    slots, pos = s["slots"][at].long(), s["positions"][at].long()
    place = _ring(pos, sinks, window)
    s["cache_k"][slots, :, place] = s["k"][at]
    s["cache_v"][slots, :, place] = s["v"][at]
    q = s["q"][at].to(f).unflatten(1, (s["Hk"], -1)) * s["d"] ** -0.5
    w = q @ s["cache_k"][slots].to(f).transpose(-1, -2)
    seen = torch.arange(window + sinks, device=DEV)[None] <= pos[:, None]
    w = w.masked_fill(~seen[:, None, None], -math.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True))
    o = (w / w.sum(-1, keepdim=True)) @ s["cache_v"][slots].to(f)
    out = torch.zeros_like(s["q"])
    out[at] = o.flatten(1, 2).to(out.dtype)
    return out, s["cache_k"], s["cache_v"]


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _plain_scan(s):
    f = torch.float32
    D, S, G = s["D"], s["S"], s["G"]
    x, dt, Bm, Cm = _apart(s, *(s[n].to(f) for n in ("x", "dt", "B_", "C_")))
    n, L = x.shape[:2]
    dt = _softplus(dt + s["dt_bias"])
    if s["starts"] is not None:
        dt = dt * _held(s)[1][..., None]  # nothing happens behind a sequence's end
    Bm, Cm = (m.repeat_interleave(D // G, 2) for m in (Bm, Cm)) if G > 1 else (Bm, Cm)
    a = torch.exp(dt[..., None] * s["A"])          # [n, L, D, S]
    h = (dt * x)[..., None] * Bm
    if s["state"] is not None:
        h[:, 0] += a[:, 0] * s["state"]
    k = 1
    while k < L:                                   # h_t over the last k tokens -> over 2 k
        h[:, k:] = h[:, k:] + a[:, k:] * h[:, :-k]
        a[:, k:] = a[:, k:] * a[:, :-k]
        k *= 2
    y = (h * Cm).sum(-1) + s["Dx"] * x
    last = h[:, -1].clone()
    y = _back(s, y)
    if s["z"] is not None:
        z = s["z"].to(f)
        y = y * z * torch.sigmoid(z)
    return y.to(s["x"].dtype), last


def _plain_scan_step(s):
    f = torch.float32
    at, D, G = s["active"], s["D"], s["G"]
    slots = s["slots"][at].long()
    x, dt, Bm, Cm = (s[n][at].to(f) for n in ("x", "dt", "B_", "C_"))
    dt = _softplus(dt + s["dt_bias"])
    Bm, Cm = (m.repeat_interleave(D // G, 1) for m in (Bm, Cm))
    h = torch.exp(dt[..., None] * s["A"]) * s["state"][slots] + (dt * x)[..., None] * Bm
    y = (h * Cm).sum(-1) + s["Dx"] * x
    if s["z"] is not None:
        z = s["z"][at].to(f)
        y = y * z * torch.sigmoid(z)
    s["state"][slots] = h
    out = torch.zeros(s["x"].shape, device=DEV, dtype=s["x"].dtype)
    out[at] = y.to(out.dtype)
    return out, s["state"]


def _plain_conv(s):
    f = torch.float32
    W = s["W"]
    x, = _apart(s, s["x"])
    n, L, D = x.shape
    old = s["state"] if s["state"] is not None else torch.zeros(n, W - 1, D, device=DEV, dtype=x.dtype)
    ext = torch.cat((old, x), 1)
    y = (ext.to(f).unfold(1, W, 1) * s["w"]).sum(-1) + s["bias"]
    if s["act"]:
        y = y * torch.sigmoid(y)
    ends = torch.tensor(s["lengths"], device=DEV)[:, None] + torch.arange(W - 1, device=DEV)
    state = ext[torch.arange(n, device=DEV)[:, None], ends]
    return _back(s, y).to(x.dtype), state


def _plain_conv_step(s):
    f = torch.float32
    at = s["active"]
    slots = s["slots"][at].long()
    ext = torch.cat((s["state"][slots], s["x"][at][:, None]), 1)
    y = (ext.to(f) * s["w"].t()).sum(1) + s["bias"]
    if s["act"]:
        y = y * torch.sigmoid(y)
    s["state"][slots] = ext[:, 1:]
    out = torch.zeros(s["x"].shape, device=DEV, dtype=s["x"].dtype)
    out[at] = y.to(out.dtype)
    return out, s["state"]


# ---------------------------------------------------------------- the library's calls


def _own_attn(s):
    import chunked_linear_attention_gb300 as cla
    out = cla.window_attention_forward(s["q"], s["k"], s["v"], s["window"], sinks=s["sinks"],
                                       cache_k=s["cache_k"], cache_v=s["cache_v"],
                                       slots=s["slots"], past=s["past"], seq_starts=s["starts"])
    return (out,) if s["cache_k"] is None else (out, s["cache_k"], s["cache_v"])


def _own_attn_step(s):
    import chunked_linear_attention_gb300 as cla
    out = cla.window_attention_step(s["q"], s["k"], s["v"], s["cache_k"], s["cache_v"],
                                    s["positions"], s["window"], sinks=s["sinks"], slots=s["slots"])
    return out, s["cache_k"], s["cache_v"]


def _own_scan(s):
    import chunked_linear_attention_gb300 as cla
    return cla.selective_scan_forward(s["x"], s["dt"], s["A"], s["B_"], s["C_"], D=s["Dx"],
                                      dt_bias=s["dt_bias"], z=s["z"], state=s["state"],
                                      seq_starts=s["starts"])


def _own_scan_step(s):
    import chunked_linear_attention_gb300 as cla
    out = cla.selective_scan_step(s["x"], s["dt"], s["A"], s["B_"], s["C_"], s["state"], D=s["Dx"],
                                  dt_bias=s["dt_bias"], z=s["z"], slots=s["slots"])
    return out, s["state"]


def _own_conv(s):
    import chunked_linear_attention_gb300 as cla
    return cla.short_conv_forward(s["x"], s["w"], bias=s["bias"], silu=s["act"], state=s["state"],
                                  seq_starts=s["starts"])


def _own_conv_step(s):
    import chunked_linear_attention_gb300 as cla
    out = cla.short_conv_step(s["x"], s["w"], s["state"], bias=s["bias"], silu=s["act"],
                              slots=s["slots"])
    return out, s["state"]


def run(state):
    if own:
        return {"attn": _own_attn, "attn_step": _own_attn_step, "scan": _own_scan,
                "scan_step": _own_scan_step, "conv": _own_conv,
                "conv_step": _own_conv_step}[state["op"]](state)
    return {"attn": _plain_attn, "attn_step": _plain_attn_step, "scan": _plain_scan,
            "scan_step": _plain_scan_step, "conv": _plain_conv,
            "conv_step": _plain_conv_step}[state["op"]](state)


# ---------------------------------------------------------------- work and the definition


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    op, B = case["op"], case["B"]
    live = B - min(case["idle"], B - 1) if op.endswith("_step") else 0
    if op.startswith("attn"):
        Hq, Hk, d, window, sinks = (case[n] for n in ("Hq", "Hk", "d", "window", "sinks"))
        if op == "attn_step":
            # the visible keys and values once, the new token's into the cache
            pairs = live * (window + sinks)
            return {"bytes": size * d * (2 * Hk * (pairs + 2 * live) + 2 * Hq * live),
                    "flops": 4 * d * Hq * pairs}
        N, n_seq = case["N"], case["packed"] or B
        tokens, L = B * N, max(1, B * N // n_seq)
        seen = window + sinks if case["past"] else min(window + sinks, L)
        kept = n_seq * min(L, window + sinks) if case["cache"] else 0
        old = n_seq * (window + sinks) if case["past"] else 0
        pairs = tokens * seen - (0 if case["past"] else n_seq * seen * (seen - 1) // 2)
        return {"bytes": size * d * (2 * Hq * tokens + 2 * Hk * (tokens + kept + old)),
                "flops": 4 * d * Hq * pairs}
    D = case["D"]
    if op.startswith("conv"):
        W = case["W"]
        if op == "conv_step":
            return {"bytes": live * D * size * (2 + 2 * (W - 1)) + 4 * D * (W + 1),
                    "flops": 2 * live * D * W}
        n_seq = case["packed"] or B
        return {"bytes": size * D * (2 * B * case["N"] + n_seq * (W - 1) * (1 + case["state"])) + 4 * D * (W + 1),
                "flops": 2 * B * case["N"] * D * W}
    S, G = case["S"], case["G"]
    row = size * (D * (3 + case["gate"]) + 2 * G * S)
    if op == "scan_step":
        return {"bytes": live * (row + 8 * D * S) + 4 * D * (S + 2), "flops": 6 * live * D * S}
    n_seq = case["packed"] or B
    return {"bytes": B * case["N"] * row + 4 * n_seq * D * S * (1 + case["state"]) + 4 * D * (S + 2),
            "flops": 6 * B * case["N"] * D * S}


def _spans(s):
    """(batch, first token, behind the last) of each sequence."""
    if s["starts"] is None:
        return [(b, 0, s["N"]) for b in range(s["B"])]
    at = [0]
    for x in s["lengths"]:
        at.append(at[-1] + x)
    return [(0, at[i], at[i + 1]) for i in range(len(s["lengths"]))]


def _place(p, s):
    return p if p < s["sinks"] else s["sinks"] + (p - s["sinks"]) % s["window"]


def _exact_attn(s):
    e = torch.float64
    window, sinks, group = s["window"], s["sinks"], s["Hq"] // s["Hk"]
    out = torch.zeros(s["q"].shape, device=DEV, dtype=e)
    caches = [None if c is None else c.clone() for c in (s["cache_k"], s["cache_v"])]
    for i, (b, t0, t1) in enumerate(_spans(s)):
        n = t1 - t0
        P = int(s["past"][i]) if s["past"] is not None else 0
        # positions that the cache holds, then the new ones: keys in the order of positions
        old = sorted(set(range(min(P, sinks))) | set(range(max(0, P - window), P)))
        pos = torch.tensor(old + list(range(P, P + n)), device=DEV)
        if caches[0] is not None:
            slot = int(s["slots"][i])
            at = torch.tensor([_place(p, s) for p in old], device=DEV, dtype=torch.long)
        for h in range(s["Hk"]):
            k, v = (x[b, h, t0:t1].to(e) for x in (s["k"], s["v"]))
            if old:
                k, v = (torch.cat((c[slot, h, at].to(e), x)) for c, x in zip((s["cache_k"], s["cache_v"]), (k, v)))
            m = len(old)
            for q0 in range(0, n, 1024):
                q1 = min(n, q0 + 1024)
                # new keys from the first that the block's first query sees
                lo = max(0, q0 - window + 1)
                part = torch.cat((torch.arange(min(m + max(0, sinks - P), m + lo), device=DEV),
                                  torch.arange(m + lo, m + q1, device=DEV)))
                pk, pq = pos[part][None], (P + torch.arange(q0, q1, device=DEV))[:, None]
                ok = (pk <= pq) & ((pk < sinks) | (pq - pk < window))
                q = s["q"][b, h * group:(h + 1) * group, t0 + q0:t0 + q1].to(e)
                w = torch.matmul(q, k[part].t()) / math.sqrt(s["d"])
                w = torch.where(ok, w, -math.inf)
                w = torch.exp(w - w.max(-1, keepdim=True).values)
                o = torch.matmul(w, v[part]) / w.sum(-1, keepdim=True)
                out[b, h * group:(h + 1) * group, t0 + q0:t0 + q1] = o
        if caches[0] is not None and n:
            kept = [p for p in range(P, P + n) if p < sinks or p >= P + n - window]
            to = torch.tensor([_place(p, s) for p in kept], device=DEV)
            of = torch.tensor([t0 + p - P for p in kept], device=DEV)
            caches[0][slot][:, to] = s["k"][b][:, of]
            caches[1][slot][:, to] = s["v"][b][:, of]
    return (out,) if caches[0] is None else (out, caches[0].to(e), caches[1].to(e))


def _exact_attn_step(s):
    e = torch.float64
    out = torch.zeros(s["q"].shape, device=DEV, dtype=e)
    ck, cv = s["cache_k"].clone(), s["cache_v"].clone()
    group = s["Hq"] // s["Hk"]
    for b in s["active"].tolist():
        slot, t = int(s["slots"][b]), int(s["positions"][b])
        ck[slot, :, _place(t, s)] = s["k"][b]
        cv[slot, :, _place(t, s)] = s["v"][b]
        m = min(t + 1, s["sinks"] + s["window"])
        q = s["q"][b].to(e).view(s["Hk"], group, s["d"])
        w = torch.einsum("hgd,hmd->hgm", q, ck[slot, :, :m].to(e)) / math.sqrt(s["d"])
        w = torch.exp(w - w.max(-1, keepdim=True).values)
        o = torch.einsum("hgm,hmd->hgd", w, cv[slot, :, :m].to(e)) / w.sum(-1, keepdim=True)
        out[b] = o.reshape(s["Hq"], s["d"])
    return out, ck.to(e), cv.to(e)


def _exact_token(s, x, dt, Bt, Ct, h):
    """One token of the scan in 64 bits: its output before the gate, and the state."""
    e = torch.float64
    per = s["D"] // s["G"]
    dt = torch.log1p(torch.exp(dt.to(e) + s["dt_bias"].to(e)))[..., None]
    Bt, Ct = (m.to(e).repeat_interleave(per, -2) for m in (Bt, Ct))
    h = h * torch.exp(dt * s["A"].to(e)) + dt * x.to(e)[..., None] * Bt
    return torch.einsum("...ds,...ds->...d", h, Ct) + s["Dx"].to(e) * x.to(e), h


def _exact_scan(s):
    e = torch.float64
    spans = _spans(s)
    out = torch.zeros(s["x"].shape, device=DEV, dtype=e)
    lens = [t1 - t0 for _, t0, t1 in spans]
    by = sorted(range(len(spans)), key=lambda i: -lens[i])  # longest first: the live ones are a prefix
    h = torch.zeros(len(spans), s["D"], s["S"], device=DEV, dtype=e)
    if s["state"] is not None:
        h = s["state"].to(e)[by]
    batch = torch.tensor([spans[i][0] for i in by], device=DEV)
    first = torch.tensor([spans[i][1] for i in by], device=DEV)
    for t in range(max(lens)):
        m = sum(x > t for x in lens)
        at = batch[:m], first[:m] + t
        out[at], h[:m] = _exact_token(s, s["x"][at], s["dt"][at], s["B_"][at], s["C_"][at], h[:m])
    if s["z"] is not None:
        z = s["z"].to(e)
        out = out * z / (1 + torch.exp(-z))
    state = torch.empty_like(h)
    state[by] = h
    return out, state


def _exact_scan_step(s):
    e = torch.float64
    at = s["active"]
    slots = s["slots"][at].long()
    out, state = torch.zeros(s["x"].shape, device=DEV, dtype=e), s["state"].to(e)
    y, h = _exact_token(s, s["x"][at], s["dt"][at], s["B_"][at], s["C_"][at], state[slots])
    if s["z"] is not None:
        z = s["z"][at].to(e)
        y = y * z / (1 + torch.exp(-z))
    state[slots] = h
    out[at] = y
    return out, state


def _exact_conv(s):
    e = torch.float64
    W, w = s["W"], s["w"].to(e)
    out = torch.zeros(s["x"].shape, device=DEV, dtype=e)
    spans = _spans(s)
    state = torch.zeros(len(spans), W - 1, s["D"], device=DEV, dtype=e)
    if s["state"] is not None:
        state = s["state"].to(e)
    for i, (b, t0, t1) in enumerate(spans):
        rows = torch.cat((state[i], s["x"][b, t0:t1].to(e)))
        y = s["bias"].to(e).repeat(t1 - t0, 1)
        for j in range(W):
            y += w[:, j] * rows[j:j + t1 - t0]
        out[b, t0:t1] = y / (1 + torch.exp(-y)) if s["act"] else y
        state[i] = rows[t1 - t0:]
    return out, state


def _exact_conv_step(s):
    e = torch.float64
    at = s["active"]
    slots = s["slots"][at].long()
    out, state = torch.zeros(s["x"].shape, device=DEV, dtype=e), s["state"].to(e)
    y = torch.einsum("bjd,dj->bd", state[slots], s["w"][:, :-1].to(e))
    y = y + s["x"][at].to(e) * s["w"][:, -1].to(e) + s["bias"].to(e)
    state[slots] = torch.cat((state[slots][:, 1:], s["x"][at].to(e)[:, None]), 1)
    out[at] = y / (1 + torch.exp(-y)) if s["act"] else y
    return out, state


def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "attn_step": _exact_attn_step, "scan": _exact_scan,
            "scan_step": _exact_scan_step, "conv": _exact_conv,
            "conv_step": _exact_conv_step}[case["op"]](s)
