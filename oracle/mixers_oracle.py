"""fp64 oracle of the fixed-state mixers: attention with a sliding window and
sinks, the selective state space scan, the short causal convolution.

Written from the definitions, one query (one token) at a time, in numpy;
shares no code with the CUDA library.  Each function also returns how far a
computation in fp32 may be from its results, from the roundings on the way
(u = 2^-24, half a step of fp32 relative to the value): the caller adds the
rounding of the output.
"""
import numpy as np

U = 2.0 ** -24


def spans(B, N, starts=None):
    """(batch, first token, behind the last) of each sequence."""
    if starts is None:
        return [(b, 0, N) for b in range(B)]
    return [(0, int(starts[i]), int(starts[i + 1])) for i in range(len(starts) - 1)]


def place(p, window, sinks):
    """Where a cache holds position p."""
    return p if p < sinks else sinks + (p - sinks) % window


def visible(t, window, sinks):
    """The positions that position t sees, in order."""
    return [j for j in range(t + 1) if j < sinks or t - j < window]


def attend(q, K, V, scale, weight_rounding=0.0):
    """One query [d] over keys and values [n, d].  Returns (out, bound)."""
    s = scale * (K @ q)
    w = np.exp(s - s.max())
    w /= w.sum()
    # a score is off by (d + 2) u of its products' absolute sum (the scaling of q and the
    # base-2 form among them), a weight by the errors of its score and of the largest, the
    # exponential by 2^-21 more, the sums over n keys by n u each
    ds = (len(q) + 6) * U * abs(scale) * (np.abs(K) @ np.abs(q)).max()
    rel = 4 * ds + 2.0 ** -20 + 3 * len(w) * U + weight_rounding
    return w @ V, rel * (w @ np.abs(V))


def window_attention(q, k, v, window, sinks=0, scale=None, caches=None, slots=None, past=None,
                     starts=None, weight_rounding=0.0):
    """q [B, Hq, N, d], k, v [B, Hk, N, d] float64; caches: (K, V) arrays
    [n_slots, Hk, sinks + window, d], updated in place.  Returns (out, bound);
    rows of no sequence are NaN."""
    B, Hq, N, d = q.shape
    Hk = k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out = np.full(q.shape, np.nan)
    bound = np.full(q.shape, np.nan)
    old = None if caches is None else [c.copy() for c in caches]
    for s, (b, t0, t1) in enumerate(spans(B, N, starts)):
        slot = -1 if caches is None else s if slots is None else int(slots[s])
        P = 0 if past is None or slot < 0 else int(past[s])
        for i in range(t1 - t0):
            see = visible(P + i, window, sinks)
            for h in range(Hk):
                K = np.stack([old[0][slot, h, place(j, window, sinks)] if j < P else
                              k[b, h, t0 + j - P] for j in see])
                V = np.stack([old[1][slot, h, place(j, window, sinks)] if j < P else
                              v[b, h, t0 + j - P] for j in see])
                for g in range(h * Hq // Hk, (h + 1) * Hq // Hk):
                    out[b, g, t0 + i], bound[b, g, t0 + i] = attend(q[b, g, t0 + i], K, V, scale,
                                                                    weight_rounding)
        if slot >= 0:
            for p in range(P, P + t1 - t0):
                if p < sinks or p >= P + t1 - t0 - window:
                    for c, x in zip(caches, (k, v)):
                        c[slot, :, place(p, window, sinks)] = x[b, :, t0 + p - P]
    return out, bound


def window_attention_step(q, k, v, caches, positions, window, sinks=0, scale=None, slots=None):
    """q [B, Hq, d], k, v [B, Hk, d]; caches updated in place.  Idle rows are 0."""
    B, Hq, d = q.shape
    Hk = k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        slot = b if slots is None else int(slots[b])
        if slot < 0:
            continue
        t = int(positions[b])
        for c, x in zip(caches, (k, v)):
            c[slot, :, place(t, window, sinks)] = x[b]
        at = [place(j, window, sinks) for j in visible(t, window, sinks)]
        for g in range(Hq):
            h = g // (Hq // Hk)
            out[b, g], bound[b, g] = attend(q[b, g], caches[0][slot, h, at], caches[1][slot, h, at],
                                            scale)
    return out, bound


def _sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def selective_scan(x, dt, A, B, C, D=None, dt_bias=None, z=None, softplus=True, state=None,
                   starts=None):
    """x, dt, z [nb, N, ch], B, C [nb, N, G, S], A [ch, S].  Returns (out,
    states, bound of out, bound of the states); rows of no sequence are NaN."""
    nb, N, ch = x.shape
    G, S = B.shape[2:]
    sp = spans(nb, N, starts)
    out, eo = np.full(x.shape, np.nan), np.full(x.shape, np.nan)
    hs = np.zeros((len(sp), ch, S)) if state is None else np.array(state, dtype=np.float64)
    es = np.zeros_like(hs)
    for s, (b, t0, t1) in enumerate(sp):
        h, e, ha = hs[s], np.zeros((ch, S)), np.abs(hs[s])
        for t in range(t0, t1):
            raw = dt[b, t] + (0.0 if dt_bias is None else dt_bias)
            r = np.logaddexp(0.0, raw) if softplus else raw
            # the step: its argument's rounding, an exponential, a quotient and a short series
            er = 2.0 ** -20 + 4 * U * np.abs(raw)
            Bt, Ct = (np.repeat(m[b, t], ch // G, axis=0) for m in (B, C))
            a = np.exp(r[:, None] * A)
            u = r * x[b, t]
            # a decay: its argument's error (as a part of a segment's sum, up to N u more), the
            # exponential 2^-21
            ea = np.abs(r[:, None] * A) * (er[:, None] + (N + 4) * U) + 2.0 ** -21
            ub = np.abs(u[:, None] * Bt)
            e = a * (e + ea * ha) + (er[:, None] + 4 * U) * ub
            h = a * h + u[:, None] * Bt
            ha = a * ha + ub
            e = e + 2 * U * ha
            y = (h * Ct).sum(1)
            ey = (np.abs(Ct) * (e + (S + 4) * U * ha)).sum(1)
            if D is not None:
                y = y + D * x[b, t]
                ey = ey + 4 * U * np.abs(D * x[b, t])
            ey = ey + 2 * U * np.abs(y)
            if z is not None:
                gate = z[b, t] * _sigmoid(z[b, t])
                ey = np.abs(gate) * (ey + 2.0 ** -20 * (1 + np.abs(z[b, t]) / 8) * np.abs(y))
                y = y * gate
            out[b, t], eo[b, t] = y, ey
        hs[s], es[s] = h, e
    return out, hs, eo, es


def short_conv(x, w, bias=None, silu=False, state=None, starts=None):
    """x [B, N, D], w [D, W], state [n_seq, W - 1, D].  Returns (out, states,
    bound of out); rows of no sequence are NaN."""
    B, N, D = x.shape
    W = w.shape[1]
    sp = spans(B, N, starts)
    out, eo = np.full(x.shape, np.nan), np.full(x.shape, np.nan)
    st = np.zeros((len(sp), W - 1, D)) if state is None else np.array(state, dtype=np.float64)
    for s, (b, t0, t1) in enumerate(sp):
        rows = np.concatenate((st[s], x[b, t0:t1]))
        for i in range(t1 - t0):
            part = rows[i:i + W] * w.T
            y = part.sum(0) + (0.0 if bias is None else bias)
            e = (W + 2) * U * (np.abs(part).sum(0) + (0.0 if bias is None else np.abs(bias)))
            if silu:
                # the slope of x sigmoid(x) stays below 1.1
                e = 1.1 * e + 2.0 ** -20 * (1 + np.abs(y) / 8) * np.abs(y * _sigmoid(y))
                y = y * _sigmoid(y)
            out[b, t0 + i], eo[b, t0 + i] = y, e
        st[s] = rows[t1 - t0:]
    return out, st, eo
