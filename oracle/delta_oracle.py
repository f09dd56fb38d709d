"""fp64 oracle of the gated delta rule and of the norms around a block.

Written from the definitions, one token (one row) at a time, in numpy; shares
no code with the CUDA library.

Gated delta rule, per sequence and value head (state S [d_v, d_k]):
    S <- exp(g_t) S;  u = beta_t (v_t - S k_t);  S <- S + u k_t^T;
    o_t = scale * S q_t
"""
import numpy as np


def delta_rule(q, k, v, g, beta, S0=None, starts=None, scale=None):
    """q, k [B, Hk, N, dk], v [B, Hv, N, dv], g, beta [B, Hv, N] float64.
    starts: packed sequences along the token axis (B = 1).  Returns
    (out [B, Hv, N, dv], states [n_seq, Hv, dv, dk]); rows of no sequence are
    NaN."""
    B, Hk, N, dk = q.shape
    Hv, dv = v.shape[1], v.shape[-1]
    scale = dk ** -0.5 if scale is None else scale
    spans = [(b, 0, N) for b in range(B)] if starts is None else [
        (0, int(starts[i]), int(starts[i + 1])) for i in range(len(starts) - 1)]
    out = np.full((B, Hv, N, dv), np.nan)
    S = np.zeros((len(spans), Hv, dv, dk)) if S0 is None else np.array(S0, dtype=np.float64)
    for s, (b, t0, t1) in enumerate(spans):
        for h in range(Hv):
            M = S[s, h]
            kh = h // (Hv // Hk)
            for t in range(t0, t1):
                M = np.exp(g[b, h, t]) * M
                u = beta[b, h, t] * (v[b, h, t] - M @ k[b, kh, t])
                M = M + np.outer(u, k[b, kh, t])
                out[b, h, t] = scale * (M @ q[b, kh, t])
            S[s, h] = M
    return out, S


def block_norm(y, w=None, gate=None, act=0, residual=None, scale=None, w_next=None, group=None,
               eps=1e-6):
    """y [rows, D] float64; act 0 none, 1 silu, 2 sigmoid.  Returns (r, h)."""
    rows, D = y.shape
    group = D if group is None else group
    n = np.empty_like(y)
    for c in range(0, D, group):
        part = y[:, c:c + group]
        n[:, c:c + group] = part / np.sqrt(np.mean(part * part, axis=1, keepdims=True) + eps)
        if w is not None:
            n[:, c:c + group] *= w
    if act:
        sg = 1.0 / (1.0 + np.exp(-gate))
        n = n * (gate * sg if act == 1 else sg)
    if scale is not None:
        n = n * scale
    r = n if residual is None else residual + n
    if w_next is None:
        return r, None
    return r, r / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + eps) * w_next
