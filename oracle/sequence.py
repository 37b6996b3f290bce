"""Float64 oracle of multi-head decay attention and of LayerNorm's gradient:
the recurrences token by token, in numpy.  Test infrastructure only; shares no
code with the library.

Each function also returns the sums of the absolute values of the terms its
results are made of, which bound how far float32 arithmetic can be off.
"""
import numpy as np


def _split(x, H):
    B, T, C = x.shape
    return np.asarray(x, np.float64).reshape(B, T, H, C // H)


def decay_attn(q, k, v, w, H, scale=1.0, state=None, lengths=None):
    """out (B, T, C), final state (B, H, D, D), and their magnitudes."""
    B, T, C = q.shape
    D = C // H
    q, k, v = (_split(a, H) for a in (q, k, v))
    lam = np.exp(-np.asarray(w, np.float64))[:, None, None]
    S = np.zeros((B, H, D, D)) if state is None else np.array(state, np.float64)
    M = np.abs(S)
    out, mag = np.zeros((B, T, H, D)), np.zeros((B, T, H, D))
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        for t in range(n):
            S[b] = lam * S[b] + k[b, t][:, :, None] * v[b, t][:, None, :]
            M[b] = lam * M[b] + np.abs(k[b, t])[:, :, None] * np.abs(v[b, t])[:, None, :]
            out[b, t] = scale * np.einsum("hi,hij->hj", q[b, t], S[b])
            mag[b, t] = abs(scale) * np.einsum("hi,hij->hj", np.abs(q[b, t]), M[b])
    return out.reshape(B, T, C), S, mag.reshape(B, T, C), M


def decay_attn_bwd(q, k, v, w, H, gy, scale=1.0, state=None, gstate=None, lengths=None):
    """(gq, gk, gv, gstate_in) and their magnitudes, by the adjoint recurrence."""
    B, T, C = q.shape
    D = C // H
    q, k, v, g = (_split(a, H) for a in (q, k, v, gy))
    lam = np.exp(-np.asarray(w, np.float64))[:, None, None]
    grads = [np.zeros((B, T, H, D)) for _ in range(3)]
    mags = [np.zeros((B, T, H, D)) for _ in range(3)]
    S = np.zeros((B, H, D, D)) if state is None else np.array(state, np.float64)
    G = np.zeros((B, H, D, D)) if gstate is None else np.array(gstate, np.float64)
    M, N = np.abs(S), np.abs(G)
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        for t in range(n):
            S[b] = lam * S[b] + k[b, t][:, :, None] * v[b, t][:, None, :]
            M[b] = lam * M[b] + np.abs(k[b, t])[:, :, None] * np.abs(v[b, t])[:, None, :]
            grads[0][b, t] = scale * np.einsum("hij,hj->hi", S[b], g[b, t])
            mags[0][b, t] = abs(scale) * np.einsum("hij,hj->hi", M[b], np.abs(g[b, t]))
        for t in range(n - 1, -1, -1):
            G[b] = G[b] + scale * q[b, t][:, :, None] * g[b, t][:, None, :]
            N[b] = N[b] + abs(scale) * np.abs(q[b, t])[:, :, None] * np.abs(g[b, t])[:, None, :]
            grads[1][b, t] = np.einsum("hij,hj->hi", G[b], v[b, t])
            mags[1][b, t] = np.einsum("hij,hj->hi", N[b], np.abs(v[b, t]))
            grads[2][b, t] = np.einsum("hij,hi->hj", G[b], k[b, t])
            mags[2][b, t] = np.einsum("hij,hi->hj", N[b], np.abs(k[b, t]))
            G[b] = lam * G[b]
            N[b] = lam * N[b]
    return ([a.reshape(B, T, C) for a in grads] + [G], [a.reshape(B, T, C) for a in mags] + [N])


def decay_attn_step(q, k, v, w, H, state, slots, scale=1.0):
    """One token per row: out (B, C), the new pool, and out's magnitude."""
    B, C = q.shape
    D = C // H
    q, k, v = (np.asarray(a, np.float64).reshape(B, H, D) for a in (q, k, v))
    lam = np.exp(-np.asarray(w, np.float64))[:, None, None]
    pool = np.array(state, np.float64)
    out, mag = np.zeros((B, H, D)), np.zeros((B, H, D))
    for b, slot in enumerate(slots):
        if slot < 0 or slot >= len(pool) or slot in list(slots[:b]):
            continue
        kv = k[b][:, :, None] * v[b][:, None, :]
        m = lam * np.abs(pool[slot]) + np.abs(kv)
        pool[slot] = lam * pool[slot] + kv
        out[b] = scale * np.einsum("hi,hij->hj", q[b], pool[slot])
        mag[b] = abs(scale) * np.einsum("hi,hij->hj", np.abs(q[b]), m)
    return out.reshape(B, C), pool, mag.reshape(B, C)


def layer_norm_fwd(x, gamma, beta, eps):
    x = np.asarray(x, np.float64)
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    return gamma * (x - mean[..., None]) * rstd[..., None] + beta, mean, rstd


def layer_norm_bwd(x, gamma, mean, rstd, gy):
    """gx, ggamma, gbeta and their magnitudes, rows as the leading dimensions."""
    C = x.shape[-1]
    x, gy = (np.asarray(a, np.float64).reshape(-1, C) for a in (x, gy))
    mean, rstd = (np.asarray(a, np.float64).reshape(-1, 1) for a in (mean, rstd))
    xh = (x - mean) * rstd
    d = gamma * gy
    gx = rstd * (d - d.mean(-1, keepdims=True) - xh * (d * xh).mean(-1, keepdims=True))
    mx = rstd * (np.abs(d) + np.abs(d).mean(-1, keepdims=True) + np.abs(xh) * np.abs(d * xh).mean(-1, keepdims=True))
    return ((gx, (gy * xh).sum(0), gy.sum(0)), (mx, np.abs(gy * xh).sum(0), np.abs(gy).sum(0)))
