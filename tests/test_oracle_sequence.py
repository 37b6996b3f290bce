"""Pins of the float64 oracle of decay attention and LayerNorm's gradient:
the double sum against the recurrence, hand-worked values, central differences,
and the identity the kernels rest on (the three token gradients are the
operator itself on exchanged arguments, two of them in reversed time)."""
import numpy as np
import pytest

from oracle import sequence as seq


def _inputs(B, T, H, D, seed, state=True):
    r = np.random.default_rng(seed)
    q, k, v, g = (r.normal(size=(B, T, H * D)) for _ in range(4))
    s, gs = (r.normal(size=(B, H, D, D)) if state else None for _ in range(2))
    return q, k, v, g, s, gs, r.uniform(0.0, 1.5, H)


def test_recurrence_equals_the_double_sum():
    B, T, H, D = 2, 7, 2, 3
    q, k, v, _, s, _, w = _inputs(B, T, H, D, 1)
    out, last, _, _ = seq.decay_attn(q, k, v, w, H, 0.5, s)
    qh, kh, vh = (a.reshape(B, T, H, D) for a in (q, k, v))
    for b in range(B):
        for h in range(H):
            for t in range(T):
                want = np.exp(-w[h] * (t + 1)) * qh[b, t, h] @ s[b, h]
                for i in range(t + 1):
                    want = want + np.exp(-w[h] * (t - i)) * (qh[b, t, h] @ kh[b, i, h]) * vh[b, i, h]
                assert np.allclose(out.reshape(B, T, H, D)[b, t, h], 0.5 * want, rtol=1e-12)
            end = np.exp(-w[h] * T) * s[b, h]
            for i in range(T):
                end = end + np.exp(-w[h] * (T - 1 - i)) * np.outer(kh[b, i, h], vh[b, i, h])
            assert np.allclose(last[b, h], end, rtol=1e-12)


def test_hand_worked_values():
    # one head of one channel, e^-w = 1/2: S = 2*3 = 6, then 6/2 + 1*4 = 7
    q = np.array([[[1.0], [10.0]]])
    k = np.array([[[2.0], [1.0]]])
    v = np.array([[[3.0], [4.0]]])
    out, last, _, _ = seq.decay_attn(q, k, v, [np.log(2.0)], 1)
    assert np.allclose(out.ravel(), [6.0, 70.0]) and np.allclose(last.ravel(), [7.0])


def test_lengths_stop_a_sequence():
    B, T, H, D = 3, 6, 2, 2
    q, k, v, g, s, gs, w = _inputs(B, T, H, D, 2)
    out, last, _, _ = seq.decay_attn(q, k, v, w, H, 1.0, s, [0, 4, 99])
    assert not out[0].any() and np.array_equal(last[0], s[0]) and not out[1, 4:].any()
    o4, l4, _, _ = seq.decay_attn(q[1:2, :4], k[1:2, :4], v[1:2, :4], w, H, 1.0, s[1:2])
    assert np.allclose(out[1, :4], o4[0]) and np.allclose(last[1], l4[0])
    (gq, gk, gv, g0), _ = seq.decay_attn_bwd(q, k, v, w, H, g, 1.0, s, gs, [0, 4, 99])
    assert not gq[0].any() and not gk[1, 4:].any() and np.array_equal(g0[0], gs[0])


@pytest.mark.parametrize("lengths", [None, [5, 3]])
def test_gradients_against_central_differences(lengths):
    B, T, H, D = 2, 5, 2, 3
    q, k, v, g, s, gs, w = _inputs(B, T, H, D, 3)
    grads, _ = seq.decay_attn_bwd(q, k, v, w, H, g, 0.7, s, gs, lengths)

    def loss(q, k, v, s):
        out, last, _, _ = seq.decay_attn(q, k, v, w, H, 0.7, s, lengths)
        return (out * g).sum() + (last * gs).sum()

    args = [q, k, v, s]
    eps = 1e-5
    for a in range(4):
        flat = args[a].ravel()
        for i in np.random.default_rng(a).choice(flat.size, 12, replace=False):
            old = flat[i]
            flat[i] = old + eps
            up = loss(*args)
            flat[i] = old - eps
            down = loss(*args)
            flat[i] = old
            # a polynomial of degree <= 1 in each entry: only rounding is left
            assert abs((up - down) / (2 * eps) - grads[a].ravel()[i]) < 1e-7


def _operator(q, k, v, w, H, x_in, reverse, si, sx, su):
    """The kernels' operator of one problem, written as sums: intra scale si,
    scale sx of the incoming state, su of what is added to it."""
    B, T, C = q.shape
    D = C // H
    q, k, v = (a.reshape(B, T, H, D) for a in (q, k, v))
    pos = np.arange(T)[::-1] if reverse else np.arange(T)
    e0 = 0 if reverse else 1
    wt = w[:, None, None]
    d = pos[:, None] - pos[None, :]
    dec = np.where(d >= 0, np.exp(-wt * np.maximum(d, 0)), 0.0)
    p = np.einsum("bthi,bshi->bhts", q, k) * dec * si
    out = np.einsum("bhts,bshj->bthj", p, v)
    out = out + sx * np.einsum("bthi,bhij,ht->bthj", q, x_in, np.exp(-wt[..., 0] * (pos + e0)))
    x = np.exp(-wt * T)[None] * x_in + su * np.einsum("bthi,bthj,ht->bhij", k, v, np.exp(-wt[..., 0] * (T - pos - e0)))
    return out.reshape(B, T, C), x


def test_gradients_are_the_operator_on_exchanged_arguments():
    B, T, H, D = 2, 6, 2, 3
    q, k, v, g, s, gs, w = _inputs(B, T, H, D, 4)
    c = 0.6
    (gq, gk, gv, g0), _ = seq.decay_attn_bwd(q, k, v, w, H, g, c, s, gs)
    t = lambda x: x.transpose(0, 1, 3, 2)  # noqa: E731
    assert np.allclose(_operator(q, k, v, w, H, s, False, c, c, 1.0)[0], seq.decay_attn(q, k, v, w, H, c, s)[0])
    assert np.allclose(_operator(g, v, k, w, H, t(s), False, c, c, 1.0)[0], gq)
    assert np.allclose(_operator(v, g, q, w, H, t(gs), True, c, 1.0, c)[0], gk)
    got, x = _operator(k, q, g, w, H, gs, True, c, 1.0, c)
    assert np.allclose(got, gv) and np.allclose(x, g0)


def test_segments_chain():
    # a sequence cut in two, each part's own state from zero, then chained
    B, T, H, D, cut = 1, 9, 2, 3, 4
    q, k, v, _, s, _, w = _inputs(B, T, H, D, 5)
    whole = _operator(q, k, v, w, H, s, False, 1.0, 1.0, 1.0)
    own = _operator(q[:, :cut], k[:, :cut], v[:, :cut], w, H, 0 * s, False, 1.0, 1.0, 1.0)[1]
    mid = np.exp(-w * cut)[None, :, None, None] * s + own
    out, last = _operator(q[:, cut:], k[:, cut:], v[:, cut:], w, H, mid, False, 1.0, 1.0, 1.0)
    assert np.allclose(out, whole[0][:, cut:]) and np.allclose(last, whole[1])


def test_step_equals_the_sequence_form():
    B, T, H, D = 3, 4, 2, 3
    q, k, v, _, s, _, w = _inputs(B, T, H, D, 6)
    out, last, _, _ = seq.decay_attn(q, k, v, w, H, 0.5, s)
    pool = np.zeros((5, H, D, D))
    slots = [4, 0, 2]
    pool[slots] = s
    for t in range(T):
        o, pool, _ = seq.decay_attn_step(q[:, t], k[:, t], v[:, t], w, H, pool, slots, 0.5)
        assert np.allclose(o, out[:, t])
    assert np.allclose(pool[slots], last) and not pool[[1, 3]].any()


def test_layer_norm_gradient_against_central_differences():
    r = np.random.default_rng(7)
    x, g, gamma, beta = r.normal(size=(4, 5)), r.normal(size=(4, 5)), r.normal(size=5), r.normal(size=5)
    _, mean, rstd = seq.layer_norm_fwd(x, gamma, beta, 1e-3)
    (gx, gg, gb), _ = seq.layer_norm_bwd(x, gamma, mean, rstd, g)

    def loss():
        return (seq.layer_norm_fwd(x, gamma, beta, 1e-3)[0] * g).sum()

    eps = 1e-6
    for arr, grad in ((x, gx), (gamma, gg), (beta, gb)):
        flat = arr.ravel()
        for i in range(flat.size):
            old = flat[i]
            flat[i] = old + eps
            up = loss()
            flat[i] = old - eps
            down = loss()
            flat[i] = old
            assert abs((up - down) / (2 * eps) - grad.ravel()[i]) < 1e-7
