"""What decay attention does to numbers: how often it rounds.

Against the float64 oracle, with the names of test_gpu_sequence.py: u = 2^-24,
n operations, A the sum of the absolute values of a result's terms.
"""
import numpy as np
import pytest

from oracle import sequence as seq
from test_gpu_sequence import U, Problem, _dev, _np, _ops, vk  # noqa: F401

pytestmark = pytest.mark.gpu


def _rounded_once(got, want, mag, n):
    """In the 2-norm, no further off than the output's own rounding of a value
    that is off by no more than e = (n u + 1.5 * 2^-16) A: the sums, and two
    bfloat16 parts of the products q.k, the state and the decayed keys.  The
    rounding of a value y is the nearest to it, so it lies at most |x - y| + (how
    far x's own lies from x) from y, and 2 |x - y| + that from x.  A second
    rounding of the same size would make it sqrt(2) times."""
    import torch
    own = np.linalg.norm(_np(torch.from_numpy(want).to(torch.bfloat16)) - want)
    tol = own + 2 * np.linalg.norm((n * U + 1.5 * 2.0 ** -16) * mag)
    assert tol < 1.2 * own                              # the bound can tell the two apart
    off = np.linalg.norm(_np(got) - want)
    assert off <= tol, (off / own, tol / own)


def _positive(B, T, H, D, w, seed):
    """Terms that do not cancel: A is the value itself."""
    p = Problem("bf16", B, T, H, D, seed, state=False, w=w)
    for n in "qkvg":
        t, d = _dev(np.abs(getattr(p, n + "d")), "bf16")
        setattr(p, n, t)
        setattr(p, n + "d", d)
    return p


@pytest.mark.parametrize("B,T,H,D", [(2, 196, 3, 64), (14, 300, 2, 64), (14, 300, 2, 128), (11, 260, 3, 40), (14, 300, 2, 90)])
def test_products_are_not_rounded(vk, B, T, H, D):  # noqa: F811
    """However many rows a call has, the decayed products and keys keep more
    bits than its outputs: each output is its own token's term but for e^-3."""
    p = _positive(B, T, H, D, 3.0, 31)
    n = _ops(D, T)
    want, _, mag, _ = seq.decay_attn(p.qd, p.kd, p.vd, p.wd, H, p.scale)
    for keep in (True, False):
        _rounded_once(p.fwd(vk, want_state=keep)[0], want, mag, n)
    wants, mags = seq.decay_attn_bwd(p.qd, p.kd, p.vd, p.wd, H, p.gd, p.scale)
    for got, want, mag in zip(p.bwd(vk)[:3], wants, mags):
        _rounded_once(got, want, mag, n)


@pytest.mark.parametrize("B,T,H,D", [(14, 300, 2, 64), (14, 300, 2, 128)])
def test_products_are_not_rounded_where_decays_are_factored(vk, B, T, H, D):  # noqa: F811
    """A key every 20 tokens: at w = 1/2 each output is one key's term but for e^-10."""
    p = _positive(B, T, H, D, 0.5, 32)
    keep = np.arange(T) % 20 == 3
    p.k, p.kd = _dev(p.kd * keep[None, :, None], "bf16")
    want, _, mag, _ = seq.decay_attn(p.qd, p.kd, p.vd, p.wd, H, p.scale)
    for state in (True, False):
        _rounded_once(p.fwd(vk, want_state=state)[0], want, mag, _ops(D, T))
