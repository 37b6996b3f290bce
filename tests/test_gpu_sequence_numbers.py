"""What decay attention does to numbers: how often it rounds, and where NaN,
infinities and values at the ends of the range go.

Against the float64 oracle, with the names of test_gpu_sequence.py: u = 2^-24,
n operations, A the sum of the absolute values of a result's terms.  A power of a
decay is off by |w n| u, its exponent's rounding, and exp2f's 2 units, 4 u; a term
has three powers at most, whose 12 u are within the 16 operations that a count
has to spare beside its sums.
"""
import numpy as np
import pytest

import test_gpu_sequence as base
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


NAN, GPU_NAN, INF = 0x7fc00000, 0x7fffffff, 0x7f800000  # float32 bits; arithmetic on the GPU gives the second


def _value(bits, dt):
    """A value of these bits (their upper half in bfloat16)."""
    import torch
    t = torch.tensor([bits if dt == "f32" else bits >> 16], device="cuda")
    return t.to(torch.int32).view(torch.float32) if dt == "f32" else t.to(torch.int16).view(torch.bfloat16)


KERNELS = [("f32", 9, 200), ("f32", 64, 33), ("f32", 128, 150), ("bf16", 20, 150), ("bf16", 64, 16),  # any size
           ("f32", 64, 300), ("bf16", 64, 300), ("bf16", 128, 300), ("bf16", 45, 300),               # tcgen05
           ("f32", 128, 2000), ("bf16", 20, 2000), ("f32", 64, 2000), ("bf16", 64, 2000), ("bf16", 128, 2000)]  # cut


def _all_bad(t):
    import torch
    return not torch.isfinite(t).any()


@pytest.mark.parametrize("bits", [NAN, GPU_NAN, INF])
@pytest.mark.parametrize("dt,D,T", KERNELS)
def test_what_is_not_finite_stays_so(vk, dt, D, T, bits):  # noqa: F811
    """One NaN or infinity among the valid tokens.  With w = 0.01, no term decays to 0
    and no value is 0, so it reaches all that the recurrence leads it to.  In q it
    reaches its row of out and, through q^T g, the column it is in of G_t, t <= its
    own, and so on."""
    import torch
    at, c = T // 2, D + 2                                # a token, and a channel: head 1, its channel 2
    for name in "qkvg":
        p = Problem(dt, 1, T, 2, D, 33, w=0.01)
        clean_out, clean_last = p.fwd(vk)
        getattr(p, name)[0, at, c] = _value(bits, dt)
        out, last = (t.clone() for t in p.fwd(vk))
        gq, gk, gv, gs = p.bwd(vk)
        o, grads = out[0].view(T, 2, D), [t[0].view(T, 2, D) for t in (gq, gk, gv)]
        assert torch.equal(o[:, 0], clean_out[0].view(T, 2, D)[:, 0])  # the other head does not see it
        for t in grads:
            assert torch.isfinite(t[:, 0]).all()
        if name == "q":                                  # out_t = q_t S_t; G_s = .. + q_t^T g_t for s <= t
            assert _all_bad(o[at, 1]) and torch.isfinite(o[at + 1:, 1]).all() and torch.isfinite(last).all()
            assert _all_bad(gs[0, 1, 2]) and _all_bad(grads[1][:at + 1, 1, 2]) and _all_bad(grads[2][:at + 1, 1])
        if name == "k":                                  # row 2 of S_t, t >= its own
            assert _all_bad(o[at:, 1]) and _all_bad(last[0, 1, 2])
            assert _all_bad(grads[0][at:, 1, 2]) and _all_bad(grads[2][at, 1])
        if name == "v":                                  # column 2 of S_t, t >= its own
            assert _all_bad(o[at:, 1, 2]) and _all_bad(last[0, 1, :, 2])
            assert _all_bad(grads[0][at:, 1]) and _all_bad(grads[1][at, 1])
        if name == "g":                                  # column 2 of G_t, t <= its own
            assert _all_bad(grads[0][at, 1]) and _all_bad(gs[0, 1, :, 2])
            assert _all_bad(grads[1][:at + 1, 1]) and _all_bad(grads[2][:at + 1, 1, 2])
    vk.device_status()


@pytest.mark.parametrize("bits", [NAN, GPU_NAN, INF])
@pytest.mark.parametrize("dt,D,T", KERNELS)
def test_states_and_decays_that_are_not_finite(vk, dt, D, T, bits):  # noqa: F811
    """One in the state before the first token, in the gradient of the one after the
    last, and a decay that is NaN."""
    import torch
    p = Problem(dt, 1, T, 2, D, 34, w=0.01)
    p.s[0, 1, 3, 2] = _value(bits, "f32")
    out, last = p.fwd(vk)
    assert _all_bad(out[0].view(T, 2, D)[:, 1, 2]) and not torch.isfinite(last[0, 1, 3, 2])
    assert torch.isfinite(out[0].view(T, 2, D)[:, 0]).all() and torch.isfinite(last[0, 0]).all()
    assert _all_bad(p.bwd(vk)[0][0].view(T, 2, D)[:, 1, 3])
    p = Problem(dt, 1, T, 2, D, 35, w=0.01)
    p.gs[0, 1, 3, 2] = _value(bits, "f32")
    gq, gk, gv, gs = (None if t is None else t[0] for t in p.bwd(vk))
    assert _all_bad(gk.view(T, 2, D)[:, 1, 3]) and _all_bad(gv.view(T, 2, D)[:, 1, 2]) and not torch.isfinite(gs[1, 3, 2])
    assert torch.isfinite(gq).all() and all(torch.isfinite(t.view(T, 2, D)[:, 0]).all() for t in (gk, gv))
    if bits != INF:
        p = Problem(dt, 1, T, 2, D, 36)
        p.w[1] = _value(bits, "f32")
        out, last = p.fwd(vk)
        grads = p.bwd(vk)
        # (gk and gv of the last token and, without a state, gq and out of the first hold no decay)
        assert _all_bad(out[0].view(T, 2, D)[:, 1]) and _all_bad(last[0, 1]) and _all_bad(grads[3][0, 1])
        assert all(_all_bad(t[0].view(T, 2, D)[1:-1, 1]) for t in grads[:3])
        assert torch.isfinite(out[0].view(T, 2, D)[:, 0]).all()
    vk.device_status()


@pytest.mark.parametrize("D,T", [(9, 100), (64, 64), (128, 200)])
def test_largest_float32_values(vk, D, T):  # noqa: F811
    """Values up to the type's largest, in v, where the state and the result are far
    below it.  The parts leave out 2^-20 of a product, twice in a row."""
    p = Problem("f32", 1, T, 1, D, 37, state=False, w=3.0, scale=2.0 ** -60)
    p.v[0, ::3, ::2] = float(np.finfo(np.float32).max)
    p.vd = _np(p.v)
    p.k *= 2.0 ** -30                                    # the state holds sums of k v
    p.kd = _np(p.k)
    out = p.fwd(vk, want_state=False)[0]
    assert vk.load_library().vrwkv_last_kernel() == b"decay_attn_kernel"
    want, _, mag, _ = seq.decay_attn(p.qd, p.kd, p.vd, p.wd, 1, p.scale)
    assert (np.abs(_np(out) - want) <= (_ops(D, T) * U + 2.0 ** -19) * mag).all()


def test_largest_float32_values_in_three_parts(vk):  # noqa: F811
    """The same on the fifth-generation tensor cores.  Values above 3.3962e38 are
    nearer to 2^128 than to bfloat16's largest, which the first part of three then
    is.  What the parts leave out: 2^-23 of a product, twice in a row."""
    for w in (3.0, 0.2):
        p = Problem("f32", 1, 300, 2, 64, 38, state=False, w=w, scale=2.0 ** -20)
        p.v[0, ::3, ::2] = float(np.finfo(np.float32).max)
        p.vd = _np(p.v)
        p.k *= 2.0 ** -60
        p.kd = _np(p.k)
        for keep in (True, False):
            out, last = p.fwd(vk, want_state=keep)
            assert vk.load_library().vrwkv_last_kernel() == b"decay_attn_tcf_kernel"
            want, S, mag, M = seq.decay_attn(p.qd, p.kd, p.vd, p.wd, 2, p.scale)
            tol = _ops(64, 300) * U + 2.0 ** -22
            assert (np.abs(_np(out) - want) <= tol * mag).all()
            assert last is None or (np.abs(_np(last) - S) <= tol * M).all()


@pytest.mark.parametrize("dt,D,T", [("bf16", 64, 200), ("bf16", 128, 200), ("bf16", 45, 200), ("bf16", 20, 200), ("f32", 64, 200),
                                    ("f32", 9, 200), ("f32", 128, 100), ("bf16", 64, 2000), ("bf16", 128, 2000), ("f32", 64, 2000)])
@pytest.mark.parametrize("scale", [1e-30, 1e-20, -1e-13, 1e20])
def test_scales_of_any_size(vk, dt, D, T, scale):  # noqa: F811
    """Outputs and gradients to the tolerances of ordinary scales.  Slow decays, so
    that factors over a block of tokens lie far apart, and no gradient of the last
    state, beside which G's other terms would not show.  At 1e-30 a part of 2^-24
    of a term is above float32's smallest normal value 1.2e-38."""
    p = Problem(dt, 2, T, 2, D, 39, lens=[T, T // 3], scale=scale, w=np.array([0.02, 0.45]))
    p.gs = p.gsd = None
    p.check_fwd(*p.fwd(vk))
    p.check_bwd(p.bwd(vk))
    vk.device_status()


@pytest.mark.parametrize("dt,rows,C", [("f32", 700, 516), ("f32", 1500, 640), ("f32", 50, 772), ("f32", 1300, 896), ("bf16", 1500, 640),
                                       ("bf16", 700, 520)])
def test_layer_norm_widths(vk, dt, rows, C):  # noqa: F811
    """Rows narrower than the kernel they go to, more of them than CTAs."""
    base.test_layer_norm(vk, dt, rows, C)


def test_wait_limits_do_not_count_the_pass_before(vk):  # noqa: F811
    """The states at the cuts take some hundred us on most SMs, while CTAs of the
    outputs' pass are set up on the others: with a limit of 20 us for a wait, these
    still report nothing and give the same bits."""
    import torch
    B, T, H, D = 1, 262144, 12, 64
    torch.manual_seed(40)
    q, k, v = (torch.randn(B, T, H * D, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    w = torch.full((H,), 0.01, device="cuda")
    want = vk.decay_attn_fwd(q, k, v, w, H, D ** -0.5)
    vk.device_status()
    vk.set_wait_limit(2e-5)
    try:
        for _ in range(3):
            got = vk.decay_attn_fwd(q, k, v, w, H, D ** -0.5)
            vk.device_status()
            assert all(torch.equal(a, b) for a, b in zip(want, got))
    finally:
        vk.set_wait_limit(2.0)


def test_a_decay(vk):  # noqa: F811
    """The single token's decay alone: a state of ones and a key of zeros.  A power,
    (|w| + 4) u, and the rounding of the product, u."""
    import torch
    H, D = 400, 8
    w, wd = _dev(np.concatenate([np.exp(np.linspace(-20, 4, H - 3)), [0.0, -0.5, -3.0]]))
    state = torch.ones(1, H, D, D, device="cuda")
    x = torch.zeros(1, H * D, device="cuda")
    vk.decay_attn_step(x, x, x, w, H, state)
    want = np.exp(-wd)[None, :, None, None]
    assert (np.abs(_np(state) - want) <= (np.abs(wd)[None, :, None, None] + 5) * U * 1.001 * want).all()


FIRST_CALLS = """
import torch
import linear_complexity_vision_b200 as vk

torch.manual_seed(41)
H, D = 2, {D}
q, k, v, g = (torch.randn(2, {T}, H * D, device="cuda", dtype=torch.{dtype}) for _ in range(4))
w, gamma = torch.full((H,), 0.1, device="cuda"), torch.ones(H * D, device="cuda")
pool = torch.zeros(2, H, D, D, device="cuda")


def run():
    out, last = vk.decay_attn_fwd(q, k, v, w, H)
    grads = vk.decay_attn_bwd(q, k, v, w, H, g)[:3]
    y, mean, rstd = vk.layer_norm_fwd(out, gamma, gamma)
    pool.zero_()
    one = vk.decay_attn_step(q[:, 0], k[:, 0], v[:, 0], w, H, pool)
    return [out, last, *grads, y, mean, rstd, *vk.layer_norm_bwd(out, gamma, mean, rstd, g), one, pool]


graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    captured = run()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in captured]
assert all(torch.equal(a, b) for a, b in zip(got, run()))
vk.device_status()
print("replayed")
"""


@pytest.mark.parametrize("dtype,D,T", [("bfloat16", 64, 1500), ("float32", 64, 1500), ("bfloat16", 90, 300), ("float32", 20, 40)])
def test_first_calls_may_be_captured(vk, dtype, D, T):  # noqa: F811
    """A process whose very first calls are captured: what the library looks up
    once must not need the stream."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(D=D, T=T, dtype=dtype)], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "replayed" in r.stdout, r.stderr[-2000:]
